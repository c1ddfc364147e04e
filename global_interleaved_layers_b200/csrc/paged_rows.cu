// paged_rows.cu -- rows into and out of a paged KV cache.
//
// Append: row t of the new keys (values) belongs to the sequence b with cu_q[b] <= t and goes
// to position p = cache_seqlens[b] + t - cu_q[b], i.e. slot p mod page_size of page
// block_table[b][p / page_size]. LOCAL keys are rotated for p (pairs (j, j + d/2), angle
// p * base^(-2j/d): "Visual guide to Gemma 4", section "p-RoPE"); a K=V row is stored as it is.
// An e4m3 row holds x / s rounded to nearest even, s = 2^k the smallest power of two with
// max|x| <= 448 s. Being a power of two, s changes no mantissa: the division and the later
// product are exact, so a row read back in bf16 has only e4m3's rounding in it (half a step,
// 2^-4 of the value), and the kernels that read the pages may fold s into a product.
// Gather is the way back: code * s.
//
// Both are bound by HBM for long chunks and by latency for a decode step's few rows: launch,
// instruction fetch (the kernels are kept small for it) and the chain from a row to its sequence,
// length, page and data. A group of d / 16 lanes owns a row's 4 heads of one tensor, 16 elements
// a lane and head in two runs of 8 that hold both members of 8 pairs; the heads share the row's
// place and angles and have their loads in flight together, and a maximum is a shuffle within
// the group. Whole warps are filled for every head dim.
// Measured (cold L2): append and gather of a decode step, 64 sequences x 16 KV heads x 256 dims, K
// and V, e4m3: 8 and 6 us; of 1,000 to 8,191 tokens of six sequences, K=V of 4 x 512: 20 and 17 us
// (4.6 and 5.4 TB/s); gather of three whole sequences, 53k tokens of 16 x 256, 206 to 213 us by the card
// (5.3 to 5.5 TB/s).
// A head at a time (the loads of one in flight) the last two took 43 and 233 us.
#include "paged.h"

namespace gattn {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowHeads = 4;      // heads of a group of lanes

__device__ __forceinline__ void bf8_to_f32(const uint4& w, float* f) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(ws[k] << 16);
    f[2 * k + 1] = __uint_as_float(ws[k] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32_to_bf8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Two floats to two e4m3 codes (nearest even, saturating), `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 f32_to_e4m3x8(const float* f) {
  return make_uint2(e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16, e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16);
}

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
  uint32_t h0, h1;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(h0), "=r"(h1) : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&h1));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// The row scale for a largest magnitude `amax`, and its reciprocal: 448 = 0.875 * 2^9, so with
// amax = m * 2^e, m in [0.5, 1), the smallest k with amax <= 448 * 2^k is e - 9 for
// m <= 0.875 and e - 8 above. k >= -126 keeps both powers normal. Zero rows: 1.
__device__ __forceinline__ float row_scale(float amax, float* inv) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7F800000u) {  // an infinity or a NaN among the row's elements
    *inv = 0.f;
    return __uint_as_float(0x7FC00000u);
  }
  if (u == 0u) {
    *inv = 1.f;
    return 1.f;
  }
  // biased exponent field E: amax = 1.f * 2^(E - 127), so e = E - 126; subnormals clamp below
  const int E = (int)(u >> 23);
  int k = E - 126 - ((u & 0x7FFFFFu) <= 0x600000u ? 9 : 8);
  if (k < -126) k = -126;
  *inv = __uint_as_float((uint32_t)(127 - k) << 23);  // k <= 120, k >= -126: exponents 7 .. 253
  return __uint_as_float((uint32_t)(127 + k) << 23);
}

// Sequence of row t, as seq_of_row, by a group of G lanes (of whole warps that call together): G
// probes a step instead of one, since each step costs a memory latency.
__device__ __forceinline__ int group_seq_of_row(const int32_t* cu, int batch, int t, int G) {
  const int lane = threadIdx.x & 31, in_group = lane & (G - 1), first = lane - in_group;
  const uint32_t mine = (G == 32 ? 0xffffffffu : (1u << G) - 1u) << first;
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (__any_sync(0xffffffffu, hi - lo > 1)) {
    const int step = (hi - lo + G) / (G + 1), probe = lo + (in_group + 1) * step;
    const bool le = probe < hi && __ldg(cu + probe) <= t;
    lo += __popc(__ballot_sync(0xffffffffu, le) & mine) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__device__ __noinline__ float2 row_turn(double pos, double inv_freq_turns) {
  float2 r;
  rope_cos_sin(pos, inv_freq_turns, &r.x, &r.y);
  return r;
}

// Place of a row: sequence and position; false when it has none (the status then says why).
__device__ __forceinline__ bool row_place(const PagedCache& c, const int32_t* cu, const int32_t* base, int batch, int t, bool in,
                                          int G, bool first_lane, int* b, int* pos) {
  *b = group_seq_of_row(cu, batch, t, G);
  const int tok0 = __ldg(cu + *b);
  const long long p = (long long)__ldg(base + *b) + (t - tok0);
  *pos = (int)p;
  if (!in || t < tok0) return false;  // past the last row, or before the first sequence
  if (p < 0 || p >= ((long long)c.max_blocks << c.page_shift)) {
    if (first_lane) atomicOr(&g_status, kStatusSeqlen);
    return false;
  }
  return true;
}

}  // namespace

template <bool E4M3>
__global__ void __launch_bounds__(kRowThreads) paged_append_kernel(PagedAppendArgs a) {
  const int d = a.c.d, group = d / 16;              // 4, 8, 16 or 32 lanes: never across a warp
  const bool is_v = blockIdx.y != 0;
  const int hkv = a.c.hkv, hb = (hkv + kRowHeads - 1) / kRowHeads;
  const uint32_t unit = (blockIdx.x * kRowThreads + threadIdx.x) / group;  // (rows that fit in memory number under 2^31)
  const int c8 = ((int)threadIdx.x & (group - 1)) * 8;
  const int t = unit / hb, h0 = (int)(unit - (uint32_t)t * hb) * kRowHeads;
  const bool in = t < min(a.total_q, __ldg(a.cu_q + a.batch));  // lanes past the end stay for the group's shuffles
  int pos, b;
  bool ok = row_place(a.c, a.cu_q, a.lens, a.batch, t, in, group, c8 == 0, &b, &pos);
  uint4 w0[kRowHeads], w1[kRowHeads];
  const uint16_t* src = (is_v ? a.new_v : a.new_k) + ((size_t)t * hkv + h0) * d + c8;
#pragma unroll
  for (int k = 0; k < kRowHeads; ++k) {
    const bool get = ok && h0 + k < hkv;
    w0[k] = get ? __ldg(reinterpret_cast<const uint4*>(src + k * d)) : make_uint4(0u, 0u, 0u, 0u);
    w1[k] = get ? __ldg(reinterpret_cast<const uint4*>(src + k * d + d / 2)) : make_uint4(0u, 0u, 0u, 0u);
  }
  int page = ok ? __ldg(a.c.table + (size_t)b * a.c.max_blocks + (pos >> a.c.page_shift)) : -1;
  float2 turn[8];
  const bool rot = !is_v && ok && c8 < a.r;
  if (rot) {
    double f = a.freq8[c8 / 8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      turn[e] = c8 + e < a.r ? row_turn((double)pos, f) : make_float2(1.f, 0.f);
      f *= a.freq_step;
    }
  }
  if (ok && (unsigned)page >= (unsigned)a.c.num_pages) {
    atomicOr(&g_status, kStatusPage);
    ok = false;
  }
  const size_t dst0 = ok ? page_row(a.c, page, h0, pos & ((1 << a.c.page_shift) - 1)) : 0;
#pragma unroll
  for (int k = 0; k < kRowHeads; ++k) {
    const bool put = ok && h0 + k < hkv;
    const size_t dst = dst0 + ((size_t)k << a.c.page_shift);
    float x0[8], x1[8];
    bf8_to_f32(w0[k], x0);
    bf8_to_f32(w1[k], x1);
    if (rot) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y0 = x0[e] * turn[e].x - x1[e] * turn[e].y;
        x1[e] = x0[e] * turn[e].y + x1[e] * turn[e].x;
        x0[e] = y0;
      }
    }
    if constexpr (E4M3) {
      // as bit patterns, |x| orders like an unsigned integer and NaN above infinity
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        top = max(top, max(__float_as_uint(x0[e]) & 0x7FFFFFFFu, __float_as_uint(x1[e]) & 0x7FFFFFFFu));
#pragma unroll 1
      for (int m = group / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
      float inv;
      const float scale = row_scale(__uint_as_float(top), &inv);
      const bool bad = top >= 0x7F800000u;  // codes of a NaN-scaled row: zero
      // at scale 2^120, 248 .. 255 would round to 256, and 256 * 2^120 is past fp32's range
      const float most = scale == 0x1p120f ? 240.f : 448.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x0[e] = bad ? 0.f : fminf(fmaxf(x0[e] * inv, -most), most);
        x1[e] = bad ? 0.f : fminf(fmaxf(x1[e] * inv, -most), most);
      }
      if (!put) continue;
      uint8_t* out = (is_v ? a.c.v : a.c.k) + dst * d;
      *reinterpret_cast<uint2*>(out + c8) = f32_to_e4m3x8(x0);
      *reinterpret_cast<uint2*>(out + d / 2 + c8) = f32_to_e4m3x8(x1);
      if (c8 == 0) (is_v ? a.c.v_scales : a.c.k_scales)[dst] = scale;
    } else {
      if (!put) continue;
      uint16_t* out = reinterpret_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + dst * d;
      *reinterpret_cast<uint4*>(out + c8) = f32_to_bf8(x0);
      *reinterpret_cast<uint4*>(out + d / 2 + c8) = f32_to_bf8(x1);
    }
  }
}

// Grid of a rows kernel, a tensor per y; 0 blocks: nothing to do.
static cudaError_t rows_grid(const PagedCache& c, int rows, dim3* grid) {
  const long long lanes = (long long)rows * ((c.hkv + kRowHeads - 1) / kRowHeads) * (c.d / 16);
  const long long blocks = (lanes + kRowThreads - 1) / kRowThreads;
  if (lanes / (c.d / 16) > 0x7fffffffll || blocks > 0x00ffffffll) return cudaErrorInvalidValue;
  *grid = dim3((unsigned)blocks, c.v != nullptr ? 2 : 1);
  return cudaSuccess;
}

template <bool E4M3>
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  dim3 grid;
  const cudaError_t e = rows_grid(a.c, a.total_q, &grid);
  if (e != cudaSuccess || grid.x == 0) return e;
  paged_append_kernel<E4M3><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <bool E4M3, bool F32>
__global__ void __launch_bounds__(kRowThreads) paged_gather_kernel(PagedGatherArgs a) {
  const int d = a.c.d, group = d / 16;
  const bool is_v = blockIdx.y != 0;
  const int hkv = a.c.hkv, hb = (hkv + kRowHeads - 1) / kRowHeads;
  const uint32_t unit = (blockIdx.x * kRowThreads + threadIdx.x) / group;
  const int c16 = ((int)threadIdx.x & (group - 1)) * 16;
  const int t = unit / hb, h0 = (int)(unit - (uint32_t)t * hb) * kRowHeads;
  const bool in = t < min(a.total_out, __ldg(a.cu_out + a.batch));
  int pos, b;
  const bool ok = row_place(a.c, a.cu_out, a.starts, a.batch, t, in, group, c16 == 0, &b, &pos);
  if (!in || t < __ldg(a.cu_out + b)) return;
  const int page = ok ? page_of(a.c, b, pos >> a.c.page_shift) : -1;  // rows without a place: zeros
  const size_t src0 = page >= 0 ? page_row(a.c, page, h0, pos & ((1 << a.c.page_shift) - 1)) : 0;
  uint4 w0[kRowHeads], w1[kRowHeads];
  float s[kRowHeads];
#pragma unroll
  for (int k = 0; k < kRowHeads; ++k) {
    w0[k] = w1[k] = make_uint4(0u, 0u, 0u, 0u);
    s[k] = 0.f;
    if (page < 0 || h0 + k >= hkv) continue;
    const size_t src = src0 + ((size_t)k << a.c.page_shift);
    const uint8_t* base = (is_v ? a.c.v : a.c.k) + src * d * (E4M3 ? 1 : 2);
    if constexpr (E4M3) {
      w0[k] = __ldg(reinterpret_cast<const uint4*>(base + c16));
      s[k] = __ldg((is_v ? a.c.v_scales : a.c.k_scales) + src);
    } else {
      w0[k] = __ldg(reinterpret_cast<const uint4*>(base + 2 * c16));
      w1[k] = __ldg(reinterpret_cast<const uint4*>(base + 2 * c16 + 16));
    }
  }
#pragma unroll
  for (int k = 0; k < kRowHeads; ++k) {
    if (h0 + k >= hkv) break;
    float f[16];
    if constexpr (E4M3) {
      const uint32_t ws[4] = {w0[k].x, w0[k].y, w0[k].z, w0[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) e4m3x4_to_f32(ws[i], f + 4 * i);
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] *= s[k];
    } else if constexpr (F32) {
      bf8_to_f32(w0[k], f);
      bf8_to_f32(w1[k], f + 8);
    }
    const size_t dst = ((size_t)t * hkv + h0 + k) * d + c16;
    if constexpr (F32) {
      float* out = static_cast<float*>(is_v ? a.out_v : a.out_k) + dst;
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(out + 4 * i) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
      uint16_t* out = static_cast<uint16_t*>(is_v ? a.out_v : a.out_k) + dst;
      *reinterpret_cast<uint4*>(out) = E4M3 ? f32_to_bf8(f) : w0[k];
      *reinterpret_cast<uint4*>(out + 8) = E4M3 ? f32_to_bf8(f + 8) : w1[k];
    }
  }
}

template <bool E4M3, bool F32>
cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t stream) {
  dim3 grid;
  const cudaError_t e = rows_grid(a.c, a.total_out, &grid);
  if (e != cudaSuccess || grid.x == 0) return e;
  paged_gather_kernel<E4M3, F32><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gattn
