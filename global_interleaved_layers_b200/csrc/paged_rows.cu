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
// Both are bound by HBM for long chunks and by launch latency for a decode step's few rows. A
// group of d / 16 lanes owns one (row, KV head, tensor), 16 elements a lane in two runs of 8 that
// hold both members of 8 pairs: 32 bytes in and 16 (or 32) out per lane, and the row's
// maximum is a shuffle within the group. Whole warps are filled for every head dim.
#include "paged.h"

namespace gattn {

namespace {

constexpr int kRowThreads = 256;

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

}  // namespace

template <bool E4M3>
__global__ void __launch_bounds__(kRowThreads) paged_append_kernel(PagedAppendArgs a) {
  const int d = a.c.d, group = d / 16;              // 4, 8, 16 or 32 lanes: never across a warp
  const int tensors = a.c.v != nullptr ? 2 : 1;
  const long long unit = ((long long)blockIdx.x * kRowThreads + threadIdx.x) / group;
  const int c8 = ((int)threadIdx.x & (group - 1)) * 8;
  const int hkv = a.c.hkv;
  const long long units = (long long)min(a.total_q, __ldg(a.cu_q + a.batch)) * hkv * tensors;
  const bool in = unit < units;  // lanes past the end stay for the group's shuffles
  const long long rest = in ? unit / tensors : 0;
  const bool is_v = in && unit % tensors != 0;
  const int t = (int)(rest / hkv), head = (int)(rest % hkv);
  bool ok = in;
  int pos = 0, b = 0;
  if (in) {
    b = seq_of_row(a.cu_q, a.batch, t);
    const long long p = (long long)__ldg(a.lens + b) + (t - __ldg(a.cu_q + b));
    if (t < __ldg(a.cu_q + b)) {  // before the first sequence
      ok = false;
    } else if (p < 0 || p >= ((long long)a.c.max_blocks << a.c.page_shift)) {
      if (c8 == 0) atomicOr(&g_status, kStatusSeqlen);
      ok = false;
    } else {
      pos = (int)p;
    }
  }
  size_t dst = 0;
  float x0[8] = {}, x1[8] = {};
  if (ok) {
    const int page = page_of(a.c, b, pos >> a.c.page_shift);
    if (page < 0) {
      ok = false;
    } else {
      dst = page_row(a.c, page, head, pos & ((1 << a.c.page_shift) - 1));
      const uint16_t* src = (is_v ? a.new_v : a.new_k) + ((size_t)t * hkv + head) * d;
      bf8_to_f32(__ldg(reinterpret_cast<const uint4*>(src + c8)), x0);
      bf8_to_f32(__ldg(reinterpret_cast<const uint4*>(src + d / 2 + c8)), x1);
    }
  }
  if (!is_v && ok && c8 < a.r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = c8 + e;
      if (j < a.r) {
        float cs, sn;
        rope_cos_sin((double)pos, rope_inv_freq_turns(j, d, a.log2_base), &cs, &sn);
        const float y0 = x0[e] * cs - x1[e] * sn;
        x1[e] = x0[e] * sn + x1[e] * cs;
        x0[e] = y0;
      }
    }
  }
  if constexpr (E4M3) {
    // as bit patterns, |x| orders like an unsigned integer and NaN above infinity
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      top = max(top, max(__float_as_uint(x0[e]) & 0x7FFFFFFFu, __float_as_uint(x1[e]) & 0x7FFFFFFFu));
    for (int m = group / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    float inv;
    const float scale = row_scale(__uint_as_float(top), &inv);
    if (!ok) return;
    const bool bad = top >= 0x7F800000u;  // codes of a NaN-scaled row: zero
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x0[e] = bad ? 0.f : x0[e] * inv;
      x1[e] = bad ? 0.f : x1[e] * inv;
    }
    if (scale == 0x1p120f) {  // 248 .. 255 would round to 256, and 256 * 2^120 is past fp32's range
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x0[e] = fminf(fmaxf(x0[e], -240.f), 240.f);
        x1[e] = fminf(fmaxf(x1[e], -240.f), 240.f);
      }
    }
    uint8_t* out = (is_v ? a.c.v : a.c.k) + dst * d;
    *reinterpret_cast<uint2*>(out + c8) = f32_to_e4m3x8(x0);
    *reinterpret_cast<uint2*>(out + d / 2 + c8) = f32_to_e4m3x8(x1);
    if (c8 == 0) (is_v ? a.c.v_scales : a.c.k_scales)[dst] = scale;
  } else {
    if (!ok) return;
    uint16_t* out = reinterpret_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + dst * d;
    *reinterpret_cast<uint4*>(out + c8) = f32_to_bf8(x0);
    *reinterpret_cast<uint4*>(out + d / 2 + c8) = f32_to_bf8(x1);
  }
}

template <bool E4M3>
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  const long long lanes = (long long)a.total_q * a.c.hkv * (a.c.v ? 2 : 1) * (a.c.d / 16);
  if (lanes == 0) return cudaSuccess;
  const long long blocks = (lanes + kRowThreads - 1) / kRowThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  paged_append_kernel<E4M3><<<(unsigned)blocks, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <bool E4M3, bool F32>
__global__ void __launch_bounds__(kRowThreads) paged_gather_kernel(PagedGatherArgs a) {
  const int d = a.c.d, group = d / 16;
  const int tensors = a.c.v != nullptr ? 2 : 1;
  const long long unit = ((long long)blockIdx.x * kRowThreads + threadIdx.x) / group;
  const int c16 = ((int)threadIdx.x & (group - 1)) * 16;
  const int hkv = a.c.hkv;
  const long long units = (long long)min(a.total_out, __ldg(a.cu_out + a.batch)) * hkv * tensors;
  if (unit >= units) return;
  const long long rest = unit / tensors;
  const bool is_v = unit % tensors != 0;
  const int t = (int)(rest / hkv), head = (int)(rest % hkv);
  const int b = seq_of_row(a.cu_out, a.batch, t);
  if (t < __ldg(a.cu_out + b)) return;  // before the first sequence
  const long long p = (long long)__ldg(a.starts + b) + (t - __ldg(a.cu_out + b));
  int page = -1;
  if (p < 0 || p >= ((long long)a.c.max_blocks << a.c.page_shift)) {
    if (c16 == 0) atomicOr(&g_status, kStatusSeqlen);
  } else {
    page = page_of(a.c, b, (int)(p >> a.c.page_shift));
  }
  float f[16] = {};
  uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
  if (page >= 0) {
    const size_t src = page_row(a.c, page, head, (int)p & ((1 << a.c.page_shift) - 1));
    const uint8_t* base = (is_v ? a.c.v : a.c.k) + src * d * (E4M3 ? 1 : 2);
    if constexpr (E4M3) {
      w0 = __ldg(reinterpret_cast<const uint4*>(base + c16));
      const float s = __ldg((is_v ? a.c.v_scales : a.c.k_scales) + src);
      const uint32_t ws[4] = {w0.x, w0.y, w0.z, w0.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) e4m3x4_to_f32(ws[k], f + 4 * k);
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] *= s;
    } else {
      w0 = __ldg(reinterpret_cast<const uint4*>(base + 2 * c16));
      w1 = __ldg(reinterpret_cast<const uint4*>(base + 2 * c16 + 16));
      if constexpr (F32) {
        bf8_to_f32(w0, f);
        bf8_to_f32(w1, f + 8);
      }
    }
  }
  const size_t dst = ((size_t)t * hkv + head) * d + c16;
  if constexpr (F32) {
    float* out = static_cast<float*>(is_v ? a.out_v : a.out_k) + dst;
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<float4*>(out + 4 * k) = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
  } else {
    uint16_t* out = static_cast<uint16_t*>(is_v ? a.out_v : a.out_k) + dst;
    *reinterpret_cast<uint4*>(out) = E4M3 ? f32_to_bf8(f) : w0;
    *reinterpret_cast<uint4*>(out + 8) = E4M3 ? f32_to_bf8(f + 8) : w1;
  }
}

template <bool E4M3, bool F32>
cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t stream) {
  const long long lanes = (long long)a.total_out * a.c.hkv * (a.c.v ? 2 : 1) * (a.c.d / 16);
  if (lanes == 0) return cudaSuccess;
  const long long blocks = (lanes + kRowThreads - 1) / kRowThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  paged_gather_kernel<E4M3, F32><<<(unsigned)blocks, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gattn
