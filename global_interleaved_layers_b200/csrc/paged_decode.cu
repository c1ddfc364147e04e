// paged_decode.cu -- attention of a few query rows over a paged KV cache (decode, short verify).
//
// The rows of a KV head are (new token, query head of its group), token-major, in groups of 8:
// the N of mma.sync m16n8k16, with 16 keys on M. A CTA takes one group of one (sequence, KV
// head) and one contiguous part of the keys its rows see (split-KV; the parts meet in
// paged_merge_kernel). Each of its warps streams 16-key blocks of its own through a private
// ring of bulk copies and does the whole block alone:
//   1. GLOBAL: the p-RoPE rotation of the block's keys ("Visual guide to Gemma 4", section
//      "p-RoPE") into a copy that only the scores read; the K=V rows as they landed are the
//      values (section "K=V technique"). LOCAL keys were rotated when they were stored.
//   2. S^T = K Q^T;  3. mask and online softmax in registers;  4. O^T += V^T P^T.
// Blocks are aligned to 16 positions, so a block lies in one page (a page holds 16 or more
// positions): one table entry per block, and consecutive page rows. Rows that no query of the
// group sees are not loaded and count as zero, whatever the page holds there.
//
// E4M3 pages: the codes stay codes. Fragments are loaded as bytes and widened to fp16 (exact),
// and the products run in fp16 with fp32 accumulation. Query rows enter in fp16 scaled by a
// power of two that brings their largest magnitude into [2^14, 2^15): a bf16 element keeps
// all its bits down to 2^-21 of the row's largest, and what is lost below is under 2^-39 of
// it. A key's scale multiplies its scores in fp32. A value's scale 2^k is folded into its
// weight: with e = s + k (log2 units), P = 2^(e - max e) is what multiplies the codes, so the
// largest weight is near 1 whatever the scales, and the softmax sum keeps a running maximum of s of its own.
//
// Bound: HBM (each visible row is read once). 16 keys of 512 dims are 16 KB (8 KB in e4m3)
// against 64 mma.sync and, for GLOBAL, the rotation of 16 x r pairs.
#include <algorithm>

#include "paged.h"

namespace gattn {

namespace {

constexpr int kPB = 16;            // keys per block
constexpr int kPR = 8;             // rows per group
constexpr int kPHeader = 1280;     // mbarriers [2][warps][4], abort flag, split size, row scales, merge maxima and sums
constexpr int kPMaxSmem = 227 * 1024;
constexpr int kSplitCostBlocks = 32;  // a CTA's fixed cost in blocks streamed (512 keys: prologue, first copies, merge)

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_16816_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The low / high two e4m3 codes of a word as two fp16.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t h;
  asm("{.reg .b16 l, u; mov.b32 {l, u}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t h;
  asm("{.reg .b16 l, u; mov.b32 {l, u}, %1; cvt.rn.f16x2.e4m3x2 %0, u;}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Row stride in bytes of a staged key / value row: 16 bytes of padding spread ldmatrix rows.
template <int D, bool E4M3>
__host__ __device__ constexpr int page_row_stride() { return D * (E4M3 ? 1 : 2) + 16; }

// Shared-memory carve-up, the same arithmetic on the host and in the kernel.
struct PagedLayout {
  int nsk, nsv;             // key (K=V) and value stages per warp
  int rr2, rst, nwords;     // rotation tables' length, rotated copy's row stride (16-bit), words per key
  uint32_t q, stp, bstp, itf, regions, region, v_off, sc_off, rot_off, ast_off, total;
};

template <int D, bool E4M3>
__host__ __device__ inline PagedLayout paged_layout(bool kv_same, int r, int nw, int nsk, int nsv) {
  PagedLayout L;
  const int rk = kv_same ? r : 0;              // keys rotated here
  const int c16 = (rk + 15) / 16;
  L.nsk = nsk;
  L.nsv = kv_same ? 0 : nsv;
  L.rr2 = 16 * c16;
  L.nwords = 8 * c16;
  L.rst = 2 * c16 * 16 + 8;
  auto up = [](uint32_t x) { return (x + 127u) / 128u * 128u; };
  L.q = kPHeader;
  L.stp = L.q + up(kPR * (D + 8) * 2);
  L.bstp = L.stp + up(L.rr2 * 8);
  L.itf = L.bstp + up(L.rr2 * 8);
  L.regions = L.itf + up(L.rr2 * 8);
  const uint32_t st = kPB * page_row_stride<D, E4M3>();
  L.v_off = nsk * st;
  L.sc_off = L.v_off + L.nsv * st;             // [stages][16] scales
  L.rot_off = L.sc_off + (E4M3 ? (nsk + L.nsv) * 64u : 0u);
  L.ast_off = L.rot_off + (c16 > 0 ? (uint32_t)kPB * L.rst * 2 : 0u);
  L.region = up(L.ast_off + L.nwords * 16);
  const uint32_t merge = (uint32_t)nw * kPR * (D + 4) * 4;
  const uint32_t body = (uint32_t)nw * L.region;
  L.total = L.regions + (body > merge ? body : merge);
  return L;
}

struct PagedRowsCfg {
  int nw, nsk, nsv;
};

// The first form that fits in shared memory: eight warps with two key and two value stages,
// then fewer stages, then four warps. K=V layers have key stages only; in e4m3 a stage is half
// the bytes and a third one fits.
template <int D, bool E4M3>
bool paged_rows_cfg(bool kv_same, int r, PagedRowsCfg* out) {
  static const PagedRowsCfg forms[] = {{8, 4, 4}, {8, 3, 3}, {8, 2, 2}, {8, 2, 1}, {8, 1, 1}, {4, 2, 1}, {4, 1, 1}};
  for (const PagedRowsCfg& f : forms)
    if (paged_layout<D, E4M3>(kv_same, r, f.nw, f.nsk, f.nsv).total <= (uint32_t)kPMaxSmem) {
      *out = f;
      return true;
    }
  return false;
}

// Keys that the rows of tokens [t0, t1) of a sequence with `len` tokens before the chunk see:
// [first, end), and the 16-position blocks [first / 16, ceil(end / 16)).
__device__ __forceinline__ int keys_first(const PagedAttendArgs& a, int len, int t0) {
  return a.is_local ? max(0, len + t0 - a.window + 1) : 0;
}

// Whether a sequence is one that this call serves; others are recorded once and left alone.
__device__ __forceinline__ bool seq_ok(const PagedAttendArgs& a, int tok0, int n, int len) {
  return tok0 >= 0 && n >= 0 && n <= a.max_q && (long long)tok0 + n <= a.total_q && len >= 0 && len <= a.max_len &&
         (long long)len + n <= ((long long)a.c.max_blocks << a.c.page_shift);
}

// Blocks per split, by one warp: candidate c = lane + 1 splits the longest range (in blocks)
// into c; the one with the least rounds x (blocks + fixed cost) over the SMs wins. The same
// value comes out in every CTA and in the merge, from the lengths alone.
__device__ __forceinline__ int blocks_per_split(const PagedAttendArgs& a, int lane) {
  int longest = 1;
  for (int b = lane; b < a.batch; b += 32) {
    const int tok0 = __ldg(a.cu_q + b), n = __ldg(a.cu_q + b + 1) - tok0, len = __ldg(a.lens + b);
    if (n > 0 && !(a.chunk_of && a.chunk_of[b] >= 0) && seq_ok(a, tok0, n, len)) longest = max(longest, (len + n + kPB - 1) / kPB - keys_first(a, len, 0) / kPB);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, m));
  if (a.splits <= 1) return longest;
  const int c = min(lane + 1, a.splits);
  const int T = (longest + c - 1) / c;
  const float invT = 1.f / (float)T;
  long long items = 0;
  for (int b = 0; b < a.batch; ++b) {
    const int tok0 = __ldg(a.cu_q + b), n = __ldg(a.cu_q + b + 1) - tok0, len = __ldg(a.lens + b);
    if (n <= 0 || (a.chunk_of && a.chunk_of[b] >= 0) || !seq_ok(a, tok0, n, len)) continue;
    const int blocks = (len + n + kPB - 1) / kPB - keys_first(a, len, 0) / kPB;
    items += (long long)__float2int_ru((float)blocks * invT) * ((n * a.group + kPR - 1) / kPR);
  }
  const float cost = (float)((items * a.c.hkv + 147) / 148) * (float)(T + kSplitCostBlocks);
  // least cost, the fewest splits of a tie
  unsigned long long key = ((unsigned long long)__float_as_uint(cost) << 32) | (uint32_t)c;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, key, m);
    if (o < key) key = o;
  }
  const int best = (int)(uint32_t)key;
  return (longest + best - 1) / best;
}

}  // namespace

template <int D, bool E4M3, int NW>
__global__ void __launch_bounds__(NW * 32) paged_rows_kernel(PagedAttendArgs a, int nsk, int nsv) {
  constexpr int HALF = D / 2, NKS = D / 16;
  constexpr int RS = page_row_stride<D, E4M3>();   // bytes
  constexpr int STAGE = kPB * RS;
  constexpr int QST = D + 8;                       // 16-bit stride of a query row
  constexpr int RED = D + 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const bool kv_same = a.c.v == nullptr;

  // ---- this CTA's item: (sequence, row group, KV head, split)
  long long idx = blockIdx.x;
  const int split = (int)(idx % a.splits); idx /= a.splits;
  const int kvh = (int)(idx % a.c.hkv); idx /= a.c.hkv;
  const int rg = (int)(idx % a.row_groups);
  const int b = (int)(idx / a.row_groups);
  const int tok0 = __ldg(a.cu_q + b), n = __ldg(a.cu_q + b + 1) - tok0, len = __ldg(a.lens + b);
  const int R = n * a.group;                       // rows of this KV head
  if (n == 0 || (a.chunk_of && a.chunk_of[b] >= 0)) return;
  if (!seq_ok(a, tok0, n, len)) {
    if (tid == 0 && split == 0 && rg == 0 && kvh == 0) atomicOr(&g_status, kStatusSeqlen);
    return;
  }
  const int row0 = rg * kPR;
  if (row0 >= R) return;
  const int t0 = row0 / a.group, t1 = (min(row0 + kPR, R) - 1) / a.group;  // first and last token
  const int first = keys_first(a, len, t0), end = len + t1 + 1;
  const int blk0 = first / kPB, blks = (end + kPB - 1) / kPB - blk0;

  extern __shared__ __align__(128) uint8_t dsm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsm);                   // [NW][4] keys, [NW][4] values
  volatile int* abort_flag = reinterpret_cast<volatile int*>(dsm + 512);
  int* s_per = reinterpret_cast<int*>(dsm + 516);
  float* s_qs = reinterpret_cast<float*>(dsm + 544);                   // [8] query row scales (e4m3)
  float* mg_m = reinterpret_cast<float*>(dsm + 640);                   // [NW][8]
  float* mg_l = mg_m + 64;
  // Splits of this group: at most a.splits, every one of `per` blocks.
  int per = blks;
  if (a.splits > 1) {
    if (warp == 0) {
      const int p = blocks_per_split(a, lane);
      if (lane == 0) *s_per = p;
    }
    __syncthreads();
    per = *s_per;
  }
  const int nsplit = (blks + per - 1) / per;
  if (split >= nsplit) return;
  const int b_lo = split * per, b_hi = min(blks, b_lo + per);

  const int r = a.r;
  const int rk = kv_same ? r : 0;                  // pairs of the keys rotated here
  const int c16 = (rk + 15) / 16;
  const PagedLayout L = paged_layout<D, E4M3>(kv_same, r, NW, nsk, nsv);
  uint16_t* qs = reinterpret_cast<uint16_t*>(dsm + L.q);
  float2* stp = reinterpret_cast<float2*>(dsm + L.stp);
  float2* bstp = reinterpret_cast<float2*>(dsm + L.bstp);
  double* itf = reinterpret_cast<double*>(dsm + L.itf);
  uint8_t* region = dsm + L.regions + (size_t)warp * L.region;
  uint8_t* kst = region;
  uint8_t* vst = region + L.v_off;
  float* scs = reinterpret_cast<float*>(region + L.sc_off);
  uint16_t* rbuf = reinterpret_cast<uint16_t*>(region + L.rot_off);
  float4* ast = reinterpret_cast<float4*>(region + L.ast_off);
  uint64_t* kbar = bars + warp * 4;
  uint64_t* vbar = bars + 32 + warp * 4;
  uint32_t rot_bits = 0;                           // 16-dim steps of the scores that read the rotated copy
  for (int s = 0; s < c16; ++s) rot_bits |= (1u << s) | (1u << (s + HALF / 16));

  // blocks of this warp: b_lo + warp, + NW, ...
  const int my_n = b_hi - b_lo > warp ? (b_hi - b_lo - warp + NW - 1) / NW : 0;

  // Rows [lo, hi) of block `blk` (relative to blk0) that some query of the group sees.
  auto rows_of = [&](int blk, int& lo, int& hi) {
    const int p0 = (blk0 + blk) * kPB;
    lo = max(first - p0, 0);
    hi = min(end - p0, kPB);
  };
  int k_issued = 0, v_issued = 0;                  // blocks whose copies were issued
  // Copies of the key (kv = 0) or value rows of this warp's block `it` into stage `st`; returns
  // whether the table entry was good.
  auto issue = [&](int it, int st, int kv) -> bool {
    const int blk = b_lo + warp + NW * it;
    int lo, hi;
    rows_of(blk, lo, hi);
    const int p0 = (blk0 + blk) * kPB;
    const int page = page_of(a.c, b, p0 >> a.c.page_shift);
    if (page < 0) hi = lo = 0;
    const size_t prow = page < 0 ? 0 : page_row(a.c, page, kvh, p0 & ((1 << a.c.page_shift) - 1));
    uint64_t* bar = kv ? vbar + st : kbar + st;
    ++(kv ? v_issued : k_issued);
    fence_proxy_async_smem();  // earlier generic accesses to this stage come first
    const uint32_t rows = hi > lo ? hi - lo : 0;
    const uint32_t bytes = rows * (D * (E4M3 ? 1 : 2)) + (E4M3 && rows > 0 ? 64u : 0u);
    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
    __syncwarp();
    uint8_t* dst = (kv ? vst : kst) + (size_t)st * STAGE;
    const uint8_t* src = kv ? a.c.v : a.c.k;
    if (lane >= lo && lane < hi)
      bulk_load(dst + lane * RS, src + (prow + lane) * (D * (E4M3 ? 1 : 2)), D * (E4M3 ? 1 : 2), bar);
    if (E4M3 && rows > 0 && lane == 31)
      bulk_load(scs + (kv ? nsk + st : st) * 16, (kv ? a.c.v_scales : a.c.k_scales) + prow, 64, bar);
    return page >= 0;
  };

  if (lane == 0) {
    for (int s = 0; s < nsk; ++s) mbar_init(kbar + s, 1);
    for (int s = 0; s < nsv && !kv_same; ++s) mbar_init(vbar + s, 1);
    fence_barrier_init();
  }
  if (tid == 0) *abort_flag = 0;

  // ---- query rows into shared memory (rows past R are zero), before any copy is in flight
  constexpr int QCH = D / 8;
  for (int i = tid; i < kPR * QCH; i += NW * 32) {
    const int row = i / QCH, c = i % QCH;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (row0 + row < R) {
      const int tk = (row0 + row) / a.group, hh = (row0 + row) % a.group;
      x = __ldg(reinterpret_cast<const uint4*>(a.q + (((size_t)tok0 + tk) * a.hq + kvh * a.group + hh) * D + c * 8));
    }
    *reinterpret_cast<uint4*>(qs + row * QST + c * 8) = x;
  }
  __syncthreads();
  uint32_t bad = 0;  // bit it % 32: the block's table entry was out of range, its rows do not count
  if (my_n > 0 && !issue(0, 0, 0)) bad |= 1u;
  // the first r pairs of every row turned for the row's position, in place
  for (int i = tid; i < min(kPR, R - row0) * r; i += NW * 32) {
    const int row = i / r, j = i % r;
    const float x0 = bf2f(qs[row * QST + j]), x1 = bf2f(qs[row * QST + j + HALF]);
    float c, s;
    rope_cos_sin((double)(len + (row0 + row) / a.group), rope_inv_freq_turns(j, D, a.log2_base), &c, &s);
    qs[row * QST + j] = f2bf(x0 * c - x1 * s);
    qs[row * QST + j + HALF] = f2bf(x0 * s + x1 * c);
  }
  // per pair: frequency, and the turns of one key and of a warp's stride of NW blocks; pairs
  // past rk (they share a 16-dim step with rotated ones) keep still
  for (int j = tid; j < L.rr2; j += NW * 32) {
    const double f = j < rk ? rope_inv_freq_turns(j, D, a.log2_base) : 0.0;
    float c, s;
    rope_cos_sin(1.0, f, &c, &s);
    itf[j] = f;
    stp[j] = make_float2(c, s);
    rope_cos_sin((double)(NW * kPB), f, &c, &s);
    bstp[j] = make_float2(c, s);
  }
  __syncthreads();
  if constexpr (E4M3) {  // bf16 rows to scaled fp16 rows, a warp per row
    for (int row = warp; row < kPR; row += NW) {
      uint32_t top = 0;
      for (int c = lane; c < D / 2; c += 32) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(qs + row * QST + 2 * c);
        top = max(top, max((w & 0x7FFFu) << 16, w & 0x7FFF0000u));
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
      // amax in [2^(E - 127), 2^(E - 126)): multiply by 2^(141 - E); zero and non-finite rows by 1
      const int E = (int)(top >> 23);
      const int k = top == 0u || E == 255 ? 0 : min(max(141 - E, -126), 126);
      const float up = __uint_as_float((uint32_t)(127 + k) << 23);
      for (int c = lane; c < D / 2; c += 32) {
        uint32_t* p = reinterpret_cast<uint32_t*>(qs + row * QST + 2 * c);
        const uint32_t w = *p;
        *p = pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
      }
      if (lane == 0) s_qs[row] = __uint_as_float((uint32_t)(127 - k) << 23);
    }
    __syncthreads();
  }

  // query fragments: held in registers up to 256 dims. e4m3 keys arrive four dims to a
  // thread, so their 16-dim step pairs (4t, 4t + 1) with k = 2t and (4t + 2, 4t + 3) with 2t + 8.
  constexpr bool kQReg = D <= 256;
  uint32_t qf[kQReg ? NKS : 1][2];
  auto qfrag = [&](int s, bool natural, uint32_t& b0, uint32_t& b1) {
    const uint16_t* p = qs + g * QST + s * 16;
    if (E4M3 && !natural) {
      const uint2 w = *reinterpret_cast<const uint2*>(p + 4 * t);
      b0 = w.x;
      b1 = w.y;
    } else {
      b0 = *reinterpret_cast<const uint32_t*>(p + 2 * t);
      b1 = *reinterpret_cast<const uint32_t*>(p + 2 * t + 8);
    }
  };
  if constexpr (kQReg) {
#pragma unroll
    for (int s = 0; s < NKS; ++s) qfrag(s, (rot_bits >> s) & 1u, qf[s][0], qf[s][1]);
  }

  bool row_ok[2];
  int qpos[2];
  float coef[2];  // scores to log2 units
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = row0 + 2 * t + h;
    row_ok[h] = row < R;
    qpos[h] = len + (row < R ? row / a.group : 0);
    coef[h] = a.softmax_scale * 1.4426950408889634f * (E4M3 ? s_qs[2 * t + h] : 1.f);
  }
  // m: running maximum of the scores s (log2 units), l = sum 2^(s - m). For e4m3 the weights
  // of the value codes have a maximum of their own: mv, of s + log2(value scale).
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f}, mv_run[2] = {-INFINITY, -INFINITY};
  float oacc[NKS][4];
#pragma unroll
  for (int mt = 0; mt < NKS; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) oacc[mt][e] = 0.f;

  int st = 0, sv = 0;               // stage of this block's keys and values
  uint32_t kph = 0, vph = 0;        // their phases
  bool ok = true;
  int it = 0;
  for (; it < my_n; ++it) {
    if (it == 0) {  // the rest of the ring, behind the first rows
      if (!kv_same)
        for (int s = 0; s < nsv && s < my_n; ++s) issue(s, s, 1);
      for (int s = 1; s < nsk && s < my_n; ++s)
        if (!issue(s, s, 0)) bad |= 1u << s;
    }
    ok = __all_sync(0xffffffffu, mbar_wait(kbar + st, kph, abort_flag));
    if (!ok) break;
    uint8_t* kd = kst + (size_t)st * STAGE;
    uint8_t* vd = kv_same ? kd : vst + (size_t)sv * STAGE;
    const int blk = b_lo + warp + NW * it;
    int lo, hi;
    rows_of(blk, lo, hi);
    if ((bad >> (it & 31)) & 1u) hi = lo = 0;
    bad &= ~(1u << (it & 31));
    const int pos0 = (blk0 + blk) * kPB;
    auto zero_rows = [&](uint8_t* base) {  // rows that do not count: P = 0 must meet finite values
      for (int i = lane; i < kPB * (RS / 16); i += 32) {
        const int row = i / (RS / 16);
        if (row < lo || row >= hi) *reinterpret_cast<uint4*>(base + row * RS + (i % (RS / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    };
    const bool ragged = lo > 0 || hi < kPB;
    if (kv_same && ragged) zero_rows(kd);

    // ---- 1. rotation of K=V keys for the scores: a lane owns words of two pairs and walks the
    // 16 keys from the angle of the first, stepping by theta_j; that angle is exact every 16th
    // block and otherwise the previous one advanced by the warp's stride.
    if (rk > 0) {
      const bool exact = (it & 15) == 0;
      for (int w = lane; w < L.nwords; w += 32) {
        const int j = 2 * w;
        float4 an;
        if (exact) {
          rope_cos_sin((double)pos0, itf[j], &an.x, &an.y);
          rope_cos_sin((double)pos0, itf[j + 1], &an.z, &an.w);
        } else {
          const float4 pa = ast[w];
          const float4 bs = *reinterpret_cast<const float4*>(bstp + j);
          an = make_float4(pa.x * bs.x - pa.y * bs.y, pa.x * bs.y + pa.y * bs.x,
                           pa.z * bs.z - pa.w * bs.w, pa.z * bs.w + pa.w * bs.z);
        }
        ast[w] = an;
        const float4 sp = *reinterpret_cast<const float4*>(stp + j);
        float ac[2] = {an.x, an.z}, as[2] = {an.y, an.w};
        const float sc[2] = {sp.x, sp.z}, ss[2] = {sp.y, sp.w};
        uint32_t w0[kPB], w1[kPB];
#pragma unroll
        for (int u = 0; u < kPB; ++u) {
          if constexpr (E4M3) {
            w0[u] = *reinterpret_cast<const uint16_t*>(kd + u * RS + j);
            w1[u] = *reinterpret_cast<const uint16_t*>(kd + u * RS + HALF + j);
          } else {
            w0[u] = *reinterpret_cast<const uint32_t*>(kd + u * RS + 2 * j);
            w1[u] = *reinterpret_cast<const uint32_t*>(kd + u * RS + 2 * (HALF + j));
          }
        }
#pragma unroll
        for (int u = 0; u < kPB; ++u) {
          float x00, x01, x10, x11;
          if constexpr (E4M3) {
            const float2 p = unpack_f16x2(e4m3_lo(w0[u])), q = unpack_f16x2(e4m3_lo(w1[u]));
            x00 = p.x; x01 = p.y; x10 = q.x; x11 = q.y;
          } else {
            x00 = __uint_as_float(w0[u] << 16); x01 = __uint_as_float(w0[u] & 0xFFFF0000u);
            x10 = __uint_as_float(w1[u] << 16); x11 = __uint_as_float(w1[u] & 0xFFFF0000u);
          }
          const float y00 = x00 * ac[0] - x10 * as[0], y01 = x01 * ac[1] - x11 * as[1];
          const float y10 = x00 * as[0] + x10 * ac[0], y11 = x01 * as[1] + x11 * ac[1];
          *reinterpret_cast<uint32_t*>(rbuf + u * L.rst + j) = E4M3 ? pack_f16x2(y00, y01) : pack_bf16x2(y00, y01);
          *reinterpret_cast<uint32_t*>(rbuf + u * L.rst + 16 * c16 + j) = E4M3 ? pack_f16x2(y10, y11) : pack_bf16x2(y10, y11);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float nc = ac[e] * sc[e] - as[e] * ss[e];
            as[e] = ac[e] * ss[e] + as[e] * sc[e];
            ac[e] = nc;
          }
        }
      }
      __syncwarp();
    }

    // ---- 2. S^T = K Q^T (four accumulator chains)
    float sacc[4] = {0.f, 0.f, 0.f, 0.f};
    {
      float sch[3][4] = {};
      const uint32_t rbase = smem_u32(rbuf) + (uint32_t)((lane & 15) * L.rst + (lane >> 4) * 8) * 2;
      const uint32_t kbase = smem_u32(kd) + (lane & 15) * RS + (lane >> 4) * 16;
      auto step = [&](int s, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        uint32_t b0, b1;
        if constexpr (kQReg) {
          b0 = qf[s][0];
          b1 = qf[s][1];
        } else {
          qfrag(s, (rot_bits >> s) & 1u, b0, b1);
        }
        float* acc = (s & 3) ? sch[(s & 3) - 1] : sacc;
        if constexpr (E4M3) mma_16816_f16(acc, a0, a1, a2, a3, b0, b1);
        else mma_16816(acc, a0, a1, a2, a3, b0, b1);
      };
      auto rotated = [&](int s) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(rbase + __popc(rot_bits & ((1u << s) - 1u)) * 32, a0, a1, a2, a3);
        step(s, a0, a1, a2, a3);
      };
      if constexpr (E4M3) {
#pragma unroll
        for (int s = 0; s < NKS; s += 2) {  // one load: 16 keys x 32 codes, two steps
          const bool r0 = (rot_bits >> s) & 1u, r1 = (rot_bits >> (s + 1)) & 1u;
          uint32_t w0 = 0, w1 = 0, w2 = 0, w3 = 0;
          if (!(r0 && r1)) ldsm_x4(kbase + s * 16, w0, w1, w2, w3);
          if (r0) rotated(s);
          else step(s, e4m3_lo(w0), e4m3_lo(w1), e4m3_hi(w0), e4m3_hi(w1));
          if (r1) rotated(s + 1);
          else step(s + 1, e4m3_lo(w2), e4m3_lo(w3), e4m3_hi(w2), e4m3_hi(w3));
        }
      } else {
#pragma unroll
        for (int s = 0; s < NKS; ++s) {
          if ((rot_bits >> s) & 1u) {
            rotated(s);
          } else {
            uint32_t a0, a1, a2, a3;
            ldsm_x4(kbase + s * 32, a0, a1, a2, a3);
            step(s, a0, a1, a2, a3);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sacc[e] += (sch[0][e] + sch[1][e]) + sch[2][e];
    }
    // scales of this thread's keys g and g + 8
    float ks[2] = {1.f, 1.f};
    if constexpr (E4M3) {
      ks[0] = scs[st * 16 + g];
      ks[1] = scs[st * 16 + g + 8];
    }
    if (!kv_same) {  // this block's keys are done with: refill their stage
      __syncwarp();
      if (it + nsk < my_n && !issue(it + nsk, st, 0)) bad |= 1u << ((it + nsk) & 31);
    }

    // ---- 3. mask and online softmax; element e: key g + 8 (e >> 1), row 2t + (e & 1)
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = g + 8 * (e >> 1), pos = pos0 + key, h = e & 1;
      const bool vis = row_ok[h] && key >= lo && key < hi && pos <= qpos[h] && (!a.is_local || pos > qpos[h] - a.window);
      sacc[e] = vis ? sacc[e] * coef[h] * ks[e >> 1] : -INFINITY;
      mx[h] = fmaxf(mx[h], sacc[e]);
    }
    auto row_max = [&](float* v) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[h] = fmaxf(v[h], __shfl_xor_sync(0xffffffffu, v[h], 4));
        v[h] = fmaxf(v[h], __shfl_xor_sync(0xffffffffu, v[h], 8));
        v[h] = fmaxf(v[h], __shfl_xor_sync(0xffffffffu, v[h], 16));
      }
    };
    row_max(mx);

    if (!kv_same) {
      ok = __all_sync(0xffffffffu, mbar_wait(vbar + sv, vph, abort_flag));
      if (!ok) break;
      if (ragged) zero_rows(vd);
    }
    uint32_t p01, p23;
    auto rescale = [&](const float* al) {
#pragma unroll
      for (int mt = 0; mt < NKS; ++mt) {
        oacc[mt][0] *= al[0];
        oacc[mt][1] *= al[1];
        oacc[mt][2] *= al[0];
        oacc[mt][3] *= al[1];
      }
    };
    // a running maximum moves only when it is passed by more than 8 (log2 units): weights stay
    // below 2^8, and the accumulators are rarely touched; the decision is warp-uniform
    if constexpr (!E4M3) {
      if (__any_sync(0xffffffffu, mx[0] > m_run[0] + 8.f || mx[1] > m_run[1] + 8.f)) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m_run[h], mx[h]);
          al[h] = mn == -INFINITY ? 1.f : exp2f(m_run[h] - mn);
          m_run[h] = mn;
          l_run[h] *= al[h];
        }
        rescale(al);
      }
      const float ms[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0], m_run[1] == -INFINITY ? 0.f : m_run[1]};
      p01 = pack_bf16x2(exp2f(sacc[0] - ms[0]), exp2f(sacc[1] - ms[1]));  // key g
      p23 = pack_bf16x2(exp2f(sacc[2] - ms[0]), exp2f(sacc[3] - ms[1]));  // key g + 8
      // the sums take the weights as the products see them, rounded to bf16
      l_run[0] += __uint_as_float(p01 << 16) + __uint_as_float(p23 << 16);
      l_run[1] += __uint_as_float(p01 & 0xFFFF0000u) + __uint_as_float(p23 & 0xFFFF0000u);
    } else {
      // log2 of the value scales (powers of two; NaN stays NaN)
      float ev[4], mxv[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float vs = kv_same ? ks[k] : scs[(nsk + sv) * 16 + g + 8 * k];
        const float lv = vs == vs ? (float)((int)(__float_as_uint(vs) >> 23) - 127) : vs;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 2 * k + h;
          ev[e] = sacc[e] == -INFINITY ? -INFINITY : sacc[e] + lv;
          mxv[h] = fmaxf(mxv[h], ev[e]);
        }
      }
      row_max(mxv);
      if (__any_sync(0xffffffffu, mx[0] > m_run[0] + 8.f || mx[1] > m_run[1] + 8.f)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m_run[h], mx[h]);
          l_run[h] *= mn == -INFINITY ? 1.f : exp2f(m_run[h] - mn);
          m_run[h] = mn;
        }
      }
      if (__any_sync(0xffffffffu, mxv[0] > mv_run[0] + 8.f || mxv[1] > mv_run[1] + 8.f)) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(mv_run[h], mxv[h]);
          al[h] = mn == -INFINITY ? 1.f : exp2f(mv_run[h] - mn);
          mv_run[h] = mn;
        }
        rescale(al);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ms = m_run[h] == -INFINITY ? 0.f : m_run[h], mv = mv_run[h] == -INFINITY ? 0.f : mv_run[h];
        l_run[h] += exp2f(sacc[h] - ms) + exp2f(sacc[2 + h] - ms);
        ev[h] = exp2f(ev[h] - mv);
        ev[2 + h] = exp2f(ev[2 + h] - mv);
      }
      p01 = pack_f16x2(ev[0], ev[1]);
      p23 = pack_f16x2(ev[2], ev[3]);
    }
    const uint32_t pb0 = movmatrix_trans(p01);  // B fragment: keys 2t, 2t + 1 of row g
    const uint32_t pb1 = movmatrix_trans(p23);  // keys 2t + 8, 2t + 9

    // ---- 4. O^T += V^T P^T
    if constexpr (E4M3) {
      // A transposed load moves two neighbouring dims of a key at a time: m-tile 2c holds the
      // even dims of the 32 from 32c, m-tile 2c + 1 the odd ones.
      const uint32_t vbase = smem_u32(vd) + ((lane & 7) + ((lane >> 4) << 3)) * RS + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t w[4];
        ldsm_x4_t(vbase + c * 32, w[0], w[1], w[2], w[3]);
        uint32_t ev2[4], od2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = __byte_perm(w[i], 0, 0x3120);  // even dims of both keys, then odd ones
          ev2[i] = e4m3_lo(x);
          od2[i] = e4m3_hi(x);
        }
        mma_16816_f16(oacc[2 * c], ev2[0], ev2[1], ev2[2], ev2[3], pb0, pb1);
        mma_16816_f16(oacc[2 * c + 1], od2[0], od2[1], od2[2], od2[3], pb0, pb1);
      }
    } else {
      const uint32_t vbase = smem_u32(vd) + ((lane & 7) + ((lane >> 4) << 3)) * RS + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int mt = 0; mt < NKS; ++mt) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(vbase + mt * 32, a0, a1, a2, a3);
        mma_16816(oacc[mt], a0, a1, a2, a3, pb0, pb1);
      }
    }
    __syncwarp();  // every lane is done with this block
    if (kv_same) {
      if (it + nsk < my_n && !issue(it + nsk, st, 0)) bad |= 1u << ((it + nsk) & 31);
    } else {
      if (it + nsv < my_n) issue(it + nsv, sv, 1);
      if (++sv == nsv) { sv = 0; vph ^= 1u; }
    }
    if (++st == nsk) { st = 0; kph ^= 1u; }
  }
  // Copies still in flight after an early exit land before the warp moves on. A stage whose
  // last copy was waited for answers at once: its barrier is in the phase after that copy's.
  if (!ok && lane == 0) {
    auto drain = [&](uint64_t* bar, int stages, int issued) {
      for (int k = issued > stages ? issued - stages : 0; k < issued; ++k) {
        const uint32_t par = (uint32_t)(k / stages) & 1u;
        const unsigned long long w0 = globaltimer_ns();
        while (!mbar_try_wait(bar + k % stages, par) && globaltimer_ns() - w0 < kWaitLimitNs) {}
      }
    };
    drain(kbar, nsk, k_issued);
    if (!kv_same) drain(vbar, nsv, v_issued);
  }

  // ---- merge the warps' states
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 4);
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 8);
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 16);
    if (g == 0) {
      mg_m[warp * 8 + 2 * t + h] = m_run[h];
      mg_l[warp * 8 + 2 * t + h] = l_run[h];
    }
  }
  __syncthreads();  // every warp has left its loop: the stages are free
  auto merged = [&](int row, float& M, float& Lsum) {
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mg_m[w * 8 + row]);
    Lsum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = mg_m[w * 8 + row];  // -inf: no finite score, the sum is 0 or NaN
      Lsum += mg_l[w * 8 + row] * (mw == -INFINITY ? 1.f : exp2f(mw - M));
    }
  };
  float* red = reinterpret_cast<float*>(dsm + L.regions);  // [NW][8][D + 4]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float M, Lsum;
    merged(2 * t + h, M, Lsum);
    const float mo = E4M3 ? mv_run[h] : m_run[h];  // the weights' own reference
    const float f = Lsum != Lsum ? Lsum : Lsum > 0.f && mo != -INFINITY ? exp2f(mo - M) / Lsum : 0.f;
    float* dst = red + (size_t)(warp * 8 + 2 * t + h) * RED;
#pragma unroll
    for (int mt = 0; mt < NKS; ++mt) {
      const int d0 = E4M3 ? (mt >> 1) * 32 + 2 * g + (mt & 1) : mt * 16 + g;
      dst[d0] = oacc[mt][h] * f;
      dst[d0 + (E4M3 ? 16 : 8)] = oacc[mt][2 + h] * f;
    }
  }
  __syncthreads();
  const int rows = min(kPR, R - row0);
  const size_t rows_total = (size_t)a.total_q * a.hq;
  const bool direct = nsplit == 1;
  for (int i = tid; i < rows * (D / 4); i += NW * 32) {
    const int row = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(red + (size_t)(w * 8 + row) * RED + c);
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    const int tk = (row0 + row) / a.group, hh = (row0 + row) % a.group;
    const size_t orow = ((size_t)tok0 + tk) * a.hq + kvh * a.group + hh;
    if (!direct) {
      *reinterpret_cast<float4*>(a.partial_o + ((size_t)split * rows_total + orow) * D + c) = acc;
    } else if (a.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + c) = acc;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + c) =
          make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
  }
  if (tid < rows) {
    float M, Lsum;
    merged(tid, M, Lsum);
    const int tk = (row0 + tid) / a.group, hh = (row0 + tid) % a.group;
    const size_t orow = ((size_t)tok0 + tk) * a.hq + kvh * a.group + hh;
    const float v = Lsum != Lsum ? Lsum : Lsum > 0.f ? (M + log2f(Lsum)) * 0.6931471805599453f : -INFINITY;
    if (!direct) a.partial_lse[(size_t)split * rows_total + orow] = v;
    else if (a.lse) a.lse[orow] = v;
  }
}

// ---------------------------------------------------------------------------
// Merge of the splits: out = sum_s exp(lse_s - M) o_s / sum_s exp(lse_s - M). A warp takes 128
// columns of one row, four per lane; rows whose keys were one split were written directly.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) paged_merge_kernel(PagedAttendArgs a) {
  __shared__ int s_per;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const int p = blocks_per_split(a, lane);
    if (lane == 0) s_per = p;
  }
  __syncthreads();
  const int D = a.c.d, chunks = (D + 127) / 128;
  const long long wid = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long rows_total = (long long)a.total_q * a.hq;
  const long long row = wid / chunks;
  if (row >= rows_total) return;
  const int c0 = (int)(wid % chunks) * 128 + lane * 4;
  const int tok = (int)(row / a.hq), head = (int)(row % a.hq);
  if (tok >= __ldg(a.cu_q + a.batch)) return;
  const int b = seq_of_row(a.cu_q, a.batch, tok);
  const int tok0 = __ldg(a.cu_q + b), n = __ldg(a.cu_q + b + 1) - tok0, len = __ldg(a.lens + b);
  if (!seq_ok(a, tok0, n, len) || (a.chunk_of && a.chunk_of[b] >= 0)) return;
  // the row's group of 8, as the attention kernel cut it
  const int r0 = ((tok - tok0) * a.group + head % a.group) / kPR * kPR;
  const int t0 = r0 / a.group, t1 = (min(r0 + kPR, n * a.group) - 1) / a.group;
  const int blks = (len + t1 + 1 + kPB - 1) / kPB - keys_first(a, len, t0) / kPB;
  const int ns = (blks + s_per - 1) / s_per;
  if (ns <= 1) return;
  float mm = -INFINITY;
  bool nan = false;
  for (int s = 0; s < ns; ++s) {
    const float l = a.partial_lse[s * rows_total + row];
    nan |= l != l;
    mm = fmaxf(mm, l);
  }
  float den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < ns; ++s) {
    const float l = a.partial_lse[s * rows_total + row];
    if (l == -INFINITY) continue;
    const float w = nan ? l : __expf(l - mm);
    den += w;
    if (c0 < D) {
      const float4 v = *reinterpret_cast<const float4*>(a.partial_o + (s * rows_total + row) * D + c0);
      acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    }
  }
  if (c0 < D) {
    const float inv = den > 0.f || den != den ? 1.f / den : 0.f;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    const size_t o = (size_t)row * D + c0;
    if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = acc;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  }
  if (c0 == 0 && a.lse) a.lse[row] = den != den ? den : mm == -INFINITY ? -INFINITY : mm + logf(den);
}

// Most splits the grid offers: enough for about four residencies of one CTA per SM, at least 256
// keys each, at most 32 (the candidates of blocks_per_split).
int paged_rows_splits(int batch, int hkv, int row_groups, int max_keys) {
  const long long units = (long long)batch * hkv * row_groups;
  const long long by_grid = (4 * 148 + units - 1) / units;
  return (int)std::max<long long>(1, std::min<long long>(32, std::min<long long>(by_grid, max_keys / 256)));
}

template <int D, bool E4M3, int NW>
static cudaError_t launch_paged_rows_t(const PagedAttendArgs& a, const PagedRowsCfg& f, cudaStream_t stream) {
  const uint32_t smem = paged_layout<D, E4M3>(a.c.v == nullptr, a.r, NW, f.nsk, f.nsv).total;
  cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<D, E4M3, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)a.batch * a.row_groups * a.c.hkv * a.splits;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  paged_rows_kernel<D, E4M3, NW><<<(unsigned)ctas, NW * 32, smem, stream>>>(a, f.nsk, f.nsv);
  return cudaGetLastError();
}

template <int D, bool E4M3>
static cudaError_t launch_paged_rows_d(const PagedAttendArgs& a, cudaStream_t stream) {
  PagedRowsCfg f;
  if (!paged_rows_cfg<D, E4M3>(a.c.v == nullptr, a.r, &f)) return cudaErrorInvalidValue;
  return f.nw == 8 ? launch_paged_rows_t<D, E4M3, 8>(a, f, stream) : launch_paged_rows_t<D, E4M3, 4>(a, f, stream);
}

cudaError_t launch_paged_rows(const PagedAttendArgs& a, bool e4m3, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.c.d) {
    case 64: e = e4m3 ? launch_paged_rows_d<64, true>(a, stream) : launch_paged_rows_d<64, false>(a, stream); break;
    case 128: e = e4m3 ? launch_paged_rows_d<128, true>(a, stream) : launch_paged_rows_d<128, false>(a, stream); break;
    case 256: e = e4m3 ? launch_paged_rows_d<256, true>(a, stream) : launch_paged_rows_d<256, false>(a, stream); break;
    case 512: e = e4m3 ? launch_paged_rows_d<512, true>(a, stream) : launch_paged_rows_d<512, false>(a, stream); break;
    default: return e;
  }
  if (e != cudaSuccess || a.splits <= 1) return e;
  const long long warps = (long long)a.total_q * a.hq * ((a.c.d + 127) / 128);
  paged_merge_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gattn
