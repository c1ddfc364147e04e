// paged_decode.cu -- attention of a few query rows over a paged KV cache (decode, short verify).
//
// The rows of a KV head are (new token, query head of its group), token-major, in groups of 8:
// the N of mma.sync m16n8k16, with 16 keys on M. One group of one (sequence, KV head) and all
// the keys its sequence sees is a unit. A warp streams 16-key blocks through a private ring of
// bulk copies and does each block alone:
//   1. GLOBAL: the p-RoPE rotation of the block's keys ("Visual guide to Gemma 4", section
//      "p-RoPE") into a copy that only the scores read; the K=V rows as they landed are the
//      values (section "K=V technique"). LOCAL keys were rotated when they were stored.
//   2. S^T = K Q^T;  3. mask and online softmax in registers;  4. O^T += V^T P^T.
// Blocks are aligned to 16 positions, so a block lies in one page (a page holds 16 or more
// positions): one table entry per block, and consecutive page rows. Rows that no query of the
// sequence sees are not loaded and count as zero, whatever the page holds there.
//
// Teams. Units go to teams of warps: the eight warps of a CTA, which deal a unit's blocks out in
// turn and merge their states in shared memory, or single warps, which own a unit and need no
// barrier. Filling a unit's ring, turning its query rows and merging cost microseconds, so a
// full batch of window-sized units goes to single warps and a few long ones to CTAs. Where
// units differ in length or do not fill the teams evenly, the blocks of all units are laid end
// to end and cut into equal runs, one per team, whatever unit boundaries they cross
// (paged_merge_kernel joins a cut unit's parts: at most two parts a team).
//
// E4M3 pages: the codes stay codes. Fragments are loaded as bytes and widened to fp16 (exact),
// and the products run in fp16 with fp32 accumulation. Query rows enter in fp16 scaled by a
// power of two that brings their largest magnitude into [2^14, 2^15): a bf16 element keeps
// all its bits down to 2^-21 of the row's largest, and what is lost below is under 2^-39 of
// it; a rotated one is rounded once, from fp32, by at most 2^-11 of itself. A key's scale
// multiplies its scores in fp32. A value's scale 2^k is folded into its weight: with e = s + k (log2
// units), P = 2^(e - max e + 7) is what multiplies the codes, so the largest weight is 2^7 to 2^15
// whatever the scales (rows of zeros: kZeroRowScale), and the softmax sum keeps a running maximum of
// s of its own. fp16's fixed step at the bottom, 2^-24, then leaves a weight off by at most 2^-32 of
// the row's largest (2^-11 of itself above that): a flat tail of a million keys by 2^-12 of the output
// altogether. With the largest weight at 1, a quarter of a million keys at 2^-25 of it were lost, 1 percent.
//
// Bound: HBM (each visible row is read once). 16 keys of 512 dims are 16 KB (8 KB in e4m3)
// against 64 mma.sync and, for GLOBAL, the rotation of 16 x r pairs.
#include <algorithm>

#include "paged.h"

namespace gattn {

namespace {

constexpr int kPB = 16;            // keys per block
constexpr int kPR = 8;             // rows per group
constexpr int kPHeader = 1408;     // mbarriers [2][warps][4], abort flag, run length, row scales, merge maxima and sums
constexpr int kPMaxSmem = 227 * 1024;
constexpr float kRaise = 8.f;      // a running maximum moves when it is passed by more than this (log2 units)
constexpr float kTop16 = 7.f;      // fp16 weights: 2^7 at the running maximum, 2^(7 + 8) < 65504 at most

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
  int rr2, rst, nwords;     // rotation tables' length, rotated copy's row stride (16-bit), words per key
  uint32_t q, q_step, stp, bstp, itf, regions, region, v_off, sc_off, rot_off, ast_off, total;
};

template <int D, bool E4M3>
__host__ __device__ inline PagedLayout paged_layout(const PagedRowsShape& f, bool kv_same, int r) {
  PagedLayout L;
  const int rk = kv_same ? r : 0;              // pairs of the keys rotated here
  const int c16 = (rk + 15) / 16;
  const int nsv = kv_same ? 0 : f.nsv;
  L.rr2 = 16 * c16;
  L.nwords = 8 * c16;
  L.rst = 2 * c16 * 16 + 8;
  auto up = [](uint32_t x) { return (x + 127u) / 128u * 128u; };
  L.q = kPHeader;
  L.q_step = up((uint32_t)f.q_rows * (D + 8) * 2);
  L.stp = L.q + L.q_step * (f.warp_teams ? f.nw : 1);
  L.bstp = L.stp + up(L.rr2 * 8);
  L.itf = L.bstp + up(L.rr2 * 8);
  L.regions = L.itf + up((uint32_t)(r > L.rr2 ? r : L.rr2) * 8);
  const uint32_t st = kPB * page_row_stride<D, E4M3>();
  L.v_off = f.nsk * st;
  L.sc_off = L.v_off + nsv * st;               // [stages][16] scales
  L.rot_off = L.sc_off + (E4M3 ? (f.nsk + nsv) * 64u : 0u);
  L.ast_off = L.rot_off + (c16 > 0 ? (uint32_t)kPB * L.rst * 2 : 0u);
  const uint32_t body = up(L.ast_off + L.nwords * 16), out = up((uint32_t)f.q_rows * (D + 4) * 4);
  // a team's result is staged where its rings were: [rows][D + 4] per warp
  L.region = body > out ? body : out;
  L.total = L.regions + (uint32_t)f.nw * L.region;
  return L;
}

// The first form that fits in shared memory: eight warps with as many stages as fit, then four.
// 64 dims always have eight with four stages (of values too, where they are separate), 256 dims
// eight with one to four; what is left are K=V rows of 512 dims and many rotated pairs.
template <int D, bool E4M3>
bool paged_rows_stages(PagedRowsShape* f, bool kv_same, int r) {
  static const int forms[][2] = {{8, 4}, {8, 3}, {8, 2}, {8, 1}, {4, 2}};
  for (const auto& x : forms) {
    f->nw = x[0];
    f->nsk = f->nsv = x[1];
    if (paged_layout<D, E4M3>(*f, kv_same, r).total <= (uint32_t)kPMaxSmem) return true;
  }
  return false;
}

// Oldest position that the token t0 after `len` earlier ones sees.
__device__ __forceinline__ int keys_first(const PagedAttendArgs& a, int len, int t0) {
  return a.is_local ? max(0, len + t0 - a.window + 1) : 0;
}

// Whether a sequence is one that this call serves; others are recorded once and left alone.
__device__ __forceinline__ bool seq_ok(const PagedAttendArgs& a, int tok0, int n, int len) {
  return tok0 >= 0 && n >= 0 && n <= a.max_q && (long long)tok0 + n <= a.total_q && len >= 0 && len <= a.max_len &&
         (long long)len + n <= ((long long)a.c.max_blocks << a.c.page_shift);
}

// ceil(rows / unit_rows) for unit_rows 8 or 40: an eighth, and a fifth of that by its reciprocal.
__device__ __forceinline__ int row_groups_of(int rows, int unit_rows) {
  const uint32_t e = (uint32_t)(rows + unit_rows - 1) >> 3;
  return unit_rows == 8 ? e : __umulhi(e, 0xCCCCCCCDu) >> 2;
}

// Blocks of each unit of sequence b and its number of units; both 0 when it is not served here.
// (Out of line, as everything that runs once per unit: a kernel's loops should stay in the
// instruction caches.)
__device__ __noinline__ void seq_units(const PagedAttendArgs& a, int b, int* blocks, int* units) {
  *blocks = *units = 0;
  if (b >= a.batch) return;
  const int tok0 = fresh(a.cu_q + b), n = fresh(a.cu_q + b + 1) - tok0, len = fresh(a.lens + b);
  if (n <= 0 || (a.chunk_of && a.chunk_of[b] >= 0) || !seq_ok(a, tok0, n, len)) return;
  *blocks = ((len + n + (1 << a.unit_shift) - 1) >> a.unit_shift) - (keys_first(a, len, 0) >> a.unit_shift);
  *units = min(row_groups_of(n * a.group, a.unit_rows), a.row_groups) * a.c.hkv;
}

// By one warp: the total over all sequences of their units (cut = 0) or of their units' blocks,
// and the sequence that holds element `x` of that line, with the total before it. Sequence
// batch when there is none. (In 32 bits: attend_plan refuses longer lines.)
__device__ __noinline__ int line_find(const PagedAttendArgs& a, int lane, int x, int* seq, int* before) {
  int total = 0;
  *seq = a.batch;
  *before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int blocks, units;
    seq_units(a, b0 + lane, &blocks, &units);
    const int w = a.cut ? blocks * units : units;
    int incl = w;
#pragma unroll 1
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += o;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, x >= total + incl - w && x < total + incl);
    if (here) {
      const int l = __ffs(here) - 1;
      *seq = b0 + l;
      *before = total + __shfl_sync(0xffffffffu, incl - w, l);
    }
    total += __shfl_sync(0xffffffffu, incl, 31);
  }
  return total;
}

// Length of a team's run of the line.
__device__ __forceinline__ int run_length(const PagedAttendArgs& a, int total) {
  if (!a.cut) return 1;
  const uint32_t per = ((uint32_t)total + a.teams - 1) / (uint32_t)a.teams;
  return (int)((per + a.run_step - 1) / (uint32_t)a.run_step * a.run_step);
}

// What paged_merge_kernel is to join where `team`'s run ends inside a unit that begins in it:
// {teams the unit runs over, first token, rows of the unit | KV head << 8, first row in the head}.
__device__ __forceinline__ int4 join_of(int teams, int tok0, int rows, int kvh, int row0) {
  return make_int4(teams, tok0, rows | kvh << 8, row0);
}

}  // namespace

template <int D, bool E4M3, int NW, bool WARP_TEAMS>
__global__ void __launch_bounds__(NW * 32) paged_rows_kernel(PagedAttendArgs a, PagedRowsShape f) {
  constexpr int HALF = D / 2, NKS = D / 16;
  constexpr int RS = page_row_stride<D, E4M3>();   // bytes
  constexpr int STAGE = kPB * RS;
  constexpr int QST = D + 8;                       // 16-bit stride of a query row
  constexpr int RED = D + 4;
  constexpr int TW = WARP_TEAMS ? 1 : NW;          // warps of a team
  follow();
  if (a.rest != nullptr && __ldcg(a.rest) == 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tw = WARP_TEAMS ? 0 : warp;            // this warp's place in its team
  const int g = lane >> 2, t = lane & 3;
  const bool kv_same = a.c.v == nullptr;
  const int nsk = f.nsk, nsv = f.nsv;

  extern __shared__ __align__(128) uint8_t dsm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsm);                   // [NW][4] keys, [NW][4] values
  volatile int* abort_flag = reinterpret_cast<volatile int*>(dsm + 512);
  float* s_qs = reinterpret_cast<float*>(dsm + 544) + (WARP_TEAMS ? warp * 8 : 0);  // [team][8] query row scales (e4m3)
  float* mg_m = reinterpret_cast<float*>(dsm + 800);                   // [NW][8]
  float* mg_l = reinterpret_cast<float*>(dsm + 1056);                  // [NW][8]

  const int r = a.r;
  const int rk = kv_same ? r : 0;                  // pairs of the keys rotated here
  const int c16 = (rk + 15) / 16;
  const PagedLayout L = paged_layout<D, E4M3>(f, kv_same, r);
  uint16_t* qs = reinterpret_cast<uint16_t*>(dsm + L.q + (WARP_TEAMS ? warp * L.q_step : 0u));
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

  if (lane == 0) {
    for (int s = 0; s < nsk; ++s) mbar_init(kbar + s, 1);
    for (int s = 0; s < nsv && !kv_same; ++s) mbar_init(vbar + s, 1);
    fence_barrier_init();
  }
  if (tid == 0) *abort_flag = 0;
  if (a.chunk_of == nullptr && blockIdx.x == 0)    // sequences that are not served are recorded here
    for (int b = tid; b < a.batch; b += NW * 32) {
      const int tok0 = fresh(a.cu_q + b), n = fresh(a.cu_q + b + 1) - tok0;
      if (n != 0 && !seq_ok(a, tok0, n, fresh(a.lens + b))) atomicOr(&g_status, kStatusSeqlen);
    }
  // per pair: frequency, and the turns of one key and of a warp's stride of TW blocks; pairs
  // past rk (they share a 16-dim step with rotated ones) keep still
  for (int j = tid; j < max(r, L.rr2); j += NW * 32) {
    const double fr = j < r ? rope_inv_freq_turns(j, D, a.log2_base) : 0.0;
    itf[j] = fr;
    if (j < L.rr2) {
      float c, s;
      rope_cos_sin(1.0, fr, &c, &s);
      stp[j] = make_float2(c, s);
      rope_cos_sin((double)(TW * kPB), fr, &c, &s);
      bstp[j] = make_float2(c, s);
    }
  }
  __syncthreads();

  // ---- this team's run [x, x_end) of the line of blocks (cut) or units
  const int team = WARP_TEAMS ? (int)blockIdx.x * NW + warp : (int)blockIdx.x;
  int b, before, x, x_end, run_len;
  {
    const int total = line_find(a, lane, a.cut ? -1 : team, &b, &before);
    const int run = run_length(a, total);
    x = min((long long)team * run, (long long)total);
    x_end = a.cut ? (int)min((long long)total, (long long)x + run) : total;   // uncut: units team, team + teams, ...
    if (x < x_end && a.cut) line_find(a, lane, x, &b, &before);
    if (a.cut && tw == 0 && lane == 0) a.joins[team] = make_int4(0, 0, 0, 0);
    run_len = run;
  }

  int st = 0, sv = 0;               // stage of the next block's keys and values
  uint32_t kph = 0, vph = 0;        // their phases
  int k_issued = 0, v_issued = 0;   // blocks whose copies were issued
  bool ok = true;

  while (x < x_end && ok) {
    // ---- the piece: blocks [b_lo, b_hi) of one unit
    int blocks, units;
    seq_units(a, b, &blocks, &units);
    if (x - before >= (a.cut ? blocks * units : units)) {  // past this sequence
      line_find(a, lane, x, &b, &before);
      seq_units(a, b, &blocks, &units);
    }
    const int u = a.cut ? (x - before) / blocks : x - before;
    const int b_lo = a.cut ? (x - before) % blocks : 0;
    const int b_hi = a.cut ? min(blocks, x_end - x + b_lo) : blocks;
    const int kvh = u % a.c.hkv, row0 = u / a.c.hkv * kPR;
    const int tok0 = fresh(a.cu_q + b), n = fresh(a.cu_q + b + 1) - tok0, len = fresh(a.lens + b);
    const int rows = min(kPR, n * a.group - row0);
    const int first = keys_first(a, len, 0), end = len + n, blk0 = first / kPB;
    if (a.cut && b_lo == 0 && b_hi < blocks && tw == 0 && lane == 0)
      a.joins[team] = join_of((x + blocks - 1) / run_len - team + 1, tok0, rows, kvh, row0);
    x += a.cut ? b_hi - b_lo : a.teams;

    // blocks of this warp: b_lo + tw, + TW, ...
    const int my_n = b_hi - b_lo > tw ? (b_hi - b_lo - tw + TW - 1) / TW : 0;
    // Page of this warp's block it: lane l holds that of block 32 w + l of the current window w
    // (and of the one before), read from the table by the whole warp at a time.
    int win = -1, pg_cur = -1, pg_old = -1;
    auto page_at = [&](int it) -> int {
      const int w = it >> 5;
      if (w > win) {
        pg_old = pg_cur;
        win = w;
        const int mine = 32 * w + lane;
        pg_cur = mine < my_n ? page_of(a.c, b, ((blk0 + b_lo + tw + TW * mine) * kPB) >> a.c.page_shift) : -1;
      }
      return __shfl_sync(0xffffffffu, w == win ? pg_cur : pg_old, it & 31);
    };
    // Rows [lo, hi) of block `blk` (relative to blk0) that some query of the sequence sees.
    auto rows_of = [&](int blk, int& lo, int& hi) {
      const int p0 = (blk0 + blk) * kPB;
      lo = max(first - p0, 0);
      hi = min(end - p0, kPB);
    };
    // Copies of the key (kv = 0) or value rows of this warp's block `it` into stage `stage`.
    auto issue = [&](int it, int stage, int kv) {
      const int blk = b_lo + tw + TW * it;
      int lo, hi;
      rows_of(blk, lo, hi);
      const int p0 = (blk0 + blk) * kPB;
      const int page = page_at(it);
      if (page < 0) hi = lo = 0;
      const size_t prow = page < 0 ? 0 : page_row(a.c, page, kvh, p0 & ((1 << a.c.page_shift) - 1));
      uint64_t* bar = kv ? vbar + stage : kbar + stage;
      ++(kv ? v_issued : k_issued);
      fence_proxy_async_smem();  // earlier generic accesses to this stage come first
      const uint32_t cnt = hi > lo ? hi - lo : 0;
      const uint32_t bytes = cnt * (D * (E4M3 ? 1 : 2)) + (E4M3 && cnt > 0 ? 64u : 0u);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      uint8_t* dst = (kv ? vst : kst) + (size_t)stage * STAGE;
      const uint8_t* src = kv ? a.c.v : a.c.k;
      if (lane >= lo && lane < hi)
        bulk_load(dst + lane * RS, src + (prow + lane) * (D * (E4M3 ? 1 : 2)), D * (E4M3 ? 1 : 2), bar);
      if (E4M3 && cnt > 0 && lane == 31)
        bulk_load(scs + (kv ? nsk + stage : stage) * 16, (kv ? a.c.v_scales : a.c.k_scales) + prow, 64, bar);
    };

    if constexpr (!WARP_TEAMS) __syncthreads();  // the last piece's results have left the rings' place
    else __syncwarp();

    // ---- query rows, a warp per row: loaded, turned (the first r pairs, for the row's position),
    // for e4m3 scaled to fp16, and stored. The loads are made before any copy of this piece is in
    // flight: queued behind the copies of the GPU's other warps they would take microseconds.
    constexpr int QI = (HALF + 63) / 64;         // words of two pairs per lane and half row
    for (int row = tw; row < rows; row += TW) {
      const int tk = (row0 + row) / a.group, hh = (row0 + row) % a.group;
      const uint16_t* src = a.q + (((size_t)tok0 + tk) * a.hq + kvh * a.group + hh) * D;
      uint32_t w0[QI], w1[QI];
#pragma unroll
      for (int i = 0; i < QI; ++i) {
        const int j = 2 * lane + 64 * i;
        w0[i] = w1[i] = 0u;
        if (j < HALF) {
          w0[i] = fresh(reinterpret_cast<const uint32_t*>(src + j));
          w1[i] = fresh(reinterpret_cast<const uint32_t*>(src + HALF + j));
        }
      }
      // x0, x1: the row's elements in fp32, rotated. They are rounded once: to bf16, or scaled to fp16
      float x0[QI][2], x1[QI][2];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < QI; ++i) {
        const int j = 2 * lane + 64 * i;
        x0[i][0] = __uint_as_float(w0[i] << 16);
        x0[i][1] = __uint_as_float(w0[i] & 0xFFFF0000u);
        x1[i][0] = __uint_as_float(w1[i] << 16);
        x1[i][1] = __uint_as_float(w1[i] & 0xFFFF0000u);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (j + e < r) {
            float c, s;
            rope_cos_sin((double)(len + tk), itf[j + e], &c, &s);
            const float y0 = x0[i][e] * c - x1[i][e] * s;
            x1[i][e] = x0[i][e] * s + x1[i][e] * c;
            x0[i][e] = y0;
          }
          if (E4M3) top = max(top, max(__float_as_uint(x0[i][e]) & 0x7FFFFFFFu, __float_as_uint(x1[i][e]) & 0x7FFFFFFFu));
        }
      }
      if constexpr (E4M3) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
        // the largest magnitude is in [2^(E - 127), 2^(E - 126)): multiply by 2^(141 - E); zero
        // and non-finite rows by 1
        const int E = (int)(top >> 23);
        const int k = top == 0u || E == 255 ? 0 : min(max(141 - E, -126), 126);
        const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          w0[i] = pack_f16x2(x0[i][0] * up, x0[i][1] * up);
          w1[i] = pack_f16x2(x1[i][0] * up, x1[i][1] * up);
        }
        if (lane == 0) s_qs[row] = __uint_as_float((uint32_t)(127 - k) << 23);
      } else {
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          w0[i] = pack_bf16x2(x0[i][0], x0[i][1]);
          w1[i] = pack_bf16x2(x1[i][0], x1[i][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < QI; ++i) {
        const int j = 2 * lane + 64 * i;
        if (j < HALF) {
          *reinterpret_cast<uint32_t*>(qs + row * QST + j) = w0[i];
          *reinterpret_cast<uint32_t*>(qs + row * QST + HALF + j) = w1[i];
        }
      }
    }
    if (my_n > 0) issue(0, st, 0);
    if constexpr (!WARP_TEAMS) __syncthreads();
    else __syncwarp();

    // query fragments: held in registers up to 256 dims. e4m3 keys arrive four dims to a
    // thread, so their 16-dim step pairs (4t, 4t + 1) with k = 2t and (4t + 2, 4t + 3) with 2t + 8.
    constexpr bool kQReg = D <= 256;
    uint32_t qf[kQReg ? NKS : 1][2];
    auto qfrag = [&](int s, bool natural, uint32_t& b0, uint32_t& b1) {
      const uint16_t* p = qs + g * QST + s * 16;
      b0 = b1 = 0u;
      if (g < rows) {
        if (E4M3 && !natural) {
          const uint2 w = *reinterpret_cast<const uint2*>(p + 4 * t);
          b0 = w.x;
          b1 = w.y;
        } else {
          b0 = *reinterpret_cast<const uint32_t*>(p + 2 * t);
          b1 = *reinterpret_cast<const uint32_t*>(p + 2 * t + 8);
        }
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
      const int row = 2 * t + h;
      row_ok[h] = row < rows;
      qpos[h] = len + (row < rows ? (row0 + row) / a.group : 0);
      coef[h] = a.softmax_scale * 1.4426950408889634f * (E4M3 && row < rows ? s_qs[row] : 1.f);
    }
    // m: running maximum of the scores s (log2 units), l = sum 2^(s - m). For e4m3 the weights
    // of the value codes have a maximum of their own: mv, of s + log2(value scale).
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f}, mv_run[2] = {-INFINITY, -INFINITY};
    float oacc[NKS][4];
#pragma unroll
    for (int mt = 0; mt < NKS; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[mt][e] = 0.f;

    if (my_n > 0) {  // the rest of the ring, behind the first rows
      if (!kv_same)
        for (int s = 0; s < nsv && s < my_n; ++s) issue(s, (sv + s) % nsv, 1);
      for (int s = 1; s < nsk && s < my_n; ++s) issue(s, (st + s) % nsk, 0);
    }
    for (int it = 0; it < my_n; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(kbar + st, kph, abort_flag));
      if (!ok) break;
      uint8_t* kd = kst + (size_t)st * STAGE;
      uint8_t* vd = kv_same ? kd : vst + (size_t)sv * STAGE;
      const int blk = b_lo + tw + TW * it;
      int lo, hi;
      rows_of(blk, lo, hi);
      if (page_at(it) < 0) hi = lo = 0;
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
        if (it + nsk < my_n) issue(it + nsk, st, 0);
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
      // a running maximum moves only when it is passed by more than kRaise: weights stay bounded, and
      // the accumulators are rarely touched; the decision is warp-uniform
      if constexpr (!E4M3) {
        if (__any_sync(0xffffffffu, mx[0] > m_run[0] + kRaise || mx[1] > m_run[1] + kRaise)) {
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
        float ev[4], mxv[2], vs[2];
  #pragma unroll
        for (int k = 0; k < 2; ++k) vs[k] = kv_same ? ks[k] : scs[(nsk + sv) * 16 + g + 8 * k];
        auto fold = [&]() {
          mxv[0] = mxv[1] = -INFINITY;
  #pragma unroll
          for (int k = 0; k < 2; ++k) {
            // log2 of the value scales (powers of two; NaN stays NaN)
            const float lv = vs[k] == vs[k] ? (float)((int)(__float_as_uint(vs[k]) >> 23) - 127) : vs[k];
  #pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = 2 * k + h;
              ev[e] = sacc[e] == -INFINITY ? -INFINITY : sacc[e] + lv;
              mxv[h] = fmaxf(mxv[h], ev[e]);
            }
          }
          row_max(mxv);
        };
        fold();
        if (__any_sync(0xffffffffu, mx[0] > m_run[0] + kRaise || mx[1] > m_run[1] + kRaise)) {
  #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m_run[h], mx[h]);
            l_run[h] *= mn == -INFINITY ? 1.f : exp2f(m_run[h] - mn);
            m_run[h] = mn;
          }
        }
        if (__any_sync(0xffffffffu, mxv[0] > mv_run[0] + kRaise || mxv[1] > mv_run[1] + kRaise)) {
          if (__any_sync(0xffffffffu, vs[0] == 1.f || vs[1] == 1.f)) {
            // rows of zeros among them? The four lanes of a key look at a quarter of its row each.
  #pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t any = 0;
  #pragma unroll 1
              for (int i = t; i < D / 16; i += 4) {
                const uint4 w = *reinterpret_cast<const uint4*>(vd + (g + 8 * k) * RS + 16 * i);
                any |= w.x | w.y | w.z | w.w;
              }
              any |= __shfl_xor_sync(0xffffffffu, any, 1);
              any |= __shfl_xor_sync(0xffffffffu, any, 2);
              if (vs[k] == 1.f && (any & 0x7F7F7F7Fu) == 0) vs[k] = kZeroRowScale;
            }
            fold();
          }
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
          ev[h] = exp2f((ev[h] - mv) + kTop16);
          ev[2 + h] = exp2f((ev[2 + h] - mv) + kTop16);
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
        if (it + nsk < my_n) issue(it + nsk, st, 0);
      } else {
        if (it + nsv < my_n) issue(it + nsv, sv, 1);
        if (++sv == nsv) { sv = 0; vph ^= 1u; }
      }
      if (++st == nsk) { st = 0; kph ^= 1u; }
    }
    if (!ok) break;

    // ---- the team's result. Row sums first: over the lanes of a row, then over the team's warps.
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
    if constexpr (!WARP_TEAMS) ok = !__syncthreads_or(*abort_flag);  // every warp is done: the rings are free
    else __syncwarp();
    if (!ok) break;
    auto merged = [&](int row, float& M, float& Lsum) {
      M = -INFINITY;
#pragma unroll
      for (int w = 0; w < TW; ++w) M = fmaxf(M, mg_m[(warp - tw + w) * 8 + row]);
      Lsum = 0.f;
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        const float mw = mg_m[(warp - tw + w) * 8 + row];  // -inf: no finite score, the sum is 0 or NaN
        Lsum += mg_l[(warp - tw + w) * 8 + row] * (mw == -INFINITY ? 1.f : exp2f(mw - M));
      }
    };
    float* red = reinterpret_cast<float*>(region);  // [rows][D + 4], this warp's share
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * t + h >= rows) continue;
      float M, Lsum;
      merged(2 * t + h, M, Lsum);
      const float mo = E4M3 ? mv_run[h] : m_run[h];  // the weights' own reference
      const float fac = Lsum != Lsum ? Lsum : Lsum > 0.f && mo != -INFINITY ? exp2f((mo - M) - (E4M3 ? kTop16 : 0.f)) / Lsum : 0.f;
      float* dst = red + (2 * t + h) * RED;
#pragma unroll
      for (int mt = 0; mt < NKS; ++mt) {
        const int d0 = E4M3 ? (mt >> 1) * 32 + 2 * g + (mt & 1) : mt * 16 + g;
        dst[d0] = oacc[mt][h] * fac;
        dst[d0 + (E4M3 ? 16 : 8)] = oacc[mt][2 + h] * fac;
      }
    }
    if constexpr (!WARP_TEAMS) __syncthreads();
    else __syncwarp();
    const bool whole = b_lo == 0 && b_hi == blocks;
    const size_t slot = (size_t)2 * team + (b_lo == 0 ? 1 : 0);  // of a cut unit's part
    for (int i = tw * 32 + lane; i < rows * (D / 4); i += TW * 32) {
      const int row = i / (D / 4), c = (i % (D / 4)) * 4;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(dsm + L.regions + (size_t)(warp - tw + w) * L.region + (row * RED + c) * 4);
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
      }
      const int tk = (row0 + row) / a.group, hh = (row0 + row) % a.group;
      const size_t orow = ((size_t)tok0 + tk) * a.hq + kvh * a.group + hh;
      if (!whole) {
        *reinterpret_cast<float4*>(a.partial_o + (slot * kPR + row) * D + c) = acc;
      } else if (a.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + c) = acc;
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + c) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
      }
    }
    if (tw * 32 + lane < rows) {
      const int row = tw * 32 + lane;
      float M, Lsum;
      merged(row, M, Lsum);
      const int tk = (row0 + row) / a.group, hh = (row0 + row) % a.group;
      const float v = Lsum != Lsum ? Lsum : Lsum > 0.f ? (M + log2f(Lsum)) * 0.6931471805599453f : -INFINITY;
      if (!whole) a.partial_lse[slot * kPR + row] = v;
      else if (a.lse) a.lse[((size_t)tok0 + tk) * a.hq + kvh * a.group + hh] = v;
    }
  }
  // Copies still in flight after an early exit land before the warp leaves. A stage whose last
  // copy was waited for answers at once: its barrier is in the phase after that copy's.
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
}

// ---------------------------------------------------------------------------
// Join of cut units: out = sum_s exp(lse_s - M) o_s / sum_s exp(lse_s - M) over the teams whose runs
// the unit crosses, in order. A block (or a few) takes the unit that one team's run begins and does
// not end, which the team has left a note of: finding such units again from the lengths cost 20
// to 35 us, mostly instruction fetch. A warp takes 128 columns of one row, four per lane.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) paged_merge_kernel(PagedAttendArgs a) {
  follow();
  if (a.rest != nullptr && __ldcg(a.rest) == 0) return;
  const int lane = threadIdx.x & 31;
  const int4 j = __ldcg(a.joins + blockIdx.x);
  if (j.x == 0) return;
  const int D = a.c.d, ur = a.unit_rows, chunks = (D + 127) / 128;
  const int w0 = blockIdx.x, w1 = w0 + j.x - 1, rows = j.z & 255, kvh = j.z >> 8, row0 = j.w;
#pragma unroll 1
  for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < rows * chunks; i += gridDim.y * 8) {
    const int ri = i / chunks, c0 = i % chunks * 128 + lane * 4, in_head = row0 + ri;  // row within the KV head
    const int tk = in_head / a.group;
    const size_t row = ((size_t)j.y + tk) * a.hq + kvh * a.group + (in_head - tk * a.group);
    auto at = [&](int w) { return ((size_t)2 * w + (w == w0 ? 1 : 0)) * ur + ri; };
    // Up to 32 parts at a time, a lane each; the reference is the largest of those seen so far.
    float mm = -INFINITY, den = 0.f, bad = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int wb = w0; wb <= w1; wb += 32) {
      const float l = wb + lane <= w1 ? __ldcg(a.partial_lse + at(wb + lane)) : -INFINITY;
      if (__any_sync(0xffffffffu, l != l)) bad = NAN;
      float m = fmaxf(mm, l);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
      if (m == -INFINITY) continue;
      const float old = __expf(mm - m), mine = l > -INFINITY ? __expf(l - m) : 0.f;
      mm = m;
      den *= old;
      acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
      const uint32_t live = __ballot_sync(0xffffffffu, l > -INFINITY);  // an empty part's output is not written
      const int count = min(32, w1 - wb + 1);
#pragma unroll 4
      for (int k = 0; k < count; ++k) {
        const float wt = __shfl_sync(0xffffffffu, mine, k);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (((live >> k) & 1u) && c0 < D) v = __ldcg(reinterpret_cast<const float4*>(a.partial_o + at(wb + k) * D + c0));
        den += wt;
        acc.x = fmaf(wt, v.x, acc.x); acc.y = fmaf(wt, v.y, acc.y); acc.z = fmaf(wt, v.z, acc.z); acc.w = fmaf(wt, v.w, acc.w);
      }
    }
    den += bad;
    if (c0 < D) {
      const float inv = den > 0.f || den != den ? 1.f / den : 0.f;
      acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;  // a NaN den makes them NaN
      const size_t o = row * D + c0;
      if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = acc;
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
    if (c0 == 0 && a.lse) a.lse[row] = den != den ? den : mm == -INFINITY ? -INFINITY : mm + logf(den);
  }
}

cudaError_t launch_paged_merge(const PagedAttendArgs& a, cudaStream_t stream) {
  if (a.teams < 2) return cudaSuccess;
  const dim3 grid(a.teams - 1, (a.unit_rows * ((a.c.d + 127) / 128) + 7) / 8);
  return launch_follower(paged_merge_kernel, grid, dim3(256), 0, stream, a);
}

// Teams for a call: `units` units of at most `max_blocks` blocks, `group_rows` rows in a group.
//   Single warps from four units per SM on (head dims to 256, whose query rows fit beside eight
//   rings). Uncut where every unit may go whole: short ones (each of a CTA's warps takes four
//   blocks or fewer: cutting would only add the merge), or window-sized ones that fill the warps'
//   rounds to 80 percent.
//   The tensor-core kernel (paged_tile.cu) takes what it can: head dims from 128, at most 64
//   rotated pairs of K=V keys (128 dims have no more). Measured, tensor-core kernel against this
//   file's, in turn on one card: 64 sequences on a window of 1,024 in e4m3, 136 against 236 us; 8 of 32k
//   keys, 512 dims, 187 against 279; five tokens each of 16 sequences against up to 32k keys in e4m3,
//   128 against 591; one sequence of 100 keys, 256 dims, 12.5 against 10.3, the one place seen where it
//   loses (TMEM, tensor maps and five roles to start for one tile).
//   Its units: 8 rows where all sequences have no more, 40 otherwise: five tokens (four drafted) of eight
//   heads are one unit. Measured at 16 sequences of 1k to 32k keys, K=V of 512 dims, units of 40
//   against units of 8, us: 16 rows 128 against 101 in e4m3, 126 against 128 in bf16; 24 rows 130
//   against 136, 130 against 177; 40 rows 136 against 212, 132 against 280; on a window of 1,024 with
//   256 dims, 16 rows 95 against 132. (8 rows in a unit of 8 take 67 and 87.)
//   More than 64 rows are a chunk (paged_api.cu).
PagedRowsShape paged_rows_shape(int head_dim, bool local, int rotated, int batch, int hkv, int rows, long long keys) {
  PagedRowsShape f{};
  if (head_dim >= 128 && (local || rotated <= 64)) {
    f.tile = 1;
    f.unit_rows = rows <= 8 ? 8 : 40;
    f.row_groups = std::max(1, (rows + f.unit_rows - 1) / f.unit_rows);
    const long long units = (long long)batch * hkv * f.row_groups;
    const long long tiles = keys / 64 + 2, rounds = (units + kSms - 1) / kSms;
    f.cut = tiles > 6 && !(local && units * 5 >= rounds * kSms * 4);
    f.parts = 2 * kSms;
    f.line = units * tiles;
    return f;
  }
  f.unit_rows = kPR;
  f.row_groups = std::max(1, (rows + kPR - 1) / kPR);
  f.q_rows = std::min(kPR, rows);
  const long long units = (long long)batch * hkv * f.row_groups, max_blocks = (keys + kPB - 1) / kPB + 1;
  f.warp_teams = head_dim <= 256 && units >= 4 * kSms ? 1 : 0;
  const long long warps = 8ll * kSms;
  if (f.warp_teams) {
    const long long rounds = (units + warps - 1) / warps;
    f.cut = max_blocks > 4 && !(local && units * 5 >= rounds * warps * 4);
  } else {
    f.cut = max_blocks > 32;
  }
  f.parts = 2 * kSms * (f.warp_teams ? 8 : 1);
  f.line = units * max_blocks;
  return f;
}

template <int D, bool E4M3, int NW>
static cudaError_t launch_paged_rows_t(PagedAttendArgs a, const PagedRowsShape& f, long long units, cudaStream_t stream) {
  static std::atomic<bool> ready[2][64];
  const uint32_t smem = paged_layout<D, E4M3>(f, a.c.v == nullptr, a.r).total;
  const long long ctas = f.warp_teams ? (units + NW - 1) / NW : units;
  const int grid = (int)std::min<long long>(f.cut ? kSms : ctas, kSms);
  a.cut = f.cut;
  a.teams = f.warp_teams ? grid * NW : grid;
  a.run_step = f.warp_teams ? 1 : NW;
  a.unit_rows = kPR;
  a.unit_shift = 4;
  cudaError_t e;
  if constexpr (D <= 256) {
    if (f.warp_teams) {
      e = allow_smem(paged_rows_kernel<D, E4M3, NW, true>, kPMaxSmem, ready[1]);
      if (e != cudaSuccess) return e;
      e = launch_follower(paged_rows_kernel<D, E4M3, NW, true>, dim3(grid), dim3(NW * 32), smem, stream, a, f);
    }
  }
  if (!f.warp_teams) {
    e = allow_smem(paged_rows_kernel<D, E4M3, NW, false>, kPMaxSmem, ready[0]);
    if (e != cudaSuccess) return e;
    e = launch_follower(paged_rows_kernel<D, E4M3, NW, false>, dim3(grid), dim3(NW * 32), smem, stream, a, f);
  }
  if (e != cudaSuccess || !f.cut) return e;
  return launch_paged_merge(a, stream);
}

template <int D, bool E4M3>
static cudaError_t launch_paged_rows_d(const PagedAttendArgs& a, PagedRowsShape f, long long units, cudaStream_t stream) {
  if (!paged_rows_stages<D, E4M3>(&f, a.c.v == nullptr, a.r)) return cudaErrorInvalidValue;
  if constexpr (D == 512)
    if (f.nw == 4) return launch_paged_rows_t<D, E4M3, 4>(a, f, units, stream);
  return f.nw == 8 ? launch_paged_rows_t<D, E4M3, 8>(a, f, units, stream) : cudaErrorInvalidValue;
}

cudaError_t launch_paged_rows(const PagedAttendArgs& a, const PagedRowsShape& f, bool e4m3, cudaStream_t stream) {
  const long long units = (long long)a.batch * a.row_groups * a.c.hkv;
  if (f.tile) return launch_paged_tile(a, f, e4m3, stream);
  switch (a.c.d) {
    case 64: return e4m3 ? launch_paged_rows_d<64, true>(a, f, units, stream) : launch_paged_rows_d<64, false>(a, f, units, stream);
    case 256: return e4m3 ? launch_paged_rows_d<256, true>(a, f, units, stream) : launch_paged_rows_d<256, false>(a, f, units, stream);
    case 512: return e4m3 ? launch_paged_rows_d<512, true>(a, f, units, stream) : launch_paged_rows_d<512, false>(a, f, units, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gattn
