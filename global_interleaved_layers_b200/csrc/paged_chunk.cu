// paged_chunk.cu -- attention of long chunks of new tokens over a paged KV cache, on sm_100a's
// tensor cores (tcgen05 with TMEM accumulators, TMA loads).
//
// The rows of a KV head are (new token, query head of its group), token-major: a 128-row tile
// holds floor(128 / group) tokens with all the heads that share the KV head, so a short chunk
// of a large group still fills tiles, and every row of a tile reads the same keys. A work unit
// is one tile (two tiles in the paired form) of one KV head against a run of 128-key tiles.
// Four launches:
//   chunk_plan_kernel   from the lengths on the device: which sequences are chunks, their tiles,
//                       units cut over long key ranges so that no unit is longer than half a
//                       cluster's share, in order of size (longest first);
//   chunk_side_kernel   what the tensor cores cannot take as it lies: rotated queries, the rotated
//                       64-dim chunks of K=V keys ("Visual guide to Gemma 4", section "p-RoPE"),
//                       e4m3 rows widened to bf16 (exact), and copies of the tiles that the ends
//                       of a sequence's keys cut, with zeros beyond the ends;
//   chunk_kernel        the attention: everything else is loaded by TMA straight from the pages,
//                       one box per page and 64-dim chunk;
//   chunk_merge_kernel  joins the units that were cut (log-sum-exp weights, fixed order).
// The side copies cost bytes once per chunk while the products cost 4 d per row and key: at 256
// rows per KV head and more the copy is a few percent of the call.
//
// chunk_kernel. Warp 0 loads (Q once per unit, then K and V stages through a ring), warp 1 issues
// the MMAs (S = Q K^T into one of two TMEM buffers, O += P V with P in TMEM), warps 2-9 run the
// softmax, two per TMEM lane quadrant, a row per lane and half the columns each, and the
// epilogue. The order S(j), PV(j-1), S(j+1) ... keeps the tensor core on the next scores while
// P(j) is formed. Persistent CTAs (pairs) walk the unit list in snake order. Paired form
// (cta_group::2, head dims >= 128, more than 128 rows): each CTA of a pair owns 128 of 256 rows
// and loads half of every K and V stage, halving the bytes per product. At head dim 512 a unit
// accumulates 256 of the output columns (a 128 x 512 fp32 tile would fill TMEM) and the scores
// are computed by both halves.
// Bound: the tensor pipe for long chunks (scores once more at d = 512); launches and the units' ends
// for short ones. Measured: 2,048 tokens after 29,777, K=V of 512 dims, 32 heads: 4.24 ms in a
// burst (974 TFLOP/s of the visible pairs, 1,460 as executed), 4.85 ms with the clocks that
// repeated calls settle at; three prompts of 700 to 2,100 tokens on a window of 1,024, 256 dims,
// 180 us, of which the side copies take 25, the plan 8, the attention 140 (a unit is ten tiles:
// its fill and its epilogue are a third of it).
#include "paged.h"
#include "tile_plan.h"

namespace gattn {

namespace {

constexpr int kCM = 128;                     // rows per CTA
constexpr int kCN = 128;                     // keys per tile
constexpr int kCThreads = 320;
constexpr int kCChunkBytes = 16384;          // 128 rows x 64 dims
constexpr int kCMaxStages = 16;
constexpr int kCBarBytes = 2048;

// LO: the rotated query chunks keep 16 bits, in two bf16 chunks (hi + lo) whose products add up.
// Rotating makes a bf16 row fp32, and rounding it back would be the largest error of a layer that
// rotates every dim (with the weights' rounding, relative to the outputs 2.1e-3 against 1.1e-3).
// Sliding-window layers have it up to 256 dims; at 512 the second copy does not fit, and
// K=V layers' keys are rounded after the same rotation anyway, of a quarter of the dims.
template <int D, bool PAIR, bool LO>
struct ChunkCfg {
  static constexpr int kDv = D > 256 ? 256 : D;               // output columns per unit
  static constexpr int kParts = D / kDv;
  static constexpr int kQChunks = D / 64;
  static constexpr int kVChunks = kDv / 64;
  static constexpr int kQBytes = (LO ? 2 : 1) * kQChunks * kCChunkBytes;
  // Single: a stage is one 64-dim chunk of 128 keys (K) or one 64-column chunk (V). Pair at
  // d >= 256: four chunks of the CTA's 64 keys, or two column chunks of 128 keys; at 128: half.
  static constexpr int kStageBytes = (PAIR && D >= 256) ? 2 * kCChunkBytes : kCChunkBytes;
  static constexpr int kKeys = PAIR ? 64 : 128;               // keys of a K stage in this CTA
  static constexpr int kKChunkBytes = kKeys * 128;
  static constexpr int kKPerStage = kStageBytes / kKChunkBytes;
  static constexpr int kVPerStage = kStageBytes / kCChunkBytes;
  static constexpr int kKStages = kQChunks / kKPerStage;
  static constexpr int kVStages = (PAIR ? kVChunks / 2 : kVChunks) / kVPerStage;
  static constexpr int kPvN = (PAIR ? 2 : 1) * kVPerStage * 64;
  static constexpr int kRing = 232448 - 1024 - kCBarBytes - kQBytes;
  static constexpr int kStages = kRing / kStageBytes < kCMaxStages ? kRing / kStageBytes : kCMaxStages;
  static constexpr int kSmemData = kQBytes + kStages * kStageBytes;
  static constexpr int kSmemBytes = kSmemData + 1024 + kCBarBytes;
  static_assert(!PAIR || D >= 128, "paired form needs two 64-dim chunks");
  static_assert(kKStages >= 1 && kVStages >= 1 && kStages >= 2 && kPvN <= 256, "ring shape");
};

struct __align__(8) ChunkBars {
  uint64_t q_full, q_empty, o_ready, o_empty, mma_done;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t ring_full[kCMaxStages], ring_empty[kCMaxStages];
  uint64_t xfull[4], xfree[4];
  uint32_t tmem_base;
  int abort_flag;
  float xch[2 * 128];
};
static_assert(sizeof(ChunkBars) <= kCBarBytes, "barrier block");

// Tiles [lo, hi) of 128 positions that the tokens [t0, t1] of a sequence see, `len` tokens
// before the chunk.
__device__ __forceinline__ void chunk_tiles(const PagedAttendArgs& a, int len, int t0, int t1, int* lo, int* hi) {
  *lo = keys_first(a, len, t0) / kCN;
  *hi = (len + t1) / kCN + 1;
}

}  // namespace

// ---------------------------------------------------------------------------
// Plan: one block. All sums are over lengths only, so every call with the same lengths cuts the
// work alike; the order within a size class (and which partial slot a cut unit gets) may vary
// and enters no result.
// ---------------------------------------------------------------------------
namespace {
constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 1024;

// Inclusive scan of v over the block; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, w, m);
      if (lane >= m) w += o;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return v + (warp ? s_warp[warp - 1] : 0);
}
}  // namespace

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(PagedAttendArgs a, ChunkPlan p) {
  __shared__ int s_warp[32];
  __shared__ int s_hist[kPlanBuckets];
  __shared__ int s_slots, s_merges, s_rest;
  __shared__ unsigned long long s_work;
  const int tid = threadIdx.x;
  follow();
  if (tid == 0) {
    s_slots = s_merges = s_rest = 0;
    s_work = 0;
  }
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) s_hist[i] = 0;
  // The workspace is sized for lengths that add up to at most total_q, which seq_ok and
  // prefixes that do not decrease ensure; with one that does, there are no chunks.
  int down = 0;
  for (int b = tid; b < a.batch; b += kPlanThreads) down |= fresh(a.cu_q + b + 1) < fresh(a.cu_q + b);
  down = __syncthreads_or(down);
  // ---- sequences: chunk index, first side tile, first unit
  int chunks = 0, tiles = 0, units = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int is = 0, nt = 0, nu = 0;
    if (b < a.batch) {
      const int tok0 = fresh(a.cu_q + b), n = fresh(a.cu_q + b + 1) - tok0, len = fresh(a.lens + b);
      if (n != 0 && !seq_ok(a, tok0, n, len)) {
        atomicOr(&g_status, kStatusSeqlen);
      } else if (!down && n > 0 && (long long)n * a.group > p.min_rows) {
        int lo, hi;
        chunk_tiles(a, len, 0, n - 1, &lo, &hi);
        is = 1;
        nt = hi - lo;
        nu = (n + p.tokens - 1) / p.tokens;
      } else if (n > 0) {
        s_rest = 1;
      }
    }
    int ti, tt, tu;
    const int ci = block_scan(is, s_warp, &ti), ct = block_scan(nt, s_warp, &tt), cu = block_scan(nu, s_warp, &tu);
    if (b < a.batch) {
      p.chunk_of[b] = is ? chunks + ci - 1 : -1;
      p.tile0[b] = tiles + ct - nt;
      p.unit0[b] = units + cu - nu;
    }
    chunks += ti;
    tiles += tt;
    units += tu;
  }
  if (tid == 0) {
    p.tile0[a.batch] = tiles;
    p.unit0[a.batch] = units;
  }
  __syncthreads();
  // ---- work: key tiles of every unit
  auto unit = [&](int u, int* b, int* qt, int* lo, int* hi) {
    int x = 0, y = a.batch;  // the last sequence with unit0 <= u (sequences without units share a value)
    while (y - x > 1) {
      const int m = (x + y) >> 1;
      if (p.unit0[m] <= u) x = m;
      else y = m;
    }
    *b = x;
    *qt = u - p.unit0[x];
    const int n = fresh(a.cu_q + x + 1) - fresh(a.cu_q + x), t0 = *qt * p.tokens;
    chunk_tiles(a, fresh(a.lens + x), t0, min(t0 + p.tokens, n) - 1, lo, hi);
  };
  unsigned long long mine = 0;
  for (int u = tid; u < units; u += kPlanThreads) {
    int b, qt, lo, hi;
    unit(u, &b, &qt, &lo, &hi);
    mine += hi - lo;
  }
  if (mine) atomicAdd(&s_work, mine);
  __syncthreads();
  // Most tiles of a piece: half a cluster's share of the work, at least four (a cut costs a
  // fp32 tile written and read again). With w = s_work the pieces of units that are cut
  // number under 2 w / most <= 4 clusters / units_x.
  const long long share = ((long long)s_work * p.units_x + 2 * p.clusters - 1) / (2 * p.clusters);
  const int most = (int)max(share, (long long)4);
  auto pieces = [&](int nt) { return nt > most ? (nt + most - 1) / most : 1; };
  for (int u = tid; u < units; u += kPlanThreads) {
    int b, qt, lo, hi;
    unit(u, &b, &qt, &lo, &hi);
    const int nt = hi - lo, ns = pieces(nt), per = (nt + ns - 1) / ns;
    atomicAdd(&s_hist[kPlanBuckets - 1 - min(per, kPlanBuckets - 1)], ns);
  }
  __syncthreads();
  int total;
  {
    const int v = s_hist[tid], incl = block_scan(v, s_warp, &total);
    s_hist[tid] = incl - v;
  }
  __syncthreads();
  for (int u = tid; u < units; u += kPlanThreads) {
    int b, qt, lo, hi;
    unit(u, &b, &qt, &lo, &hi);
    const int nt = hi - lo, ns = pieces(nt), per = (nt + ns - 1) / ns;
    int slot = 0;
    if (ns > 1) {
      slot = atomicAdd(&s_slots, ns);
      p.merges[atomicAdd(&s_merges, 1)] = make_int4(b, qt, slot, ns);
    }
    const int at = atomicAdd(&s_hist[kPlanBuckets - 1 - min(per, kPlanBuckets - 1)], ns);
    for (int s = 0; s < ns; ++s) {
      // ns pieces of at most `per` tiles; rounding may leave a late one empty: it is then skipped
      const int k0 = min(lo + s * per, hi), k1 = min(k0 + per, hi);
      p.list[2 * (at + s)] = make_int4(b, qt, k0, k1);
      p.list[2 * (at + s) + 1] = make_int4(ns > 1 ? slot + s : -1, 0, 0, 0);
    }
  }
  __syncthreads();
  if (tid == 0) {
    p.header[0] = total;
    p.header[1] = s_merges;
    p.header[2] = s_rest;
  }
}

// ---------------------------------------------------------------------------
// Side copies.
// ---------------------------------------------------------------------------
namespace {

// Column of a side copy that holds `dim`, or -1 when its 64-dim chunk is not copied.
__device__ __forceinline__ int chunk_col(uint32_t mask, int dim) {
  const int c = dim >> 6;
  if (!((mask >> c) & 1u)) return -1;
  return __popc(mask & ((1u << c) - 1u)) * 64 + (dim & 63);
}

__device__ __forceinline__ void turn8(const float* x0, const float* x1, const float* c, const float* s, float* y0, float* y1) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y0[e] = x0[e] * c[e] - x1[e] * s[e];
    y1[e] = x0[e] * s[e] + x1[e] * c[e];
  }
}

constexpr int kSideThreads = 256;
constexpr int kSideHeads = 4;    // heads whose loads are in flight together
constexpr int kSideQHeads = 8;   // query heads of an item

}  // namespace

// Threads walk items: 8 pairs (j, j + d/2) of one row in a few heads, whose angles are formed
// once. First the query rows, then the key rows of every tile (those with rotated chunks; with
// e4m3 all), then, for bf16 pages, the tiles that a sequence's ends cut.
template <bool E4M3>
__global__ void __launch_bounds__(kSideThreads) chunk_side_kernel(PagedAttendArgs a, ChunkPlan p) {
  __shared__ double s_freq[256];
  follow();
  const int d = a.c.d, half = d / 2, groups = d / 16, hkv = a.c.hkv;
  for (int j = threadIdx.x; j < half; j += kSideThreads) s_freq[j] = j < a.r ? rope_inv_freq_turns(j, d, a.log2_base) : 0.0;
  __syncthreads();
  const int rot_groups = min(groups, (a.r + 63) / 64 * 8);   // whole 64-dim chunks
  const int qh = (a.hq + kSideQHeads - 1) / kSideQHeads, kh = (hkv + kSideHeads - 1) / kSideHeads;
  const int kg = E4M3 ? groups : rot_groups;
  const long long nq = p.q_mask ? (long long)a.total_q * qh * rot_groups : 0;
  const long long nk = E4M3 || p.k_mask ? (long long)p.tile0[a.batch] * kCN * kh * kg : 0;
  const long long ne = E4M3 ? 0 : (long long)a.batch * 2 * kCN * kh * groups;
  auto angles = [&](int pos, int j0, float* c, float* s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.f;
      s[e] = 0.f;
      if (j0 + e < a.r) rope_cos_sin((double)pos, s_freq[j0 + e], &c[e], &s[e]);
    }
  };
  for (long long i = (long long)blockIdx.x * kSideThreads + threadIdx.x; i < nq + nk + ne; i += (long long)gridDim.x * kSideThreads) {
    if (i < nq) {
      const int g = (int)(i % rot_groups), j0 = 8 * g;
      const int h0 = (int)(i / rot_groups % qh) * kSideQHeads, t = (int)(i / rot_groups / qh);
      if (t >= fresh(a.cu_q + a.batch) || t < fresh(a.cu_q)) continue;
      const int b = seq_of_row(a.cu_q, a.batch, t);
      if (p.chunk_of[b] < 0) continue;
      const int c0 = chunk_col(p.q_mask, j0), c1 = chunk_col(p.q_mask, j0 + half);
      float c[8], s[8];
      angles(fresh(a.lens + b) + t - fresh(a.cu_q + b), j0, c, s);
#pragma unroll 1
      for (int h = h0; h < min(h0 + kSideQHeads, a.hq); h += kSideHeads) {
        const size_t row = (size_t)t * a.hq + h;
        uint4 w0[kSideHeads], w1[kSideHeads];
#pragma unroll
        for (int k = 0; k < kSideHeads; ++k) {
          if (h + k >= a.hq) break;
          w0[k] = fresh(reinterpret_cast<const uint4*>(a.q + (row + k) * d + j0));
          w1[k] = fresh(reinterpret_cast<const uint4*>(a.q + (row + k) * d + j0 + half));
        }
#pragma unroll
        for (int k = 0; k < kSideHeads; ++k) {
          if (h + k >= a.hq) break;
          float x0[8], x1[8], y0[8], y1[8];
          bf8_to_f32(w0[k], x0);
          bf8_to_f32(w1[k], x1);
          turn8(x0, x1, c, s, y0, y1);
          uint16_t* dst = p.q_side + (row + k) * (p.q_lo ? 2 * p.q_cols : p.q_cols);
          const uint4 hi0 = f32_to_bf8(y0), hi1 = f32_to_bf8(y1);
          if (c0 >= 0) *reinterpret_cast<uint4*>(dst + c0) = hi0;
          if (c1 >= 0) *reinterpret_cast<uint4*>(dst + c1) = hi1;
          if (!p.q_lo) continue;
          // what the rounding left; nothing beside an infinity, which says all
          float h0[8], h1[8];
          bf8_to_f32(hi0, h0);
          bf8_to_f32(hi1, h1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y0[e] = fabsf(h0[e]) < INFINITY ? y0[e] - h0[e] : 0.f;
            y1[e] = fabsf(h1[e]) < INFINITY ? y1[e] - h1[e] : 0.f;
          }
          if (c0 >= 0) *reinterpret_cast<uint4*>(dst + p.q_cols + c0) = f32_to_bf8(y0);
          if (c1 >= 0) *reinterpret_cast<uint4*>(dst + p.q_cols + c1) = f32_to_bf8(y1);
        }
      }
      continue;
    }
    const bool edges = i >= nq + nk;
    const long long ik = edges ? i - nq - nk : i - nq;
    const int gs = edges ? groups : kg;
    const int g = (int)(ik % gs), j0 = 8 * g, h = (int)(ik / gs % kh) * kSideHeads;
    const long long row = ik / gs / kh;
    const int in_tile = (int)(row % kCN), tile = (int)(row / kCN);
    int b = 0, kt;
    if (edges) {
      b = tile >> 1;
      if (p.chunk_of[b] < 0) continue;
      kt = 0;
    } else {
      int y = a.batch;  // the last sequence with tile0 <= tile (those without tiles share a value)
      while (y - b > 1) {
        const int m = (b + y) >> 1;
        if (p.tile0[m] <= tile) b = m;
        else y = m;
      }
      kt = tile - p.tile0[b];
    }
    const int len = fresh(a.lens + b), end = len + fresh(a.cu_q + b + 1) - fresh(a.cu_q + b);
    const int first = keys_first(a, len, 0);
    kt = edges && (tile & 1) ? (end - 1) / kCN : first / kCN + kt;
    // The copy of the first tile is the first of two, unless it is the last one too.
    if (edges && ((tile & 1) ? (kt + 1) * kCN == end : kt * kCN == first || (kt + 1) * kCN > end)) continue;
    const int pos = kt * kCN + in_tile;
    bool have = pos >= first && pos < end;
    size_t src = 0;
    if (have) {
      const int page = page_of(a.c, b, pos >> a.c.page_shift);
      have = page >= 0;
      src = have ? page_row(a.c, page, h, pos & ((1 << a.c.page_shift) - 1)) : 0;
    }
    const size_t head_step = (size_t)1 << a.c.page_shift;
    const int c0 = edges ? -1 : chunk_col(p.k_mask, j0), c1 = edges ? -1 : chunk_col(p.k_mask, j0 + half);
    const long long copy_row = edges ? ((long long)2 * p.chunk_of[b] + (tile & 1)) * kCN + in_tile : row;
    const bool copy = E4M3 || edges;
    // The rows of the heads: K, and where they are copied V, as they lie.
    using Raw = typename std::conditional<E4M3, uint2, uint4>::type;
    auto fetch = [&](const uint8_t* pool, Raw* w0, Raw* w1) {
#pragma unroll
      for (int k = 0; k < kSideHeads; ++k) {
        const uint8_t* at = pool + ((src + k * head_step) * d + j0) * (E4M3 ? 1 : 2);
        const bool get = have && h + k < hkv;
        w0[k] = get ? fresh(reinterpret_cast<const Raw*>(at)) : Raw{};
        w1[k] = get ? fresh(reinterpret_cast<const Raw*>(at + half * (E4M3 ? 1 : 2))) : Raw{};
      }
    };
    auto widen = [&](Raw w, float scale, float* f) {
      if constexpr (E4M3) {
        e4m3x4_to_f32(w.x, f);
        e4m3x4_to_f32(w.y, f + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= scale;
      } else {
        bf8_to_f32(w, f);
      }
    };
    auto scale_of = [&](const float* scales, int k) { return E4M3 && have && h + k < hkv ? fresh(scales + src + k * head_step) : 0.f; };
    {
      Raw w0[kSideHeads], w1[kSideHeads];
      float sc[kSideHeads], c[8], s[8];
      fetch(a.c.k, w0, w1);
#pragma unroll
      for (int k = 0; k < kSideHeads; ++k) sc[k] = scale_of(a.c.k_scales, k);
      if (c0 >= 0 || c1 >= 0) angles(pos, j0, c, s);
#pragma unroll
      for (int k = 0; k < kSideHeads; ++k) {
        if (h + k >= hkv) break;
        float x0[8], x1[8], y0[8], y1[8];
        widen(w0[k], sc[k], x0);
        widen(w1[k], sc[k], x1);
        if (copy) {
          uint16_t* dst = p.k_copy + ((size_t)(h + k) * p.copy_rows + copy_row) * d + j0;
          *reinterpret_cast<uint4*>(dst) = f32_to_bf8(x0);
          *reinterpret_cast<uint4*>(dst + half) = f32_to_bf8(x1);
        }
        if (c0 >= 0 || c1 >= 0) {
          uint16_t* dst = p.k_rot + ((size_t)(h + k) * p.rot_rows + row) * p.k_cols;
          turn8(x0, x1, c, s, y0, y1);
          if (c0 >= 0) *reinterpret_cast<uint4*>(dst + c0) = f32_to_bf8(y0);
          if (c1 >= 0) *reinterpret_cast<uint4*>(dst + c1) = f32_to_bf8(y1);
        }
      }
    }
    if (copy && a.c.v != nullptr) {
      Raw w0[kSideHeads], w1[kSideHeads];
      float sc[kSideHeads];
      fetch(a.c.v, w0, w1);
#pragma unroll
      for (int k = 0; k < kSideHeads; ++k) sc[k] = scale_of(a.c.v_scales, k);
#pragma unroll
      for (int k = 0; k < kSideHeads; ++k) {
        if (h + k >= hkv) break;
        float x0[8], x1[8];
        widen(w0[k], sc[k], x0);
        widen(w1[k], sc[k], x1);
        uint16_t* dst = p.v_copy + ((size_t)(h + k) * p.copy_rows + copy_row) * d + j0;
        *reinterpret_cast<uint4*>(dst) = f32_to_bf8(x0);
        *reinterpret_cast<uint4*>(dst + half) = f32_to_bf8(x1);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The attention kernel.
// ---------------------------------------------------------------------------
template <int D, bool PAIR, bool LO>
__global__ void __launch_bounds__(kCThreads, 1)
chunk_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ PagedAttendArgs a,
             const __grid_constant__ ChunkPlan p) {
  using Cfg = ChunkCfg<D, PAIR, LO>;
  follow();
  if (__ldcg(p.header) == 0) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_smem = smem;
  uint8_t* ring = smem + Cfg::kQBytes;
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem + Cfg::kSmemData);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int tpc = p.tokens / (PAIR ? 2 : 1);  // tokens of one CTA's tile

  // ---- the unit schedule: snake order over the list, which runs from long to short
  const int num_units = p.header[0] * p.units_x;
  const int nclusters = (int)gridDim.x / (PAIR ? 2 : 1);
  const int cid = (int)blockIdx.x / (PAIR ? 2 : 1);
  const int nrounds = (num_units + nclusters - 1) / nclusters;
  struct Unit {
    int b, kvh, part, tok0, n, len, t0, kt_lo, ntiles, slot;
  };
  auto unit_of_round = [&](int r, Unit& w) -> bool {
    const int u = r * nclusters + ((r & 1) ? nclusters - 1 - cid : cid);
    if (u >= num_units) return false;
    const int ux = u % p.units_x;
    const int4 e = __ldcg(p.list + 2 * (u / p.units_x)), f = __ldcg(p.list + 2 * (u / p.units_x) + 1);
    w.b = e.x;
    w.part = ux % Cfg::kParts;
    w.kvh = ux / Cfg::kParts;
    w.tok0 = fresh(a.cu_q + e.x);
    w.n = fresh(a.cu_q + e.x + 1) - w.tok0;
    w.len = fresh(a.lens + e.x);
    w.t0 = e.y * p.tokens;
    w.kt_lo = e.z;
    w.ntiles = e.w - e.z;
    w.slot = f.x;
    return true;  // a piece without tiles writes an empty partial
  };

  if (threadIdx.x == 0) {
    const uint32_t loads = PAIR && leader ? 2u : 1u;  // the even CTA's barriers count the odd CTA's word too
    mbar_init(&bars->q_full, loads);
    mbar_init(&bars->q_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->p_full[b], PAIR ? 16 : 8);
      mbar_init(&bars->pv_done[b], 1);
    }
    mbar_init(&bars->o_ready, 1);
    mbar_init(&bars->o_empty, PAIR ? 16 : 8);
    mbar_init(&bars->mma_done, 1);
    for (int q = 0; q < 4; ++q) {
      mbar_init(&bars->xfull[q], 2);
      mbar_init(&bars->xfree[q], 2);
    }
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(&bars->ring_full[s], loads);
      mbar_init(&bars->ring_empty[s], 1);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&bars->tmem_base, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&bars->tmem_base, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // One thread, by elect.sync: a copy issued by divergent lanes costs some 200 cycles, and with
    // pages of 16 a tile takes 32 boxes.
    if (elect_one()) {
      auto load = [&](void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
        tma_load_3d(dst, map, bar, c0, c1, c2);
      };
      auto col_of = [](uint32_t mask, int c) { return __popc(mask & ((1u << c) - 1u)) * 64; };
      const int ps = 1 << a.c.page_shift;
      const int kbox = min(ps, Cfg::kKeys), vbox = min(ps, kCN);      // rows of a page box
      const int kboxes = Cfg::kKeys / kbox, vboxes = kCN / vbox;
      const int k_off = (int)rank * (PAIR ? 64 : 0);                  // this CTA's keys of a K tile
      int st = 0;
      uint32_t ph = 0;
      auto next = [&]() { if (++st == Cfg::kStages) { st = 0; ph ^= 1u; } };
      bool ok = true;
      int unit_iter = 0, q_issued = 0;
      for (int r = 0; r < nrounds && ok; ++r) {
        Unit w;
        if (!unit_of_round(r, w)) continue;
        if (w.ntiles == 0) continue;
        if (unit_iter > 0) {
          ok = mbar_wait(&bars->q_empty, (uint32_t)(unit_iter - 1) & 1u, abort_flag);
          if (!ok) break;
        }
        mbar_arrive_expect_tx(&bars->q_full, (Cfg::kQChunks + (LO ? __popc(p.q_mask) : 0)) * 128u * (uint32_t)(tpc * a.group));
#pragma unroll 1
        for (int c = 0; c < Cfg::kQChunks; ++c) {
          const bool rot = (p.q_mask >> c) & 1u;
          load(q_smem + c * kCChunkBytes, rot ? &maps.qs : &maps.q, &bars->q_full, rot ? col_of(p.q_mask, c) : c * 64,
               w.kvh * a.group, w.tok0 + w.t0 + (int)rank * tpc);
          if (LO && rot)
            load(q_smem + (Cfg::kQChunks + c) * kCChunkBytes, &maps.qs, &bars->q_full, p.q_cols + col_of(p.q_mask, c), w.kvh * a.group,
                 w.tok0 + w.t0 + (int)rank * tpc);
        }
        ++q_issued;
        const int first = keys_first(a, w.len, 0), end = w.len + w.n, seq_kt0 = first / kCN;
        const int side0 = p.tile0[w.b];
        const int edge0 = 2 * p.chunk_of[w.b];
        // Rows of tile kt in the copies: -1 when the tile is read from the pages.
        auto copy_row = [&](int kt) -> int {
          if (p.e4m3) return (side0 + kt - seq_kt0) * kCN;
          if ((kt + 1) * kCN > end) return (edge0 + 1) * kCN;
          if (kt * kCN < first) return edge0 * kCN;
          return -1;
        };
        // Table entries of a tile's boxes are read one tile ahead, and looked at when they are used.
        const int32_t* table = a.c.table + (size_t)w.b * a.c.max_blocks;
        auto entries = [&](int kt, int off, int box, int count, int most, int* e) {
          const bool pages = copy_row(kt) < 0;
#pragma unroll
          for (int i = 0; i < most; ++i)
            e[i] = pages && i < count ? fresh(table + ((kt * kCN + off + i * box) >> a.c.page_shift)) : 0;
        };
        // Plane (page, head); a bad page's is past the pool, where a box reads zeros.
        auto plane_of = [&](int e) -> int {
          if ((unsigned)e >= (unsigned)a.c.num_pages) {
            atomicOr(&g_status, kStatusPage);
            return a.c.num_pages * a.c.hkv;
          }
          return e * a.c.hkv + w.kvh;
        };
        constexpr int KB = Cfg::kKeys / 16, VB = kCN / 16;
        int ke[KB], ke_next[KB], ve[VB], ve_next[VB];
        entries(w.kt_lo, k_off, kbox, kboxes, KB, ke_next);
        entries(w.kt_lo, 0, vbox, vboxes, VB, ve_next);
#pragma unroll 1
        for (int jj = 0; jj <= w.ntiles && ok; ++jj) {
          if (jj < w.ntiles) {
            const int kt = w.kt_lo + jj, cr = copy_row(kt);
            const int k_row = kt * kCN + k_off;
#pragma unroll
            for (int i = 0; i < KB; ++i) ke[i] = plane_of(ke_next[i]);
            if (jj + 1 < w.ntiles) entries(kt + 1, k_off, kbox, kboxes, KB, ke_next);
#pragma unroll 1
            for (int s = 0; s < Cfg::kKStages; ++s) {
              ok = mbar_wait(&bars->ring_empty[st], ph ^ 1u, abort_flag);
              if (!ok) break;
              uint64_t* bar = &bars->ring_full[st];
              mbar_arrive_expect_tx(bar, Cfg::kStageBytes);
              uint8_t* dst = ring + st * Cfg::kStageBytes;
              const int c0 = Cfg::kKPerStage * s;
              const uint32_t side = cr >= 0 ? ~0u : p.k_mask >> c0;  // chunks that are not read from the pages
#pragma unroll
              for (int i = 0; i < KB; ++i) {
                if (i >= kboxes) break;
#pragma unroll
                for (int sub = 0; sub < Cfg::kKPerStage; ++sub)
                  if (!((side >> sub) & 1u))
                    load(dst + sub * Cfg::kKChunkBytes + i * kbox * 128, &maps.k, bar, (c0 + sub) * 64,
                         (k_row + i * kbox) & (ps - 1), ke[i]);
              }
#pragma unroll 1
              for (int sub = 0; sub < Cfg::kKPerStage; ++sub) {
                if (!((side >> sub) & 1u)) continue;
                uint8_t* at = dst + sub * Cfg::kKChunkBytes;
                if ((p.k_mask >> (c0 + sub)) & 1u)
                  load(at, &maps.k_rot, bar, col_of(p.k_mask, c0 + sub), (side0 + kt - seq_kt0) * kCN + k_off, w.kvh);
                else
                  load(at, &maps.k_copy, bar, (c0 + sub) * 64, cr + k_off, w.kvh);
              }
              next();
            }
          }
          if (jj >= 1 && ok) {
            const int kt = w.kt_lo + jj - 1, cr = copy_row(kt);
#pragma unroll
            for (int i = 0; i < VB; ++i) ve[i] = plane_of(ve_next[i]);
            if (jj < w.ntiles) entries(kt + 1, 0, vbox, vboxes, VB, ve_next);
#pragma unroll 1
            for (int s = 0; s < Cfg::kVStages; ++s) {
              ok = mbar_wait(&bars->ring_empty[st], ph ^ 1u, abort_flag);
              if (!ok) break;
              uint64_t* bar = &bars->ring_full[st];
              mbar_arrive_expect_tx(bar, Cfg::kStageBytes);
              uint8_t* dst = ring + st * Cfg::kStageBytes;
              const int col = w.part * Cfg::kDv + (PAIR ? 2 * s + (int)rank : s) * Cfg::kVPerStage * 64;
              if (cr >= 0) {
#pragma unroll
                for (int sub = 0; sub < Cfg::kVPerStage; ++sub)
                  load(dst + sub * kCChunkBytes, &maps.v_copy, bar, col + sub * 64, cr, w.kvh);
              } else {
#pragma unroll
                for (int i = 0; i < VB; ++i) {
                  if (i >= vboxes) break;
#pragma unroll
                  for (int sub = 0; sub < Cfg::kVPerStage; ++sub)
                    load(dst + sub * kCChunkBytes + i * vbox * 128, &maps.v, bar, col + sub * 64, (kt * kCN + i * vbox) & (ps - 1),
                         ve[i]);
                }
              }
              next();
            }
          }
        }
        ++unit_iter;
      }
      // This CTA's copies land before it can leave: the last fill of each slot (its phase has parity
      // ph ^ 1 in the order walked here) and the last Q.
      {
        for (int s = 0; s < Cfg::kStages; ++s) {
          const unsigned long long w0 = globaltimer_ns();
          while (!mbar_try_wait(&bars->ring_full[st], ph ^ 1u) && globaltimer_ns() - w0 < kWaitLimitNs) {}
          next();
        }
        if (q_issued > 0) {
          const unsigned long long w0 = globaltimer_ns();
          while (!mbar_try_wait(&bars->q_full, (uint32_t)(q_issued - 1) & 1u) && globaltimer_ns() - w0 < kWaitLimitNs) {}
        }
      }
    }
    __syncwarp();
  } else if (PAIR && warp == 1 && !leader) {
    // ------------------------------------------------------------ arrivals of the odd CTA's loads
    // Every CTA's copies complete on its own barriers, and this thread passes the odd CTA's on to the
    // even one, which issues the MMAs. (Copies that complete on the other CTA's barrier,
    // cta_group::2, take 4,000 to 6,000 cycles each and 4.1 TB/s together with 96 KB in flight
    // per SM; on the own one 900 to 1,900 cycles and 10 TB/s.)
    if (elect_one()) {
      auto pass = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (!mbar_wait(bar, parity, abort_flag)) return false;
        fence_proxy_async_smem();
        mbar_arrive_cluster(smem_u32(bar) & kPeerBitMask);
        return true;
      };
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      int unit_iter = 0;
      for (int r = 0; r < nrounds && ok; ++r) {
        Unit w;
        if (!unit_of_round(r, w)) continue;
        if (w.ntiles == 0) continue;
        ok = pass(&bars->q_full, (uint32_t)unit_iter & 1u);
        ++unit_iter;
#pragma unroll 1
        for (int s = 0; s < w.ntiles * (Cfg::kKStages + Cfg::kVStages) && ok; ++s) {
          ok = pass(&bars->ring_full[st], ph);
          if (++st == Cfg::kStages) { st = 0; ph ^= 1u; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader && elect_one()) {
      constexpr int M = PAIR ? 2 * kCM : kCM;
      constexpr int PV_N = Cfg::kPvN;
      const uint32_t idesc_qk = umma_idesc_bf16(M, kCN, 0, 0);
      const uint32_t idesc_pv = umma_idesc_bf16(M, PV_N, 0, 1);
      const uint64_t q_desc0 = sdesc_sw128(smem_u32(q_smem), 16, 1024);
      const uint64_t k_desc0 = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t v_desc0 = sdesc_sw128(smem_u32(ring), kCChunkBytes, 1024);
      auto commit_both = [&](uint64_t* bar) {
        if constexpr (PAIR) umma_commit_pair_both(bar);
        else umma_commit(bar);
      };
      int st = 0;
      uint32_t ph = 0;
      auto next = [&]() { if (++st == Cfg::kStages) { st = 0; ph ^= 1u; } };
      bool ok = true;
      int g = 0;  // tiles of earlier units
      int unit_iter = 0;
      for (int r = 0; r < nrounds && ok; ++r) {
        Unit w;
        if (!unit_of_round(r, w)) continue;
        if (w.ntiles == 0) continue;
        ok = wait_bar<PAIR>(&bars->q_full, (uint32_t)unit_iter & 1u, abort_flag);
        for (int jj = 0; jj <= w.ntiles && ok; ++jj) {
          if (jj < w.ntiles) {
            const int t = g + jj;
            const uint32_t s_col = (t & 1) ? kColS1 : kColS0;
            // S(t) overwrites the buffer whose P fed PV(t - 2)
            if (t >= 2) ok = wait_bar<PAIR>(&bars->pv_done[t & 1], (uint32_t)((t - 2) >> 1) & 1u, abort_flag);
            tc_fence_after();
            for (int s = 0; s < Cfg::kKStages && ok; ++s) {
              ok = wait_bar<PAIR>(&bars->ring_full[st], ph, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint64_t kd = k_desc0 + (uint64_t)((st * Cfg::kStageBytes) >> 4);
#pragma unroll
              for (int sub = 0; sub < Cfg::kKPerStage; ++sub) {
                const int c = Cfg::kKPerStage * s + sub;
                const uint64_t qd = q_desc0 + (uint64_t)((c * kCChunkBytes) >> 4);
                const uint64_t kds = kd + (uint64_t)((sub * Cfg::kKChunkBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  if constexpr (PAIR) umma_ss_pair(tmem + s_col, qd + 2 * kk, kds + 2 * kk, idesc_qk, (c | kk) != 0);
                  else umma_ss(tmem + s_col, qd + 2 * kk, kds + 2 * kk, idesc_qk, (c | kk) != 0);
                }
                if (LO && ((p.q_mask >> c) & 1u)) {
                  const uint64_t qlo = qd + (uint64_t)((Cfg::kQChunks * kCChunkBytes) >> 4);
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) {
                    if constexpr (PAIR) umma_ss_pair(tmem + s_col, qlo + 2 * kk, kds + 2 * kk, idesc_qk, true);
                    else umma_ss(tmem + s_col, qlo + 2 * kk, kds + 2 * kk, idesc_qk, true);
                  }
                }
              }
              commit_both(&bars->ring_empty[st]);
              next();
            }
            if (!ok) break;
            commit_both(&bars->s_full[t & 1]);
            if (jj == w.ntiles - 1) commit_both(&bars->q_empty);  // the unit's last read of Q
          }
          if (jj >= 1) {
            const int pt = g + jj - 1;
            const uint32_t p_col = (pt & 1) ? kColS1 : kColS0;
            ok = wait_bar<PAIR>(&bars->p_full[pt & 1], (uint32_t)(pt >> 1) & 1u, abort_flag);
            if (!ok) break;
            // the unit's first value MMA overwrites O: the previous unit's epilogue has read it
            if (jj == 1 && unit_iter > 0) {
              ok = wait_bar<PAIR>(&bars->o_empty, (uint32_t)(unit_iter - 1) & 1u, abort_flag);
              if (!ok) break;
            }
            tc_fence_after();
            for (int s = 0; s < Cfg::kVStages && ok; ++s) {
              ok = wait_bar<PAIR>(&bars->ring_full[st], ph, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint64_t vd = v_desc0 + (uint64_t)((st * Cfg::kStageBytes) >> 4);
              const uint32_t o_col = kColO + s * PV_N;
#pragma unroll
              for (int kk = 0; kk < kCN / 16; ++kk) {
                const bool acc = (jj - 1) != 0 || kk != 0;
                if constexpr (PAIR) umma_ts_pair(tmem + o_col, tmem + p_col + kk * 8, vd + 128 * kk, idesc_pv, acc);
                else umma_ts(tmem + o_col, tmem + p_col + kk * 8, vd + 128 * kk, idesc_pv, acc);
              }
              commit_both(&bars->ring_empty[st]);
              next();
            }
            if (!ok) break;
            commit_both(&bars->pv_done[pt & 1]);
          }
        }
        if (!ok) break;
        commit_both(&bars->o_ready);
        g += w.ntiles;
        ++unit_iter;
      }
      if constexpr (PAIR) umma_commit_pair_local(&bars->mma_done);
      else umma_commit(&bars->mma_done);
      const unsigned long long w0 = globaltimer_ns();
      while (!mbar_try_wait(&bars->mma_done, 0) && globaltimer_ns() - w0 < kWaitLimitNs) {}
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float coef = a.softmax_scale * 1.4426950408889634f;
    constexpr int kHC = kCN / 2;
    constexpr int kHO = Cfg::kDv / 2;
    float* xch = bars->xch;
    uint32_t xk = 0;
    auto exchange = [&](float v, bool& okx) -> float {
      xch[half * kCM + row] = v;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->xfull[quad]);
      okx = __all_sync(0xffffffffu, mbar_wait(&bars->xfull[quad], xk & 1u, abort_flag));
      tc_fence_after();
      const float other = okx ? xch[(1 - half) * kCM + row] : v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->xfree[quad]);
      if (okx) okx = __all_sync(0xffffffffu, mbar_wait(&bars->xfree[quad], xk & 1u, abort_flag));
      ++xk;
      return other;
    };
    const int row_tok = row / a.group, row_head = row - row_tok * a.group;  // this row's token and head in the tile
    bool ok = true;
    int g = 0, unit_iter = 0;
    for (int r = 0; r < nrounds && ok; ++r) {
      Unit w;
      if (!unit_of_round(r, w)) continue;
      const int tile_t0 = w.t0 + (int)rank * tpc;        // first token of this CTA's tile
      const int tok = tile_t0 + row_tok;
      const bool valid = row_tok < tpc && tok < w.n;
      const size_t part_row = ((size_t)max(w.slot, 0) * a.c.hkv + w.kvh) * (PAIR ? 256 : 128) + rank * 128 + row;
      if (w.ntiles == 0) {  // an empty piece of a cut unit
        if (half == 0 && w.part == 0) p.part_lse[part_row] = -INFINITY;
        continue;
      }
      const int qpos = w.len + tok;
      // every row of this tile sees every key of a tile at or before min_q and after max_q - window
      const int min_q = w.len + tile_t0, max_q = w.len + max(min(tile_t0 + tpc, w.n), tile_t0 + 1) - 1;
      float m_used = -INFINITY;
      float l_part = 0.f;
      for (int jj = 0; jj < w.ntiles && ok; ++jj) {
        const int t = g + jj, b = t & 1;
        const uint32_t s_col = (b ? kColS1 : kColS0) + half * kHC;
        ok = __all_sync(0xffffffffu, wait_bar<PAIR>(&bars->s_full[b], (uint32_t)(t >> 1) & 1u, abort_flag));
        if (!ok) break;
        tc_fence_after();
        float sv[kHC];
        uint32_t* tr = reinterpret_cast<uint32_t*>(sv);
#pragma unroll
        for (int c = 0; c < kHC / 32; ++c) tmem_ld_x32(tmem + lane_off + s_col + c * 32, tr + c * 32);
        tmem_ld_wait();
        const int k_tile = (w.kt_lo + jj) * kCN;
        const bool partial = k_tile + kCN - 1 > min_q || (a.is_local && k_tile <= max_q - a.window);
        float mx8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx8[i] = -INFINITY;
        if (partial) {
          const int k0 = k_tile + half * kHC;
          const int c_hi = qpos - k0;
          const int c_lo = a.is_local ? qpos - a.window + 1 - k0 : 0;
#pragma unroll
          for (int c = 0; c < kHC; ++c) {
            sv[c] = (c >= c_lo && c <= c_hi) ? sv[c] : -INFINITY;
            mx8[c & 7] = fmaxf(mx8[c & 7], sv[c]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kHC; ++c) mx8[c & 7] = fmaxf(mx8[c & 7], sv[c]);
        }
        const float m_half = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                   fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * coef;
        const float m_tile = fmaxf(m_half, exchange(m_half, ok));
        if (!ok) break;
        // the running maximum is raised only when it grows by more than 2^8 (or was empty)
        float alpha = 1.f;
        bool rescale_o = false;
        if (m_tile > m_used + kRescaleThreshold || (m_used == -INFINITY && m_tile > -INFINITY)) {
          if (m_used != -INFINITY) {
            alpha = fast_exp2(m_used - m_tile);
            l_part *= alpha;
            rescale_o = true;
          }
          m_used = m_tile;
        }
        const float m_sub = (m_used == -INFINITY) ? 0.f : m_used;
        uint32_t pk[kHC / 2];
        float rs4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kHC / 2; ++c) {
          const float p0 = fast_exp2(fmaf(sv[2 * c], coef, -m_sub));
          const float p1 = fast_exp2(fmaf(sv[2 * c + 1], coef, -m_sub));
          rs4[c & 3] += p0 + p1;
          pk[c] = pack_bf16x2(p0, p1);
        }
        l_part += (rs4[0] + rs4[1]) + (rs4[2] + rs4[3]);
        tmem_st_x32(tmem + lane_off + (b ? kColS1 : kColS0) + half * (kHC / 2), pk);
        // O is rescaled by whole warps, once PV(t - 1) has finished; a unit's first tile never
        // needs it. PV(t - 1) is the only phase of its barrier that can still be pending here.
        const bool rescale_warp = __any_sync(0xffffffffu, rescale_o);
        if (rescale_warp && jj >= 1) {
          ok = __all_sync(0xffffffffu, wait_bar<PAIR>(&bars->pv_done[(t - 1) & 1], (uint32_t)((t - 1) >> 1) & 1u, abort_flag));
          if (!ok) {
            tmem_st_wait();
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kHO / 32; ++c) {
            uint32_t o[32];
            tmem_ld_x32(tmem + lane_off + kColO + half * kHO + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_x32(tmem + lane_off + kColO + half * kHO + c * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!PAIR || leader) mbar_arrive(&bars->p_full[b]);
          else mbar_arrive_cluster(smem_u32(&bars->p_full[b]) & kPeerBitMask);
        }
      }
      if (!ok) break;
      const float l_sum = l_part + exchange(l_part, ok);
      if (!ok) break;
      ok = __all_sync(0xffffffffu, wait_bar<PAIR>(&bars->o_ready, (uint32_t)unit_iter & 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const float inv_l = l_sum > 0.f ? 1.f / l_sum : l_sum == 0.f ? 0.f : l_sum;  // a NaN sum stays one
      const bool cut = w.slot >= 0;
      const bool wide = cut || a.out_f32;
      const size_t orow = ((size_t)w.tok0 + tok) * a.hq + w.kvh * a.group + row_head;
      // destination of this row's kDv columns: a cut unit's partial, or the output
      uint8_t* dst = cut ? reinterpret_cast<uint8_t*>(p.part_o + (part_row * Cfg::kParts + w.part) * Cfg::kDv)
                         : static_cast<uint8_t*>(a.out) + (orow * D + w.part * Cfg::kDv) * (a.out_f32 ? 4 : 2);
      constexpr int kOC = kHO / 32;
      constexpr int kOG = kOC >= 2 ? 2 : 1;
#pragma unroll 1
      for (int cg = 0; cg < kOC; cg += kOG) {
        uint32_t ohg[kOG][32];
#pragma unroll
        for (int k = 0; k < kOG; ++k) tmem_ld_x32(tmem + lane_off + kColO + half * kHO + (cg + k) * 32, ohg[k]);
        tmem_ld_wait();
        if (cg + kOG >= kOC) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (!PAIR || leader) mbar_arrive(&bars->o_empty);
            else mbar_arrive_cluster(smem_u32(&bars->o_empty) & kPeerBitMask);
          }
        }
        if (!valid) continue;
#pragma unroll
        for (int k = 0; k < kOG; ++k) {
          const uint32_t* oh = ohg[k];
          const int col = half * kHO + (cg + k) * 32;
          if (wide) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(dst + 4 * (col + 4 * i)) =
                  make_float4(__uint_as_float(oh[4 * i]) * inv_l, __uint_as_float(oh[4 * i + 1]) * inv_l,
                              __uint_as_float(oh[4 * i + 2]) * inv_l, __uint_as_float(oh[4 * i + 3]) * inv_l);
          } else {
            uint32_t wd[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              wd[i] = pack_bf16x2(__uint_as_float(oh[2 * i]) * inv_l, __uint_as_float(oh[2 * i + 1]) * inv_l);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + 2 * (col + 8 * i)) = make_uint4(wd[4 * i], wd[4 * i + 1], wd[4 * i + 2], wd[4 * i + 3]);
          }
        }
      }
      if (half == 0 && valid && w.part == 0) {
        const float lse = l_sum > 0.f ? (m_used + log2f(l_sum)) * 0.6931471805599453f : l_sum == 0.f ? -INFINITY : l_sum;
        if (cut) p.part_lse[part_row] = lse;
        else if (a.lse != nullptr) a.lse[orow] = lse;
      }
      g += w.ntiles;
      ++unit_iter;
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // a pair leaves together: no remote arrival or copy may target a CTA that has left
    __syncwarp();
    cluster_sync_all();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
    else tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Join of cut units: a warp takes 128 columns of one row, the pieces in order.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) chunk_merge_kernel(PagedAttendArgs a, ChunkPlan p) {
  follow();
  if ((int)blockIdx.x >= __ldcg(p.header + 1)) return;
  const int lane = threadIdx.x & 31;
  const int D = a.c.d, chunks = (D + 127) / 128;
  const int rows = p.rows, tpc = kCM / a.group;          // rows of a unit (128 per CTA), tokens per 128
  const int4 e = __ldcg(p.merges + blockIdx.x);          // sequence, unit, first slot, pieces
  const int kvh = blockIdx.y;
  const int tok0 = fresh(a.cu_q + e.x), n = fresh(a.cu_q + e.x + 1) - tok0;
  const size_t head_step = (size_t)a.c.hkv * rows;       // from a piece's part to the next's
#pragma unroll 1
  for (int i = blockIdx.z * 8 + (threadIdx.x >> 5); i < rows * chunks; i += gridDim.z * 8) {
    const int row = i / chunks, c0 = (i - row * chunks) * 128 + lane * 4;
    const int cta = row / kCM, r = row % kCM, rt = r / a.group;
    const int tok = e.y * p.tokens + cta * tpc + rt;
    if (rt >= tpc || tok >= n) continue;
    const size_t pr0 = ((size_t)e.z * a.c.hkv + kvh) * rows + row;
    // Up to 32 pieces at a time, a lane each, as paged_merge_kernel has it.
    float mm = -INFINITY, den = 0.f, bad = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < e.w; s0 += 32) {
      const float l = s0 + lane < e.w ? __ldcg(p.part_lse + pr0 + (s0 + lane) * head_step) : -INFINITY;
      if (__any_sync(0xffffffffu, l != l)) bad = NAN;
      float m = fmaxf(mm, l);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
      if (m == -INFINITY) continue;
      const float old = __expf(mm - m), mine = l > -INFINITY ? __expf(l - m) : 0.f;
      mm = m;
      den *= old;
      acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
      const uint32_t live = __ballot_sync(0xffffffffu, l > -INFINITY);
      const int count = min(32, e.w - s0);
#pragma unroll 4
      for (int k = 0; k < count; ++k) {
        const float wt = __shfl_sync(0xffffffffu, mine, k);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (((live >> k) & 1u) && c0 < D) v = __ldcg(reinterpret_cast<const float4*>(p.part_o + (pr0 + (s0 + k) * head_step) * D + c0));
        den += wt;
        acc.x = fmaf(wt, v.x, acc.x); acc.y = fmaf(wt, v.y, acc.y); acc.z = fmaf(wt, v.z, acc.z); acc.w = fmaf(wt, v.w, acc.w);
      }
    }
    den += bad;
    const size_t orow = ((size_t)tok0 + tok) * a.hq + kvh * a.group + (r - rt * a.group);
    if (c0 < D) {
      const float inv = den > 0.f || den != den ? 1.f / den : 0.f;
      acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
      const size_t o = orow * D + c0;
      if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = acc;
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
    if (c0 == 0 && a.lse) a.lse[orow] = den != den ? den : mm == -INFINITY ? -INFINITY : mm + logf(den);
  }
}

template <int D, bool PAIR, bool LO>
static cudaError_t launch_chunk_t(const ChunkMaps& maps, const PagedAttendArgs& a, const ChunkPlan& p, int units_bound,
                                  cudaStream_t stream) {
  using Cfg = ChunkCfg<D, PAIR, LO>;
  static std::atomic<bool> ready[64];
  const cudaError_t e = allow_smem(chunk_kernel<D, PAIR, LO>, Cfg::kSmemBytes, ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kCThreads);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  const int clusters = p.clusters < units_bound ? p.clusters : units_bound;
  cfg.gridDim = dim3((unsigned)(clusters * (PAIR ? 2 : 1)));
  return cudaLaunchKernelEx(&cfg, chunk_kernel<D, PAIR, LO>, maps, a, p);
}

template <int D>
static cudaError_t launch_chunk_d(bool pair, const ChunkMaps& maps, const PagedAttendArgs& a, const ChunkPlan& p, int units_bound,
                                  cudaStream_t stream) {
  if (p.q_lo)
    return pair ? launch_chunk_t<D, true, true>(maps, a, p, units_bound, stream) : launch_chunk_t<D, false, true>(maps, a, p, units_bound, stream);
  return pair ? launch_chunk_t<D, true, false>(maps, a, p, units_bound, stream) : launch_chunk_t<D, false, false>(maps, a, p, units_bound, stream);
}

cudaError_t launch_chunk(const ChunkMaps& maps, const PagedAttendArgs& a, const ChunkPlan& p, int units_bound,
                         int slots, cudaStream_t stream) {
  cudaError_t e = launch_follower(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, p);
  if (e != cudaSuccess) return e;
  e = launch_follower(p.e4m3 ? chunk_side_kernel<true> : chunk_side_kernel<false>, dim3(kSms * 4), dim3(kSideThreads), 0, stream, a, p);
  if (e != cudaSuccess) return e;
  const bool pair = p.rows > kCM;
  switch (a.c.d) {
    case 64:
      e = p.q_lo ? launch_chunk_t<64, false, true>(maps, a, p, units_bound, stream) : launch_chunk_t<64, false, false>(maps, a, p, units_bound, stream);
      break;
    case 128: e = launch_chunk_d<128>(pair, maps, a, p, units_bound, stream); break;
    case 256: e = launch_chunk_d<256>(pair, maps, a, p, units_bound, stream); break;
    case 512:
      e = pair ? launch_chunk_t<512, true, false>(maps, a, p, units_bound, stream) : launch_chunk_t<512, false, false>(maps, a, p, units_bound, stream);
      break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  // A unit that is cut has two pieces at least. A warp takes 128 columns of up to four rows: a mixed
  // step takes 125 us and three sliding-window prompts, which cut no unit, 180 (a row a warp 129
  // and 192, sixteen 145 and 176).
  const dim3 grid((unsigned)((slots + 1) / 2), (unsigned)a.c.hkv, (unsigned)((p.rows * ((a.c.d + 127) / 128) + 31) / 32));
  return launch_follower(chunk_merge_kernel, grid, dim3(256), 0, stream, a, p);
}

}  // namespace gattn
