// paged_tile.cu -- decode and verify over a paged KV cache on the tcgen05 tensor cores: up to a
// few dozen query rows per KV head against a long run of keys.
//
// The products are transposed, keys on the MMA's M and rows on N, so that few rows waste
// nothing but N's granularity of 16:
//   S^T = K Q^T      M = KT keys (128; 64 for bf16 rows of 512 dims), N, K = head dim
//   O^T += V^T P^T   M = 128 head dims per block, N, K = KT keys
// and a page's rows are operands as they lie: K-major for the scores, MN-major for the values.
// A K=V row is loaded once and serves both ("Visual guide to Gemma 4", section "K=V technique").
// Its rotated dims (section "p-RoPE"; at most 64 pairs: dims [0, 64) and [d/2, d/2 + 64)) are
// turned into a side buffer that only the scores read.
//
// E4M3 pages are not widened at all: codes go into kind::f8f6f4 MMAs. The other operand is 16-bit
// information split into two e4m3 columns, x = hi + lo / 16 with hi = rn(x) and lo = rn(16 (x - hi));
// a column has accumulators of its own, so the factor is taken back in fp32. Query rows are scaled
// by a power of two to a largest magnitude in [128, 256), weights to at most 2^8.75: 16 (x - hi) is
// then 256 at most. hi and lo take 4 bits each, 8 together, down to e4m3's fixed step at the bottom,
// 2^-9 (2^-13 in lo): an element is off by at most 2^-8 of itself (as rounding it to bf16 would
// leave it) or 2^-14, whichever is more, 2^-21 of the row's largest. For a query element that is
// the end of it. A softmax row may have a hundred thousand weights of that size, equal ones
// among them whose errors would add up (flat tail at 2^-19.4 of the largest, 131,072 keys: 3 percent
// of the output; without the factor of 16, 9), so a weight's lo is rounded with a dither: half a
// step times a number in [-1, 1) that goes through the key positions by the golden ratio. It leaves
// a weight off by up to 2^-13, without bias, and neighbours' errors cancel (the same tail: 1.4e-4 by
// arithmetic, 6e-4 measured, of fp32's own additions; weights that are zero stay zero). N is twice
// the rows, and with N's granularity of 16 the second half of 8 rows is free. The rotated dims are
// fp16 (codes turned in fp32, one rounding of 2^-11) in kind::f16 MMAs on hi's accumulators. A key's
// scale multiplies its scores; a value's scale 2^k is folded into its weight: with e = s + k in log2 units, the
// weight is 2^(e - mv + 7) for a running mv near max e, and the softmax sum takes 2^(s - m) with
// an m of its own, so scales of any size only move exponents (rows of zeros: kZeroRowScale).
//
// Work. A unit is up to NR rows of one (sequence, KV head) against all keys its sequence sees.
// Units go round the CTAs, or the tiles of all units are laid end to end and cut into equal runs,
// one per CTA (paged_merge_kernel joins the parts). Persistent: barrier phases run on across
// units, the next unit's query rows are prepared and its first tiles loaded and scored while
// the last one's products and output finish.
//
// Roles (512 threads): warp 0 loads (TMA; a ring slot is 16 KB, one 128-byte column chunk of 128
// keys or two of 64, so that a page as long as the tile is one copy); warp 1 owns TMEM and issues
// the score MMAs, a tile ahead; warp 2 issues the value MMAs; warp 3 hands out the CTA's runs,
// four ahead, and clears the rows of a sequence's first and last tile that no query sees (pages
// may hold anything there, NaN included); warps 4-7 prepare query rows and turn K=V chunks; warps
// 8-15 are two softmax groups, a thread owning a key (its TMEM lane) and 8 or 20 rows. For units
// of 8 rows the groups take every other tile, each with references, sums and an output of its
// own, joined at the unit's end; for 40 rows each has half of them. The references are only
// raised when a score passes them by more than the weights' headroom; until then a tile costs
// each warp one vote and one meeting of four warps, no reduction.
// Every wait is bounded: one that runs out records a timeout and the CTA unwinds.
//
// Bound: HBM, each visible row read once. Measured (cold L2): 8 sequences of 30k to 32k keys, 512
// dims, bf16, 185 to 198 us by the card, with the join (5.1 to 5.5 TB/s; the loads' share of HBM is
// 24 B a cycle and SM, a 64 KB tile takes 3,000 cycles of the 2,700 that allows); 64 sequences on a window of 1,024,
// 256 dims, e4m3, 136 us (3.7 TB/s: a unit is nine tiles, and its first scores and its output
// leave gaps); 40 rows of 16 sequences against 1k to 32k keys, 512 dims, e4m3, 128 us: there the ring
// holds not two tiles beside the query rows' and weights' two columns each, and a tile's chain
// (load, rotation, scores, weights, values) of 10,000 cycles bounds it.
// Instruction fetch and the latency of single warps count as much as bytes here: the first form,
// with a lane per box and waits in every role's loop, took 506 and 400 us of the first and third.
#include <algorithm>

#include "paged.h"

namespace gattn {

namespace {

constexpr int kTThreads = 512;
constexpr int kTSlotBytes = 16384;     // of a ring slot: one 128-byte column chunk of 128 keys, or two of 64
constexpr int kTMaxSlots = 14;
constexpr float kTop8 = 7.f;           // e4m3: the running maximum's weight is 2^7,
constexpr float kHeadroom8 = 1.75f;    // others up to 2^8.75 < 448
constexpr float kLo = 16.f;            // factor of the lo columns

// One unit's run of tiles.
struct __align__(16) TilePiece {
  int b, kvh, row0, rows;
  int tok0, len, first, end;
  int kt0, ntiles;          // first tile, tiles (0: there are no more pieces)
  int slot, pad;            // place of a cut unit's part, or -1
};

template <int SG, int H>
struct __align__(16) TileHeader {
  uint64_t full[kTMaxSlots], empty[kTMaxSlots], edge[kTMaxSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t rot_in[4];       // the producer has started the loads of a tile's rotated chunks
  uint64_t rot_ready[2];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_empty, o_meet, hmeet[2], mma_done[2];
  uint64_t piece_full[8], piece_empty[8];
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) int viol[2][2][4];  // [meeting parity][softmax group][quadrant]
  alignas(16) float red[2][2][2][4][H <= 8 ? 8 : 32];  // [meeting parity][group][maxima or weights' maxima][quadrant][row]
  float sums[2][2][4][H <= 8 ? 8 : 32];    // [unit parity][group][quadrant][row]
  float step[2][2][H];      // a group's factors for sums and output when its references move
  float refs[2][2][2][H];   // [unit parity][group]: references of the sums and of the weights
  // Of a unit's rows (unit mod 8: query rows are prepared up to two units ahead of the scores, which
  // run up to three ahead of the output): score factor (e4m3), output row (token x query heads +
  // head), position.
  float qsc[8][SG * H];
  int orow[8][SG * H];
  int qpos[8][SG * H];
  TilePiece piece[8];
  double itf[64];           // theta_j / (2 pi), 0 past the rotated pairs
};

// Shape of a CTA for units of NR = SG * H rows. Two softmax groups: with SG = 2 each has half of
// the rows, with SG = 1 every other tile (and an output of its own, joined at the end).
template <int D, bool E4M3, bool SAME, int SG, int H>
struct TileCfg {
  static constexpr int KT = (!E4M3 && D == 512) ? 64 : 128;   // keys per tile
  static constexpr int NR = SG * H;                           // rows of a unit
  static constexpr int TG = 3 - SG;                           // groups that share the rows
  static constexpr int HW = 4;                                // warps for query rows and rotation
  // columns: the MMA's N, in 16s (8s with 64 keys on M, for the scores: NQ below)
  static constexpr int N = E4M3 ? (2 * NR + 15) / 16 * 16 : (NR + 15) / 16 * 16;
  static constexpr int LO = NR;                               // first lo column
  // Sliding-window layers rotate every dim of a query row, and rounding it back to bf16 would be the
  // largest error of their outputs (relative 1.8e-3; the weights' rounding 1.1e-3): it stays hi + lo
  // there too, in bf16 columns. (Not 40 rows of 512 dims, beside which no tile would fit.)
  static constexpr bool QLO = !E4M3 && !SAME && !(D == 512 && NR > 8);
  static constexpr int SN = QLO ? (2 * NR + 15) / 16 * 16 : N;  // columns of a score buffer
  static constexpr int CH = E4M3 ? D / 128 : D / 64;          // 128-byte chunks of a row
  static constexpr int PB = D / 128;                          // 128-dim blocks of the output
  static constexpr int CHUNK = KT * 128;                      // bytes of a chunk of a tile
  static constexpr int G = kTSlotBytes / CHUNK;               // chunks of a ring slot
  static constexpr int NS = CH / G;                           // slots of a tile's keys (or values)
  static constexpr int PER = CH / PB / G;                     // slots of a 128-dim block
  static constexpr int NQ = QLO ? SN : KT == 64 && NR <= 8 ? 8 : N;  // query rows with padding
  static constexpr int QROT = E4M3 ? 2 * NQ * 128 : 0;        // fp16 rows of the rotated dims
  static constexpr int QB = CH * NQ * 128 + QROT;
  static constexpr int P_B = E4M3 ? N * 128 : KT / 64 * N * 128;
  static constexpr int ROT = 2 * KT * 128;                    // two chunks of 64 dims, 16 bits
  static constexpr int HEADER = (sizeof(TileHeader<SG, H>) + 1023) / 1024 * 1024;
  static constexpr int BUDGET = 232448 - 1024 - HEADER;
  static constexpr int COL_O = 2 * SN;
  static_assert(COL_O + TG * PB * N <= 512, "TMEM columns");
  static_assert(CH % G == 0 && PER >= 1, "slots of a tile");
};

// Frequencies of the first 64 rotary pairs, theta_j / (2 pi), and the factor of 64 pairs on.
struct TileTurns {
  double freq[64];
  double step64;
};

// Buffers of a launch: two query buffers where they leave at least two tiles of ring.
struct TileBufs {
  int nq, nrot, kslots, vslots;  // value ring only for separate values
};
template <int D, bool E4M3, bool SAME, int SG, int H>
__host__ __device__ inline TileBufs tile_bufs(bool rot) {
  using C = TileCfg<D, E4M3, SAME, SG, H>;
  constexpr bool kv_same = SAME;
  // As much ring as three tiles, then a second buffer for the rotated copy, then one for the
  // next unit's query rows.
  TileBufs b;
  const int tile = C::NS * kTSlotBytes * (kv_same ? 1 : 2);
  int left = C::BUDGET - C::QB - 2 * C::P_B - (rot ? C::ROT : 0);
  b.nq = b.nrot = 1;
  if (!rot) b.nrot = 0;
  if (rot && left - C::ROT >= 3 * tile) {
    b.nrot = 2;
    left -= C::ROT;
  }
  if (left - C::QB >= 2 * tile + tile / 2 && (left - C::QB >= 3 * tile || left < 3 * tile)) {
    b.nq = 2;
    left -= C::QB;
  }
  int slots = left / kTSlotBytes;
  if (slots > kTMaxSlots) slots = kTMaxSlots;
  // the loads run at most four tiles ahead of the rotation (rot_in has four barriers)
  if (rot && slots > 4 * C::NS) slots = 4 * C::NS;
  // the slots of a block lie together
  constexpr int even = ~(C::PER - 1);
  if (kv_same) {
    b.kslots = slots & even;
    b.vslots = 0;
  } else {
    b.kslots = (slots / 2) & even;
    b.vslots = (slots - b.kslots) & even;
  }
  return b;
}

// Position in load order to block of 128 dims: the blocks with rotated dims first.
template <int PB>
__device__ __forceinline__ int block_at(int i) {
  if constexpr (PB == 4) return i == 1 ? 2 : i == 2 ? 1 : i;
  return i;
}
// Chunk (128 bytes of a row) at position i of the load order.
template <int PB, bool E4M3>
__device__ __forceinline__ int chunk_at(int i) {
  if constexpr (E4M3) return block_at<PB>(i);
  return 2 * block_at<PB>(i >> 1) + (i & 1);
}

__device__ __forceinline__ void tma_load_4d(void* smem, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(smem)),
      "l"(m), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Instruction descriptors: e4m3 operands (format 0), or fp16 ones (format 0 of kind::f16), fp32 D.
__host__ __device__ constexpr uint32_t idesc_zero_fmt(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld_x4(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void tmem_ld_x8(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(a));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x4(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
template <int H>
__device__ __forceinline__ void tmem_ld_n(uint32_t a, uint32_t* r) {
  static_assert(H == 8 || H == 20, "rows of a thread");
  if constexpr (H == 8) {
    tmem_ld_x8(a, r);
  } else {
    tmem_ld_x16(a, r);
    tmem_ld_x4(a + 16, r + 16);
  }
}
template <int H>
__device__ __forceinline__ void tmem_st_n(uint32_t a, const uint32_t* r) {
  if constexpr (H == 8) {
    tmem_st_x8(a, r);
  } else {
    tmem_st_x16(a, r);
    tmem_st_x4(a + 16, r + 16);
  }
}

// A bounded wait. The first try is in line (a role alone on its scheduler pays five cycles and
// more for every instruction, and the barrier is mostly in the phase already); what follows is a
// call, so that the six loops of a CTA stay small together. Each try suspends the warp for a
// while, so the limit on tries is seconds; running out of them records a timeout.
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = false;
#pragma unroll 1
  for (int n = 0; !ok && !*abort; ++n) {
    ok = mbar_try_wait(bar, parity);
    if (n == 1 << 24) {
      atomicOr(&g_status, kStatusTimeout);
      *abort = 1;
    }
  }
  return ok;
}
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || wait_more(bar, parity, abort);
}
// The same by a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_more(bar, parity, abort));
}

__device__ __noinline__ float2 turn_of(double pos, double inv_freq_turns) {
  float2 r;
  rope_cos_sin(pos, inv_freq_turns, &r.x, &r.y);
  return r;
}

// Whether the value row at position pos, whose table entry is known to be good, is one of zeros.
__device__ __noinline__ bool zero_row(const PagedAttendArgs& a, const uint8_t* pool, const TilePiece& p, int pos) {
  const int page = fresh(a.c.table + (size_t)p.b * a.c.max_blocks + (pos >> a.c.page_shift));
  const uint4* row = reinterpret_cast<const uint4*>(pool + page_row(a.c, page, p.kvh, pos & ((1 << a.c.page_shift) - 1)) * a.c.d);
#pragma unroll 1
  for (int i = 0; i < a.c.d / 16; ++i) {
    const uint4 w = fresh(row + i);
    if ((w.x | w.y | w.z | w.w) & 0x7F7F7F7Fu) return false;
  }
  return true;
}

// The CTA's pieces in turn, by one warp: units team, team + teams, ..., or a run of the line of
// all units' tiles.
struct TileWalk {
  int x, x_end, before, b, run;
  __device__ __forceinline__ void start(const PagedAttendArgs& a, int lane) {
    const int team = blockIdx.x;
    const int total = line_find(a, lane, a.cut ? -1 : team, &b, &before);
    run = run_length(a, total);
    x = (int)min((long long)team * run, (long long)total);
    x_end = a.cut ? (int)min((long long)total, (long long)x + run) : total;
    if (a.cut && x < x_end) line_find(a, lane, x, &b, &before);
    if (a.cut && lane == 0) a.joins[team] = make_int4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void next(const PagedAttendArgs& a, int lane, TilePiece& p) {
    p.ntiles = 0;
    if (x >= x_end) return;
    int blocks, units;
    seq_units(a, b, &blocks, &units);
    if (x - before >= (a.cut ? blocks * units : units)) {
      line_find(a, lane, x, &b, &before);
      seq_units(a, b, &blocks, &units);
    }
    const uint32_t in = x - before, per = a.cut ? blocks : 1;
    const uint32_t u = in / per, lo = in - u * per, hkv = a.c.hkv;
    const int hi = a.cut ? min(blocks, x_end - x + (int)lo) : blocks;
    p.slot = lo == 0 && hi == blocks ? -1 : 2 * (int)blockIdx.x + (lo == 0 ? 1 : 0);
    p.b = b;
    p.kvh = u % hkv;
    p.row0 = u / hkv * a.unit_rows;
    p.tok0 = fresh(a.cu_q + b);
    const int n = fresh(a.cu_q + b + 1) - p.tok0;
    p.len = fresh(a.lens + b);
    p.rows = min(a.unit_rows, n * a.group - p.row0);
    p.first = keys_first(a, p.len, 0);
    p.end = p.len + n;
    p.kt0 = (p.first >> a.unit_shift) + lo;
    p.ntiles = hi - lo;
    p.pad = 0;
    if (p.slot >= 0 && lo == 0 && lane == 0)
      a.joins[blockIdx.x] = join_of((x + blocks - 1) / run - (int)blockIdx.x + 1, p.tok0, p.rows, p.kvh, p.row0);
    x += a.cut ? p.ntiles : a.teams;
  }
};

// Sums over a warp's lanes of 2 CNT values each: at every step a lane hands half of its values
// to the lane W away and adds the other's; with one value left it adds whole ones.
template <int W, int CNT>
__device__ __forceinline__ int scatter_sums(float* x, int lane) {
  if constexpr (W == 0) {
    return 0;
  } else {
    const bool up = (lane & W) != 0;
    if constexpr (CNT > 0) {
#pragma unroll
      for (int q = 0; q < CNT; ++q) {
        const float send = up ? x[q] : x[q + CNT], keep = up ? x[q + CNT] : x[q];
        x[q] = keep + __shfl_xor_sync(0xffffffffu, send, W);
      }
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], W);
    }
    return (up ? CNT : 0) + scatter_sums<W / 2, CNT / 2>(x, lane);
  }
}

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(x) : "memory");
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace

template <int D, bool E4M3, bool SAME, int SG, int H>
__global__ void __launch_bounds__(kTThreads, 1)
paged_tile_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const __grid_constant__ PagedAttendArgs a, const __grid_constant__ TileTurns turns) {
  using C = TileCfg<D, E4M3, SAME, SG, H>;
  constexpr int KT = C::KT, N = C::N, NQ = C::NQ, NR = C::NR, CH = C::CH, PB = C::PB, HALF = D / 2;
  constexpr int G = C::G, NS = C::NS, TG = C::TG;
  // slot of a tile that holds the second half's rotated dims (the first holds the first half's)
  constexpr int ROT2 = G == 2 ? 1 : E4M3 ? (PB > 1 ? 1 : 0) : (PB > 1 ? 2 : 1);
  follow();
  if (a.rest != nullptr && __ldcg(a.rest) == 0) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using Header = TileHeader<SG, H>;
  Header* hd = reinterpret_cast<Header*>(base);
  constexpr bool kv_same = SAME;
  const bool rot = SAME && a.r > 0;
  const TileBufs bufs = tile_bufs<D, E4M3, SAME, SG, H>(rot);
  uint8_t* q_s = base + C::HEADER;
  uint8_t* p_s = q_s + bufs.nq * C::QB;
  uint8_t* rot_s = p_s + 2 * C::P_B;
  uint8_t* kring = rot_s + bufs.nrot * C::ROT;
  uint8_t* vring = kring + bufs.kslots * kTSlotBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int s = 0; s < kTMaxSlots; ++s) {
      mbar_init(&hd->full[s], 1);
      mbar_init(&hd->empty[s], 1);
      mbar_init(&hd->edge[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hd->q_full[i], C::HW);
      mbar_init(&hd->q_empty[i], 1);
      mbar_init(&hd->rot_ready[i], C::HW);
      mbar_init(&hd->s_full[i], 1);
      mbar_init(&hd->p_full[i], 4 * SG);  // the groups that form a tile's weights
      mbar_init(&hd->pv_done[i], 1);
      mbar_init(&hd->hmeet[i], 4);
      mbar_init(&hd->mma_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&hd->rot_in[i], 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&hd->piece_full[i], 1);
      mbar_init(&hd->piece_empty[i], 15);  // every warp but the one that hands pieces out
    }
    mbar_init(&hd->o_empty, 8);
    mbar_init(&hd->o_meet, 8);
    hd->abort_flag = 0;
    fence_barrier_init();
  }
  // rows that no unit writes (N's granularity) stay zero in the query and weight buffers
#pragma unroll 1
  for (int i = threadIdx.x; i < (bufs.nq * C::QB + 2 * C::P_B) / 16; i += kTThreads)
    reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
  for (int j = threadIdx.x; j < 64; j += kTThreads) hd->itf[j] = j < a.r ? turns.freq[j] : 0.0;
  if (a.chunk_of == nullptr && blockIdx.x == 0)
#pragma unroll 1
    for (int b = threadIdx.x; b < a.batch; b += kTThreads) {
      const int tok0 = fresh(a.cu_q + b), n = fresh(a.cu_q + b + 1) - tok0;
      if (n != 0 && !seq_ok(a, tok0, n, fresh(a.lens + b))) atomicOr(&g_status, kStatusSeqlen);
    }
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(&hd->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = hd->tmem_base;
  volatile int* abort_flag = &hd->abort_flag;
  TilePiece p;
  // Piece i of this CTA; false at the end (or on abort).
  auto piece_at = [&](int i, TilePiece& out) -> bool {
    if (!warp_wait(&hd->piece_full[i & 7], (uint32_t)(i >> 3) & 1u, abort_flag)) return false;
    out = hd->piece[i & 7];
    __syncwarp();
    if (lane == 0) mbar_arrive(&hd->piece_empty[i & 7]);
    return out.ntiles > 0;
  };
  // The same for a role of one thread (warps 0 to 2).
  auto piece_next = [&](int i, TilePiece& out) -> bool {
    if (!thread_wait(&hd->piece_full[i & 7], (uint32_t)(i >> 3) & 1u, abort_flag)) return false;
    out = hd->piece[i & 7];
    mbar_arrive(&hd->piece_empty[i & 7]);
    return out.ntiles > 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    // The warp walks together, a lane per page box of a tile for what differs between boxes; one
    // thread, by elect.sync, issues (copies issued by divergent lanes cost some 200 cycles each).
    const int ps = 1 << a.c.page_shift, box = min(ps, KT), boxes = KT / box;
    int ks = 0, vs = 0, t = 0;
    uint32_t kph = 0, vph = 0, edge_ph = 0;    // edge_ph bit s: parity of slot s's next edge load
    uint32_t last_full = 0, last_edge = 0;     // slots whose last load completes on full / edge
    bool ok = true;
#pragma unroll 1
    for (int piece = 0; ok && piece_at(piece, p); ++piece) {
      const int32_t* table = a.c.table + (size_t)p.b * a.c.max_blocks;
      // Whether some query sees this lane's box of tile kt, and its table entry, read a tile ahead
      auto seen = [&](int kt) { return lane < boxes && kt * KT + lane * box < p.end && kt * KT + (lane + 1) * box > p.first; };
      auto entry = [&](int kt) { return seen(kt) ? fresh(table + ((kt * KT + lane * box) >> a.c.page_shift)) : -1; };
      int next = entry(p.kt0);
#pragma unroll 1
      for (int lt = 0; lt < p.ntiles && ok; ++lt, ++t) {
        const int kt = p.kt0 + lt, row = boxes > 1 ? 0 : (kt * KT) & (ps - 1);
        const bool used = seen(kt);
        int plane = next * a.c.hkv + p.kvh;
        if (used && (unsigned)next >= (unsigned)a.c.num_pages) {
          atomicOr(&g_status, kStatusPage);
          plane = a.c.num_pages * a.c.hkv;     // past the pool: zeros
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, used);
        const uint32_t bytes = (uint32_t)(__popc(mask) * box * 128 * G);
        if (lt + 1 < p.ntiles) next = entry(kt + 1);
        const bool cut = kt * KT < p.first || (kt + 1) * KT > p.end;
#pragma unroll 1
        for (int v = 0; v < (SAME ? 1 : 2) && ok; ++v) {
          const CUtensorMap* map = v ? &v_map : &k_map;
          uint8_t* ring = v ? vring : kring;
          const int bar0 = v ? bufs.kslots : 0, slots = v ? bufs.vslots : bufs.kslots;
          const bool clear = cut && (SAME || v);
          uint64_t* bars = (clear ? hd->edge : hd->full) + bar0;
          int s = v ? vs : ks;
          uint32_t f = v ? vph : kph, filled = 0;
#pragma unroll 1
          for (int i = 0; i < NS; ++i) {
            ok = warp_wait(&hd->empty[bar0 + s], f ^ 1u, abort_flag);
            if (!ok) break;
            filled |= 1u << s;
            uint64_t* bar = &bars[s];
            uint8_t* dst = ring + s * kTSlotBytes;
            const int c = chunk_at<PB, E4M3>(i * G);
            if (elect_one()) mbar_arrive_expect_tx(bar, bytes);
#pragma unroll 1
            for (uint32_t m = mask; m != 0; m &= m - 1) {
              const int bx = __ffs(m) - 1, pl = __shfl_sync(0xffffffffu, plane, bx);
              if (elect_one()) {
                tma_load_4d(dst + bx * box * 128, map, bar, 0, row, c, pl);  // both chunks, if the box is the tile
                if (G == 2 && boxes > 1) tma_load_4d(dst + C::CHUNK + bx * box * 128, map, bar, 0, row, c + 1, pl);
              }
            }
            // The rotated chunks' loads have begun: their slots' barriers are in the phase to wait for.
            if (rot && i == ROT2 && lane == 0) mbar_arrive(&hd->rot_in[t & 3]);
            if (++s == slots) { s = 0; f ^= 1u; }
          }
          filled <<= bar0;
          last_edge = clear ? last_edge | filled : last_edge & ~filled;
          last_full = clear ? last_full & ~filled : last_full | filled;
          if (clear) edge_ph ^= filled;
          if (v) {
            vs = s;
            vph = f;
          } else {
            ks = s;
            kph = f;
          }
        }
      }
    }
    if (lane == 0) {
      // the last load of every slot lands before the CTA can leave (the barrier's phase parity: of a
      // plain load the one its slot's next fill would flip, of an edge load the last used)
#pragma unroll 1
      for (int s = 0; s < bufs.kslots + bufs.vslots; ++s) {
        if (!(((last_full | last_edge) >> s) & 1u)) continue;
        const bool on_edge = (last_edge >> s) & 1u;
        const bool k = s < bufs.kslots;
        const int nxt = k ? ks : bufs.kslots + vs;
        const uint32_t ph = k ? kph : vph;
        const uint32_t par = on_edge ? ((edge_ph >> s) & 1u) ^ 1u : (s < nxt ? ph : ph ^ 1u);
        const unsigned long long w0 = globaltimer_ns();
        while (!mbar_try_wait(on_edge ? &hd->edge[s] : &hd->full[s], par) && globaltimer_ns() - w0 < kWaitLimitNs) {}
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ score MMAs
    if (elect_one()) {
      const uint32_t id16 = E4M3 ? idesc_zero_fmt(KT, NQ, 0, 0) : umma_idesc_bf16(KT, NQ, 0, 0);
      const uint32_t id8 = idesc_zero_fmt(KT, NQ, 0, 0);
      // descriptor of the K-major operand at 16-byte unit `at` of shared memory
      const uint64_t desc0 = sdesc_sw128(0, 16, 1024);
      auto desc_at = [&](uint32_t at) { return desc0 + at; };
      int ks = 0, t = 0;
      uint32_t kph = 0;
      bool ok = true;
#pragma unroll 1
      for (int piece = 0; ok && piece_next(piece, p); ++piece) {
        const int qb = piece % bufs.nq;
        ok = thread_wait(&hd->q_full[qb], (uint32_t)(piece / bufs.nq) & 1u, abort_flag);
        const uint32_t q_addr = smem_u32(q_s + qb * C::QB) >> 4, ring_addr = smem_u32(kring) >> 4;
#pragma unroll 1
        for (int lt = 0; lt < p.ntiles && ok; ++lt, ++t) {
          const uint32_t sb = tmem + (uint32_t)(t & 1) * C::SN;
          // S^T(t) overwrites the scores that softmax(t - 2) read
          if (t >= 2) ok = thread_wait(&hd->p_full[t & 1], (uint32_t)((t - 2) >> 1) & 1u, abort_flag);
          uint32_t acc = 0;
          const int ks0 = ks;
          // First the chunks' unrotated steps, then the rotated copy. The waits come before the MMAs
          // (which the ring's depth allows: the loads are tiles ahead) so that the MMAs issue back to
          // back, all descriptors one addition off a slot's.
          uint32_t at[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            ok = ok && thread_wait(&hd->full[ks], kph, abort_flag);
            at[i] = ring_addr + (uint32_t)ks * (kTSlotBytes >> 4);
            if (++ks == bufs.kslots) { ks = 0; kph ^= 1u; }
          }
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < NS; ++i) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
              const int c = chunk_at<PB, E4M3>(i * G) + j;
              const uint64_t kd = desc_at(at[i] + j * (C::CHUNK >> 4));
              const uint64_t qd = desc_at(q_addr + (uint32_t)(c * (NQ * 8)));
              if constexpr (E4M3) {
                // the rotated dims are the first 64 of the row and of its second half
                const bool first = rot && (c * 128 == 0 || c * 128 == HALF), second = rot && HALF == 64;
                if (!first) {
                  umma_f8(sb, kd, qd, id8, acc);
                  umma_f8(sb, kd + 2, qd + 2, id8, 1);
                  acc = 1;
                }
                if (!second) {
                  umma_f8(sb, kd + 4, qd + 4, id8, acc);
                  umma_f8(sb, kd + 6, qd + 6, id8, 1);
                  acc = 1;
                }
              } else if (!(rot && (c == 0 || c == HALF / 64))) {
                umma_ss(sb, kd, qd, id16, acc);
                umma_ss(sb, kd + 2, qd + 2, id16, 1);
                umma_ss(sb, kd + 4, qd + 4, id16, 1);
                umma_ss(sb, kd + 6, qd + 6, id16, 1);
                acc = 1;
              }
            }
            if (!SAME) {
              int slot = ks0 + i;
              if (slot >= bufs.kslots) slot -= bufs.kslots;
              umma_commit(&hd->empty[slot]);
            }
          }
          if (ok && rot) {
            ok = thread_wait(&hd->rot_ready[t % bufs.nrot], (uint32_t)(t / bufs.nrot) & 1u, abort_flag);
            tc_fence_after();
            const uint32_t rot_addr = smem_u32(rot_s + (t % bufs.nrot) * C::ROT) >> 4;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok) break;
              const uint64_t kd = desc_at(rot_addr + i * (C::CHUNK >> 4)), qd = desc_at(q_addr + (uint32_t)((E4M3 ? CH + i : i * (HALF / 64)) * (NQ * 8)));
              umma_ss(sb, kd, qd, id16, acc);
              umma_ss(sb, kd + 2, qd + 2, id16, 1);
              umma_ss(sb, kd + 4, qd + 4, id16, 1);
              umma_ss(sb, kd + 6, qd + 6, id16, 1);
              acc = 1;
            }
          }
          if (!ok) break;
          umma_commit(&hd->s_full[t & 1]);
          if (lt == p.ntiles - 1) umma_commit(&hd->q_empty[qb]);
        }
      }
      umma_commit(&hd->mma_done[0]);
      const unsigned long long w0 = globaltimer_ns();
      while (!mbar_try_wait(&hd->mma_done[0], 0) && globaltimer_ns() - w0 < kWaitLimitNs) {}
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ value MMAs
    if (elect_one()) {
      const uint32_t id = E4M3 ? idesc_zero_fmt(128, N, 1, 0) : umma_idesc_bf16(128, N, 1, 0);
      const int slots = SAME ? bufs.kslots : bufs.vslots, bar0 = SAME ? 0 : bufs.kslots;
      uint8_t* ring = SAME ? kring : vring;
      int vs = 0, t = 0;
      uint32_t vph = 0;
      bool ok = true;
#pragma unroll 1
      for (int piece = 0; ok && piece_next(piece, p); ++piece) {
#pragma unroll 1
        for (int lt = 0; lt < p.ntiles && ok; ++lt, ++t) {
          ok = thread_wait(&hd->p_full[t & 1], (uint32_t)(t >> 1) & 1u, abort_flag);
          // a unit's first products overwrite the output that the last unit's epilogue has read
          if (ok && lt == 0 && piece > 0) ok = thread_wait(&hd->o_empty, (uint32_t)(piece - 1) & 1u, abort_flag);
          const uint32_t p_addr = smem_u32(p_s + (t & 1) * C::P_B);
          uint32_t at[PB];
          const int vs0 = vs;
#pragma unroll
          for (int i = 0; i < PB; ++i) {
            if (!SAME)                    // K=V chunks have landed: the scores of this tile needed them
#pragma unroll
              for (int j = 0; j < C::PER; ++j) ok = ok && thread_wait(&hd->full[bar0 + vs + j], vph, abort_flag);
            at[i] = (smem_u32(ring) >> 4) + (uint32_t)vs * (kTSlotBytes >> 4);
            vs += C::PER;
            if (vs == slots) { vs = 0; vph ^= 1u; }
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t pd = sdesc_sw128(p_addr, 16, 1024), vdesc0 = sdesc_sw128(0, C::CHUNK, 1024);
#pragma unroll
          for (int i = 0; i < PB; ++i) {
            const uint64_t vd = vdesc0 + at[i];
            const uint32_t d = tmem + C::COL_O + (uint32_t)((TG == 2 ? (t & 1) * PB : 0) + block_at<PB>(i)) * N;
#pragma unroll
            for (int kk = 0; kk < KT / (E4M3 ? 32 : 16); ++kk) {
              const uint32_t acc = kk != 0 ? 1u : (uint32_t)(lt >= TG);
              if constexpr (E4M3) umma_f8(d, vd + 256 * kk, pd + 2 * kk, id, acc);
              else umma_ss(d, vd + 128 * kk, pd + (kk >> 2) * (N * 8) + 2 * (kk & 3), id, acc);
            }
#pragma unroll
            for (int j = 0; j < C::PER; ++j) {
              int slot = vs0 + i * C::PER + j;
              if (slot >= slots) slot -= slots;
              umma_commit(&hd->empty[bar0 + slot]);
            }
          }
          if (!ok) break;
          umma_commit(&hd->pv_done[t & 1]);
        }
      }
      umma_commit(&hd->mma_done[1]);
      const unsigned long long w0 = globaltimer_ns();
      while (!mbar_try_wait(&hd->mma_done[1], 0) && globaltimer_ns() - w0 < kWaitLimitNs) {}
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ pieces, clearing of cut tiles
    TileWalk walk;
    walk.start(a, lane);
    int made = 0, last = -100;             // pieces handed out; the index of the end mark
    auto hand_out = [&]() -> bool {
      if (last != -100) return true;
      if (made >= 8 && !warp_wait(&hd->piece_empty[made & 7], (uint32_t)((made >> 3) - 1) & 1u, abort_flag)) return false;
      walk.next(a, lane, p);
      if (lane == 0) hd->piece[made & 7] = p;
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd->piece_full[made & 7]);
      if (p.ntiles == 0) last = made;
      ++made;
      return true;
    };
    bool ok = true;
    const int slots = kv_same ? bufs.kslots : bufs.vslots, bar0 = kv_same ? 0 : bufs.kslots;
    uint8_t* ring = kv_same ? kring : vring;
    int s = 0;
    uint32_t edge_ph = 0;
#pragma unroll 1
    for (int piece = -4; ok && piece != last; ++piece) {  // pieces are handed out four ahead
      ok = hand_out();
      __syncwarp();
      if (piece < 0) continue;
      p = hd->piece[piece & 7];            // handed out four pieces ago: not replaced before eight
#pragma unroll 1
      for (int lt = 0; lt < p.ntiles && ok; ++lt) {
        const int k0 = (p.kt0 + lt) * KT;
        const int lo = max(p.first - k0, 0), hi = min(p.end - k0, KT);
#pragma unroll 1
        for (int i = 0; i < NS && ok; ++i) {
          if (lo > 0 || hi < KT) {
            ok = warp_wait(&hd->edge[bar0 + s], (edge_ph >> s) & 1u, abort_flag);
            if (!ok) break;
            edge_ph ^= 1u << s;
#pragma unroll 1
            for (int j = 0; j < G; ++j) {
              uint4* rows = reinterpret_cast<uint4*>(ring + s * kTSlotBytes + j * C::CHUNK);
#pragma unroll 1
              for (int x = lane; x < lo * 8; x += 32) rows[x] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
              for (int x = hi * 8 + lane; x < KT * 8; x += 32) rows[x] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&hd->full[bar0 + s]);
          }
          if (++s == slots) s = 0;
        }
      }
    }
  } else if (warp < 4 + C::HW) {
    // ------------------------------------------------------------ query rows, rotation of K=V chunks
    const int hw = warp - 4;
    const int ht = threadIdx.x - 128;
    TilePiece np;
    bool more = piece_at(0, np);
    int q_piece = 0;
    auto prepare = [&]() -> bool {         // query rows of piece np, when there is one; false on abort
      if (!more) return true;
      const int qb = q_piece % bufs.nq;
      if (q_piece >= bufs.nq &&
          !warp_wait(&hd->q_empty[qb], (uint32_t)(q_piece / bufs.nq - 1) & 1u, abort_flag))
        return false;
      uint8_t* qd = q_s + qb * C::QB;
      constexpr int QI = (HALF + 63) / 64;   // words of two pairs per lane and half row
      constexpr int RW = NR / C::HW;         // rows of a warp, one after the other: they share tokens, and angles
      int angle_tk = -1;
      float2 c0[QI], c1[QI];
#pragma unroll 1
      for (int row = hw * RW; row < (hw + 1) * RW; ++row) {
        const bool have = row < np.rows;
        const int tk = (np.row0 + row) / a.group, hh = np.row0 + row - tk * a.group;
        const int orow = (np.tok0 + tk) * a.hq + np.kvh * a.group + hh;
        const uint16_t* src = a.q + (size_t)orow * D;
        if (lane == 0) {
          hd->orow[q_piece & 7][row] = orow;
          hd->qpos[q_piece & 7][row] = np.len + tk;
        }
        uint32_t w0[QI], w1[QI];
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          const bool get = have && 2 * lane + 64 * i < HALF;
          w0[i] = get ? fresh(reinterpret_cast<const uint32_t*>(src + 2 * lane + 64 * i)) : 0u;
          w1[i] = get ? fresh(reinterpret_cast<const uint32_t*>(src + HALF + 2 * lane + 64 * i)) : 0u;
        }
        if (have && tk != angle_tk) {
          angle_tk = tk;
          double f0 = turns.freq[2 * lane], f1 = turns.freq[2 * lane + 1];  // 64 pairs on each time
#pragma unroll
          for (int i = 0; i < QI; ++i) {
            const int j = 2 * lane + 64 * i;
            c0[i] = c1[i] = make_float2(1.f, 0.f);
            if (64 * i < a.r) {
              if (j < a.r) c0[i] = turn_of((double)(np.len + tk), f0);
              if (j + 1 < a.r) c1[i] = turn_of((double)(np.len + tk), f1);
              f0 *= turns.step64;
              f1 *= turns.step64;
            }
          }
        }
        // y: the row's elements in fp32, rotated; {first half's two, second half's two}
        float y[QI][2][2];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          y[i][0][0] = __uint_as_float(w0[i] << 16);
          y[i][0][1] = __uint_as_float(w0[i] & 0xFFFF0000u);
          y[i][1][0] = __uint_as_float(w1[i] << 16);
          y[i][1][1] = __uint_as_float(w1[i] & 0xFFFF0000u);
          if (have && 64 * i < a.r) {
            const float x00 = y[i][0][0], x01 = y[i][0][1], x10 = y[i][1][0], x11 = y[i][1][1];
            y[i][0][0] = x00 * c0[i].x - x10 * c0[i].y;
            y[i][0][1] = x01 * c1[i].x - x11 * c1[i].y;
            y[i][1][0] = x00 * c0[i].y + x10 * c0[i].x;
            y[i][1][1] = x01 * c1[i].y + x11 * c1[i].x;
          }
          if (E4M3)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(y[i][e >> 1][e & 1]) & 0x7FFFFFFFu);
        }
        float up = 1.f;
        if constexpr (E4M3) {
#pragma unroll
          for (int m = 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
          // the largest magnitude is in [2^(E - 127), 2^(E - 126)): to [2^7, 2^8) by 2^(134 - E). A
          // NaN or an infinity must reach the row's scores, and goes into the row's factor.
          const int E = (int)(top >> 23);
          const int k = top == 0u || E == 255 ? 0 : min(max(134 - E, -126), 126);
          up = __uint_as_float((uint32_t)(127 + k) << 23);
          if (lane == 0)
            hd->qsc[q_piece & 7][row] =
                E == 255 ? __uint_as_float(0x7FC00000u)
                         : a.softmax_scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 - k) << 23);
        }
#pragma unroll
        for (int i = 0; i < QI; ++i) {
          if (2 * lane + 64 * i >= HALF) continue;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int dim = part * HALF + 64 * i + 2 * lane;
            if constexpr (!E4M3) {
              const float x0 = y[i][part][0], x1 = y[i][part][1];
              const uint32_t w = pack_bf16x2(x0, x1);
              uint8_t* chunk = qd + (dim >> 6) * NQ * 128;
              *reinterpret_cast<uint32_t*>(chunk + sw128(row, (dim & 63) * 2)) = w;
              if (C::QLO && 64 * i < a.r) {
                // what the rounding left; nothing beside an infinity, which says all
                const float h0 = __uint_as_float(w << 16), h1 = __uint_as_float(w & 0xFFFF0000u);
                *reinterpret_cast<uint32_t*>(chunk + sw128(C::LO + row, (dim & 63) * 2)) =
                    pack_bf16x2(fabsf(h0) < INFINITY ? x0 - h0 : 0.f, fabsf(h1) < INFINITY ? x1 - h1 : 0.f);
              }
            } else {
              const float x0 = y[i][part][0] * up, x1 = y[i][part][1] * up;
              const uint32_t hi = e4m3x2(x0, x1);
              const float2 h = unpack_f16x2(e4m3_lo(hi));
              uint8_t* chunk = qd + (dim >> 7) * NQ * 128;
              *reinterpret_cast<uint16_t*>(chunk + sw128(row, dim & 127)) = (uint16_t)hi;
              *reinterpret_cast<uint16_t*>(chunk + sw128(C::LO + row, dim & 127)) = (uint16_t)e4m3x2(kLo * (x0 - h.x), kLo * (x1 - h.y));
              if (i == 0) *reinterpret_cast<uint32_t*>(qd + (CH + part) * NQ * 128 + sw128(row, 4 * lane)) = pack_f16x2(x0, x1);
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd->q_full[qb]);
      ++q_piece;
      return true;
    };
    bool ok = prepare();
    int t = 0, ks = 0;
    uint32_t kph = 0;
    // Rotation: thread (unit ku of 4 pairs, key group kg): keys kg, kg + KG, ... of the tile.
    constexpr int KG = C::HW * 2;          // 16 or 8 groups of keys
    const int ku = ht & 15, kg = ht >> 4;
    float sc[4], ss[4], tc[4], ts[4];      // turns of KG keys and of a tile
    if (rot) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 one = turn_of((double)KG, hd->itf[4 * ku + e]), all = turn_of((double)KT, hd->itf[4 * ku + e]);
        sc[e] = one.x;
        ss[e] = one.y;
        tc[e] = all.x;
        ts[e] = all.y;
      }
    }
#pragma unroll 1
    for (int piece = 0; ok && more; ++piece) {
      // with two query buffers the next unit's rows are made ahead of this one's tiles; with one
      // they wait for this unit's last scores
      p = np;
      more = piece_at(piece + 1, np);
      if (bufs.nq == 2) ok = prepare();
      if (rot) {
        float ac[4], as[4];
#pragma unroll 1
        for (int lt = 0; lt < p.ntiles && ok; ++lt, ++t) {
          const int key0 = (p.kt0 + lt) * KT + kg;
          if ((lt & 15) == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 cs = turn_of((double)key0, hd->itf[4 * ku + e]);
              ac[e] = cs.x;
              as[e] = cs.y;
            }
          }
          // the slots of the two rotated chunks, whose loads have begun (so that their barriers'
          // phases are the ones to wait for), and the copy's buffer, whose last scores are done
          int s1 = ks + ROT2;
          const bool wrap = s1 >= bufs.kslots;
          if (wrap) s1 -= bufs.kslots;
          ok = warp_wait(&hd->rot_in[t & 3], (uint32_t)(t >> 2) & 1u, abort_flag);
          if (ok && t >= bufs.nrot)
            ok = warp_wait(&hd->s_full[(t - bufs.nrot) & 1], (uint32_t)((t - bufs.nrot) >> 1) & 1u, abort_flag);
          if (ok) ok = warp_wait(&hd->full[ks], kph, abort_flag);
          if (ok) ok = warp_wait(&hd->full[s1], wrap ? kph ^ 1u : kph, abort_flag);
          if (!ok) break;
          const uint8_t* c0 = kring + ks * kTSlotBytes;
          const uint8_t* c1 = kring + s1 * kTSlotBytes;
          uint8_t* dst = rot_s + (t % bufs.nrot) * C::ROT;
          float bc[4], bs[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            bc[e] = ac[e];
            bs[e] = as[e];
          }
#pragma unroll 4
          for (int key = 0; key < KT / KG; ++key) {
            const int row = kg + KG * key;
            float x0[4], x1[4], y0[4], y1[4];
            if constexpr (E4M3) {
              // dims 4 ku .. in the first chunk's first 64 columns; the partners in the second
              // chunk's, or (128 dims) the first chunk's last 64
              e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(c0 + sw128(row, 4 * ku)), x0);
              e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(c1 + sw128(row, (PB > 1 ? 0 : 64) + 4 * ku)), x1);
            } else {
              const uint2 u0 = *reinterpret_cast<const uint2*>(c0 + sw128(row, 8 * ku));
              const uint2 u1 = *reinterpret_cast<const uint2*>(c1 + sw128(row, 8 * ku));
              x0[0] = __uint_as_float(u0.x << 16); x0[1] = __uint_as_float(u0.x & 0xFFFF0000u);
              x0[2] = __uint_as_float(u0.y << 16); x0[3] = __uint_as_float(u0.y & 0xFFFF0000u);
              x1[0] = __uint_as_float(u1.x << 16); x1[1] = __uint_as_float(u1.x & 0xFFFF0000u);
              x1[2] = __uint_as_float(u1.y << 16); x1[3] = __uint_as_float(u1.y & 0xFFFF0000u);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y0[e] = x0[e] * bc[e] - x1[e] * bs[e];
              y1[e] = x0[e] * bs[e] + x1[e] * bc[e];
              const float nc = bc[e] * sc[e] - bs[e] * ss[e];
              bs[e] = bc[e] * ss[e] + bs[e] * sc[e];
              bc[e] = nc;
            }
            const uint32_t off = sw128(row, 8 * ku);
            *reinterpret_cast<uint2*>(dst + off) =
                E4M3 ? make_uint2(pack_f16x2(y0[0], y0[1]), pack_f16x2(y0[2], y0[3])) : make_uint2(pack_bf16x2(y0[0], y0[1]), pack_bf16x2(y0[2], y0[3]));
            *reinterpret_cast<uint2*>(dst + C::CHUNK + off) =
                E4M3 ? make_uint2(pack_f16x2(y1[0], y1[1]), pack_f16x2(y1[2], y1[3])) : make_uint2(pack_bf16x2(y1[0], y1[1]), pack_bf16x2(y1[2], y1[3]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&hd->rot_ready[t % bufs.nrot]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // the next tile's first angle
            const float nc = ac[e] * tc[e] - as[e] * ts[e];
            as[e] = ac[e] * ts[e] + as[e] * tc[e];
            ac[e] = nc;
          }
          ks += NS;
          if (ks >= bufs.kslots) { ks -= bufs.kslots; kph ^= 1u; }
        }
      }
      if (ok && bufs.nq == 1) ok = prepare();
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    const int quad = warp & 3, half = (warp - 4 - C::HW) >> 2;
    const int rh = SG == 2 ? half * H : 0;                    // first row of this group
    const uint32_t lane_tmem = tmem + ((uint32_t)(quad * 32) << 16) + rh;
    const uint32_t my_o = lane_tmem + C::COL_O + (TG == 2 ? half * PB * N : 0);
    const bool key_lane = KT == 128 || lane < 16;             // TMEM lanes of M = 64: 16 per quadrant
    const int u = KT == 128 ? quad * 32 + lane : quad * 16 + (lane & 15);
    // Headroom over the running references: weights of up to 2^8, in e4m3 up to 2^8.75 < 448 (its
    // reference is kept kTop8 = 7 below the maximum, so that the largest weight is 2^7).
    constexpr float kRoom = 8.f, kRoom8 = kTop8 + kHeadroom8;
    // Where this thread's weights go: byte column of its key, swizzled, by row mod 8
    uint32_t col[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int cb = E4M3 ? u : (u & 63) * 2, r7 = (j + rh) & 7;
      col[j] = (((cb >> 4) ^ r7) << 4) | (cb & 15);
    }
    const uint32_t p_mine = smem_u32(p_s) + rh * 128 + (E4M3 ? 0 : (u >> 6) * N * 128);
    uint32_t meets = 0;
    bool ok = true;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd->hmeet[half]);
      ok = warp_wait(&hd->hmeet[half], meets & 1u, abort_flag);
      ++meets;
    };
    // e4m3: this thread's key's scales are read a tile of its group ahead, the table entry that leads
    // to them two tiles ahead, past the ends of units too, so that no tile waits for either
    float ks_next = kZeroRowScale, vs_next = kZeroRowScale;
    int entry = -1;
    auto read_entry = [&](const TilePiece& w, int lt) {
      const int pos = (w.kt0 + lt) * KT + u;
      entry = lt < w.ntiles && pos >= w.first && pos < w.end ? fresh(a.c.table + (size_t)w.b * a.c.max_blocks + (pos >> a.c.page_shift)) : -1;
    };
    auto read_scales = [&](const TilePiece& w, int lt) {  // of tile lt, by its entry; and the next one's entry
      const int pos = (w.kt0 + lt) * KT + u;
      ks_next = vs_next = kZeroRowScale;   // of keys that are not there, too
      if ((unsigned)entry < (unsigned)a.c.num_pages) {
        const size_t row = page_row(a.c, entry, w.kvh, pos & ((1 << a.c.page_shift) - 1));
        ks_next = fresh(a.c.k_scales + row);
        if (!SAME) vs_next = fresh(a.c.v_scales + row);
      }
      read_entry(w, lt + TG);
    };
    int t0 = 0;                            // tiles of the units before
#pragma unroll 1
    for (int piece = 0; ok && piece_at(piece, p); ++piece) {
      const int lt0 = TG == 2 ? (half ^ t0) & 1 : 0;  // this group's first tile; then every TG-th
      // m: reference of the sums; mv: of the weights (bf16: the same one). A row that has seen no key
      // has the lowest finite number.
      float m_run[H], mv_run[E4M3 ? H : 1], l_acc[H];
#pragma unroll
      for (int q = 0; q < H; ++q) {
        m_run[q] = -3.3e38f;
        if constexpr (E4M3) mv_run[q] = -3.3e38f;
        l_acc[q] = 0.f;
      }
      // the references are the same in every lane and warp of the group; a copy in shared memory
      // serves what runs once in a while (the group meets before anyone reads it)
      if (quad == 0 && lane < H) hd->refs[piece & 1][half][0][lane] = hd->refs[piece & 1][half][1][lane] = -3.3e38f;
      if (E4M3 && piece == 0) {
        read_entry(p, lt0);
        read_scales(p, lt0);
      }
#pragma unroll 1
      for (int lt = lt0; lt < p.ntiles && ok; lt += TG) {
        float kscale = 1.f, vscale = 1.f;
        if constexpr (E4M3) {
          kscale = ks_next;
          vscale = SAME ? ks_next : vs_next;
          read_scales(p, lt + TG);
        }
        const int t = t0 + lt, bb = t & 1, k0 = (p.kt0 + lt) * KT;
        ok = warp_wait(&hd->s_full[bb], (uint32_t)(t >> 1) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        // sv: scores in log2 units; lv: log2 of the value scale, a power of two (NaN stays NaN)
        float sv[H], lv = 0.f;
        tmem_ld_n<H>(lane_tmem + bb * C::SN, reinterpret_cast<uint32_t*>(sv));
        if constexpr (E4M3) {
          lv = vscale == vscale ? (float)((int)(__float_as_uint(vscale) >> 23) - 127) : vscale;
          float s2[H];
          tmem_ld_n<H>(lane_tmem + bb * C::SN + C::LO, reinterpret_cast<uint32_t*>(s2));
          tmem_ld_wait();
          const float* cf = &hd->qsc[piece & 7][rh];
#pragma unroll
          for (int q = 0; q < H; ++q) sv[q] = fmaf(s2[q], 1.f / kLo, sv[q]) * (cf[q] * kscale);
        } else {
          const float cf = a.softmax_scale * 1.4426950408889634f;
          if constexpr (C::QLO) {
            float s2[H];
            tmem_ld_n<H>(lane_tmem + bb * C::SN + C::LO, reinterpret_cast<uint32_t*>(s2));
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < H; ++q) sv[q] = (sv[q] + s2[q]) * cf;
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < H; ++q) sv[q] *= cf;
          }
        }
        // tiles that every row sees whole need no mask (rows past the unit's read zero queries)
        if (k0 + KT - 1 > p.len || k0 < p.first || (a.is_local && k0 < p.end - a.window) || !key_lane) {
          const int pos = key_lane ? k0 + u : 0x7fffffff;
#pragma unroll
          for (int q = 0; q < H; ++q) {
            const int qp = hd->qpos[piece & 7][rh + q];
            if (pos > qp || (a.is_local && pos <= qp - a.window)) sv[q] = -INFINITY;
          }
        }
        // ---- does any score pass its reference by more than the headroom?
        float over = -INFINITY, over8 = -INFINITY;
#pragma unroll
        for (int q = 0; q < H; ++q) {
          over = fmaxf(over, sv[q] - m_run[q]);
          if constexpr (E4M3) over8 = fmaxf(over8, sv[q] - mv_run[q]);
        }
        bool pass = over > kRoom || (E4M3 && over8 + lv > kRoom8);
        pass = __any_sync(0xffffffffu, pass);
        if (lane == 0) hd->viol[meets & 1u][half][quad] = pass;
        meet();
        if (!ok) break;
        const int4 vv = *reinterpret_cast<const int4*>(hd->viol[(meets - 1) & 1u][half]);
        if (vv.x | vv.y | vv.z | vv.w) {
          // the four warps agree on the tile's maxima and raise the references to them
          auto& red = hd->red[meets & 1u][half];
          if constexpr (E4M3) {
            if (vscale == 1.f && zero_row(a, SAME ? a.c.k : a.c.v, p, k0 + u)) lv = -126.f;  // log2 of kZeroRowScale
            __syncwarp();
          }
          {
            float y[H], z[H];
#pragma unroll
            for (int q = 0; q < H; ++q) {
              y[q] = warp_max(sv[q]);
              z[q] = E4M3 ? warp_max(sv[q] + lv) : 0.f;
            }
            if (lane == 0) {
#pragma unroll
              for (int q = 0; q < H; q += 4) {
                *reinterpret_cast<float4*>(&red[0][quad][q]) = make_float4(y[q], y[q + 1], y[q + 2], y[q + 3]);
                if (E4M3) *reinterpret_cast<float4*>(&red[1][quad][q]) = make_float4(z[q], z[q + 1], z[q + 2], z[q + 3]);
              }
            }
          }
          meet();
          if (!ok) break;
          // one warp forms the new references and the factors, the others take them from it
          auto& refs = hd->refs[piece & 1][half];
          if (quad == 0 && lane < H) {
            auto top4 = [&](const float(*x)[H <= 8 ? 8 : 32]) { return fmaxf(fmaxf(x[0][lane], x[1][lane]), fmaxf(x[2][lane], x[3][lane])); };
            const float m_old = refs[0][lane], m_new = fmaxf(m_old, top4(red[0]));
            float f = fast_exp2(m_old - m_new);
            refs[0][lane] = m_new;
            hd->step[half][0][lane] = f;
            if constexpr (E4M3) {
              const float mv_old = refs[1][lane], mv_new = fmaxf(mv_old, top4(red[1]) - kTop8);
              refs[1][lane] = mv_new;
              f = fast_exp2(mv_old - mv_new);
            }
            hd->step[half][1][lane] = f;
          }
          meet();
          if (!ok) break;
          float al[H];
#pragma unroll
          for (int q = 0; q < H; ++q) {
            m_run[q] = refs[0][q];
            if constexpr (E4M3) mv_run[q] = refs[1][q];
            l_acc[q] *= hd->step[half][0][q];
            al[q] = hd->step[half][1][q];
          }
          // The group's output is touched once the products of its tile before are done (its first
          // tile in a unit has nothing to rescale).
          if (lt >= TG) {
            ok = warp_wait(&hd->pv_done[(t - TG) & 1], (uint32_t)((t - TG) >> 1) & 1u, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < PB * (E4M3 ? 2 : 1); ++i) {
              uint32_t o[H];
              const uint32_t ta = my_o + (uint32_t)((i % PB) * N + (i / PB) * C::LO);
              tmem_ld_n<H>(ta, o);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < H; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * al[q]);
              tmem_st_n<H>(ta, o);
            }
            tmem_st_wait();
          }
        }
        // ---- weights: buffer bb was read by the products of tile t - 2
        if (t >= 2) {
          ok = warp_wait(&hd->pv_done[bb], (uint32_t)((t - 2) >> 1) & 1u, abort_flag);
          if (!ok) break;
        }
        const uint32_t pb = p_mine + bb * C::P_B;
        if constexpr (E4M3) {
          // lo's dither, by the key's position: [-1/2, 1/2) of its smallest step, 2^-9
          const float dither = (float)(int)((uint32_t)(k0 + u) * 2654435769u) * 0x1p-41f;
#pragma unroll
          for (int q = 0; q < H; q += 2) {
            l_acc[q] += fast_exp2(sv[q] - m_run[q]);
            l_acc[q + 1] += fast_exp2(sv[q + 1] - m_run[q + 1]);
            const float w0 = fast_exp2(sv[q] + lv - mv_run[q]), w1 = fast_exp2(sv[q + 1] + lv - mv_run[q + 1]);
            const uint32_t hi = e4m3x2(w0, w1);
            const float2 h = unpack_f16x2(e4m3_lo(hi));
            const uint32_t lo = e4m3x2(fmaf(w0 - h.x, kLo, dither), fmaf(w1 - h.y, kLo, dither));
            st_shared_u8(pb + q * 128 + col[q & 7], hi);
            st_shared_u8(pb + (q + 1) * 128 + col[(q + 1) & 7], hi >> 8);
            // LO is a multiple of 8 rows: the same swizzle
            st_shared_u8(pb + (C::LO + q) * 128 + col[q & 7], lo);
            st_shared_u8(pb + (C::LO + q + 1) * 128 + col[(q + 1) & 7], lo >> 8);
          }
        } else {
#pragma unroll
          for (int q = 0; q < H; ++q) {
            const __nv_bfloat16 w = __float2bfloat16_rn(fast_exp2(sv[q] - m_run[q]));
            l_acc[q] += __bfloat162float(w);
            if (key_lane) st_shared_u16(pb + q * 128 + col[q & 7], __bfloat16_as_ushort(w));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&hd->p_full[bb]);
      }
      if (!ok) break;
      // ---- the unit's (or its part's) output. The rows' sums: halves of the values go to the lanes of
      // either half of the warp until each lane holds one row, then over the four warps.
      {
        constexpr int HP = H <= 8 ? 8 : 32;
        float x[HP];
#pragma unroll
        for (int q = 0; q < HP; ++q) x[q] = q < H ? l_acc[q] : 0.f;
        const int mine = scatter_sums<16, HP / 2>(x, lane);  // the row this lane ends up with
        if ((lane & (32 / HP - 1)) == 0) hd->sums[piece & 1][half][quad][mine] = x[0];
        meet();
        if (!ok) break;
      }
      // The next unit's first scales are read under this one's output.
      const TilePiece& np = hd->piece[(piece + 1) & 7];
      const int lt0_next = TG == 2 ? (half ^ (t0 + p.ntiles)) & 1 : 0;
      if constexpr (E4M3) {
        ok = warp_wait(&hd->piece_full[(piece + 1) & 7], (uint32_t)((piece + 1) >> 3) & 1u, abort_flag);
        if (!ok) break;
        read_entry(np, lt0_next);
      }
      // The groups that share the rows meet: their sums and references are there to read.
      if (TG == 2) {
        if (lane == 0) mbar_arrive(&hd->o_meet);
        ok = warp_wait(&hd->o_meet, (uint32_t)piece & 1u, abort_flag);
        if (!ok) break;
      }
      t0 += p.ntiles;
      for (int i = 1; i <= min(TG, p.ntiles) && ok; ++i)
        ok = warp_wait(&hd->pv_done[(t0 - i) & 1], (uint32_t)((t0 - i) >> 1) & 1u, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if constexpr (E4M3) read_scales(np, lt0_next);
      // lane q forms row q's factors (of either group's output), log-sum-exp and place
      float fac[TG] = {};
      int place = -1;
      if (lane < H && rh + lane < p.rows) {
        float l[TG], m[TG], mv[TG], top = -3.0e38f, sum = 0.f;
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int gi = TG == 2 ? g : half;
          const float* x = &hd->sums[piece & 1][gi][0][lane];
          constexpr int Q = H <= 8 ? 8 : 32;
          l[g] = (x[0] + x[Q]) + (x[2 * Q] + x[3 * Q]);
          m[g] = fmaxf(hd->refs[piece & 1][gi][0][lane], -3.0e38f);
          mv[g] = fmaxf(hd->refs[piece & 1][gi][1][lane], -3.0e38f);
          top = fmaxf(top, m[g]);
        }
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          fac[g] = fast_exp2(m[g] - top);
          sum += l[g] * fac[g];
        }
        const int row = rh + lane;
        place = p.slot >= 0 ? p.slot * NR + row : hd->orow[piece & 7][row];
        const float inv = sum > 0.f ? __fdividef(1.f, sum) : sum == 0.f ? 0.f : sum;  // a NaN sum stays one
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          fac[g] *= inv;
          if (E4M3) fac[g] *= fast_exp2(mv[g] - m[g]);
        }
        if (quad == 0 && (TG == 1 || half == 0)) {
          const float lse = sum > 0.f ? (top + __log2f(sum)) * 0.6931471805599453f : sum == 0.f ? -INFINITY : sum;
          if (p.slot >= 0) a.partial_lse[place] = lse;
          else if (a.lse) a.lse[place] = lse;
        }
      }
      const bool wide = p.slot >= 0 || a.out_f32;
      uint8_t* out = p.slot >= 0 ? reinterpret_cast<uint8_t*>(a.partial_o) : static_cast<uint8_t*>(a.out);
      // A block of 128 dims at a time, 32 dims a warp; groups that share the rows take turns. With
      // one tile only its group has an output.
      const int gone = TG == 2 && p.ntiles == 1 ? (t0 & 1) : -1;
#pragma unroll 1
      for (int m = TG == 2 ? half : 0; m < PB; m += TG) {
        float v[H];
#pragma unroll
        for (int q = 0; q < H; ++q) v[q] = 0.f;
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          if (g == gone) continue;
          const uint32_t ta = lane_tmem + C::COL_O + (uint32_t)((g * PB + m) * N);
          uint32_t o[H], o2[H];
          tmem_ld_n<H>(ta, o);
          if constexpr (E4M3) tmem_ld_n<H>(ta + C::LO, o2);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < H; ++q) {
            const float x = E4M3 ? fmaf(__uint_as_float(o2[q]), 1.f / kLo, __uint_as_float(o[q])) : __uint_as_float(o[q]);
            v[q] += x * __shfl_sync(0xffffffffu, fac[g], q);
          }
        }
        const size_t col = m * 128 + quad * 32 + lane;
#pragma unroll
        for (int q = 0; q < H; ++q) {
          const int pl = __shfl_sync(0xffffffffu, place, q);
          if (pl < 0) continue;
          if (wide) reinterpret_cast<float*>(out)[(size_t)pl * D + col] = v[q];
          else reinterpret_cast<__nv_bfloat16*>(out)[(size_t)pl * D + col] = __float2bfloat16_rn(v[q]);
        }
      }
      // O^T has been read: the next unit's first products may overwrite it
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd->o_empty);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// 4-D map over a page pool's rows as 128-byte column chunks: boxes of `rows` rows of `chunks` chunks.
static bool tile_map(CUtensorMap* m, const void* base, const PagedCache& c, bool e4m3, int rows, int chunks) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int esz = e4m3 ? 1 : 2, ps = 1 << c.page_shift;
  cuuint64_t dims[4] = {(cuuint64_t)(128 / esz), (cuuint64_t)ps, (cuuint64_t)(c.d * esz / 128), (cuuint64_t)c.num_pages * c.hkv};
  cuuint64_t strides[3] = {(cuuint64_t)c.d * esz, 128, (cuuint64_t)c.d * ps * esz};
  cuuint32_t box[4] = {(cuuint32_t)(128 / esz), (cuuint32_t)rows, (cuuint32_t)chunks, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The last table made on this thread is kept: every layer of a kind has the same one.
static const TileTurns& tile_turns(int d, double log2_base) {
  static thread_local TileTurns t;
  static thread_local int last_d = 0;
  static thread_local double last_base = 0.0;
  if (last_d != d || last_base != log2_base) {
    for (int j = 0; j < 64; ++j) t.freq[j] = exp2(-2.0 * j / d * log2_base) * 0.15915494309189533577;
    t.step64 = exp2(-128.0 / d * log2_base);
    last_d = d;
    last_base = log2_base;
  }
  return t;
}

template <int D, bool E4M3, bool SAME, int SG, int H>
static cudaError_t launch_tile_t(PagedAttendArgs a, bool cut, long long units, cudaStream_t stream) {
  using C = TileCfg<D, E4M3, SAME, SG, H>;
  const TileBufs b = tile_bufs<D, E4M3, SAME, SG, H>(SAME && a.r > 0);
  if (b.kslots < C::NS || (!SAME && b.vslots < C::NS)) return cudaErrorInvalidValue;
  static std::atomic<bool> ready[64];
  cudaError_t e = allow_smem(paged_tile_kernel<D, E4M3, SAME, SG, H>, 232448, ready);
  if (e != cudaSuccess) return e;
  const int box = std::min(1 << a.c.page_shift, C::KT), chunks = box == C::KT ? C::G : 1;
  CUtensorMap k, v;
  if (!tile_map(&k, a.c.k, a.c, E4M3, box, chunks)) return cudaErrorInvalidValue;
  v = k;
  if (!SAME && !tile_map(&v, a.c.v, a.c, E4M3, box, chunks)) return cudaErrorInvalidValue;
  const int grid = cut ? kSms : (int)std::min<long long>(units, kSms);
  a.cut = cut;
  a.teams = grid;
  a.run_step = 1;
  a.unit_rows = C::NR;
  a.unit_shift = C::KT == 128 ? 7 : 6;
  e = launch_follower(paged_tile_kernel<D, E4M3, SAME, SG, H>, dim3(grid), dim3(kTThreads), 232448, stream, k, v, a, tile_turns(D, a.log2_base));
  if (e != cudaSuccess || !cut) return e;
  return launch_paged_merge(a, stream);
}

template <int D, bool E4M3>
static cudaError_t launch_tile_d(const PagedAttendArgs& a, const PagedRowsShape& f, long long units, cudaStream_t stream) {
  const bool same = a.c.v == nullptr;
  switch (f.unit_rows) {
    case 8: return same ? launch_tile_t<D, E4M3, true, 1, 8>(a, f.cut, units, stream) : launch_tile_t<D, E4M3, false, 1, 8>(a, f.cut, units, stream);
    case 40: return same ? launch_tile_t<D, E4M3, true, 2, 20>(a, f.cut, units, stream) : launch_tile_t<D, E4M3, false, 2, 20>(a, f.cut, units, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_paged_tile(const PagedAttendArgs& a, const PagedRowsShape& f, bool e4m3, cudaStream_t stream) {
  const long long units = (long long)a.batch * a.row_groups * a.c.hkv;
  switch (a.c.d) {
    case 128: return e4m3 ? launch_tile_d<128, true>(a, f, units, stream) : launch_tile_d<128, false>(a, f, units, stream);
    case 256: return e4m3 ? launch_tile_d<256, true>(a, f, units, stream) : launch_tile_d<256, false>(a, f, units, stream);
    case 512: return e4m3 ? launch_tile_d<512, true>(a, f, units, stream) : launch_tile_d<512, false>(a, f, units, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gattn
