// paged.h -- the paged KV cache as the kernels see it, and the launch interfaces of the
// paged-cache operators and of the draft verification.
#pragma once
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"

namespace gattn {

// One lane of a converged warp. tcgen05.mma takes its descriptors from uniform registers: behind
// this predicate the compiler knows that one thread runs and moves them there directly, behind
// `lane == 0` it adds a loop over the active lanes to every MMA (measured per 128 x 16 x 16 MMA:
// 51 cycles against 111 to 204).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{.reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q;}" : "=r"(p));
  return p != 0;
}

// Allow `kernel` `bytes` of dynamic shared memory on the current device, once per device.
template <typename F>
cudaError_t allow_smem(F kernel, int bytes, std::atomic<bool>* ready /* [64] */) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready[dev].store(true, std::memory_order_release);
  return e;
}

enum : int { kStatusPage = 4 };  // device status word: a block-table entry outside the pool

// A load in a kernel that follows closely (follow(), below): its blocks may be resident while a
// kernel before it still writes what it is going to read, its predecessors' results in the
// workspace as well as the call's inputs. The read-only path (__ldg, ld.global.nc) is for data that
// no one writes while the kernel lives, and the compiler may move such a load over the wait; an
// ordinary one is ordered by it.
template <typename T>
__device__ __forceinline__ T fresh(const T* p) {
  return *p;
}

struct PagedCache {
  uint8_t* k;               // [pages, Hkv, page_size, d] bf16 or e4m3
  uint8_t* v;               // null for K=V
  float* k_scales;          // [pages, Hkv, page_size], e4m3 only
  float* v_scales;
  const int32_t* table;     // [batch, max_blocks]
  int num_pages, page_shift, max_blocks;  // page_size = 1 << page_shift
  int hkv, d;
};

// Page of block `blk` of sequence b, or -1 (recorded) when the entry is outside the pool.
__device__ __forceinline__ int page_of(const PagedCache& c, int b, int blk) {
  const int pg = fresh(c.table + (size_t)b * c.max_blocks + blk);
  if ((unsigned)pg < (unsigned)c.num_pages) return pg;
  atomicOr(&g_status, kStatusPage);
  return -1;
}

// Index of (page, head, slot) among the rows of the pool.
__device__ __forceinline__ size_t page_row(const PagedCache& c, int page, int head, int slot) {
  return (((size_t)page * c.hkv + head) << c.page_shift) + slot;
}

// A row of zeros has the scale 1 (gemma_attn_paged_append), whatever its neighbours'. Where value
// scales are folded into softmax weights, such a row is taken to have this one as soon as it would
// raise the weights' reference: it adds nothing to an output, and the weights that do count would
// go to the bottom of their type. Rows are looked at for that only there, and only those with the
// scale 1: where a cache has no other scale that costs 2 to 8 percent (on every tile 5 to 40).
constexpr float kZeroRowScale = 0x1p-126f;

// Sequence of row t: the b with cu[b] <= t < cu[b + 1] (t < cu[batch], cu[0] = 0).
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int batch, int t) {
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (fresh(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The kernels of an attend call follow one another closely: each lets the next be launched as soon
// as all its blocks run, and waits for the one before it to complete (and, through it, all before
// that) ahead of its first access to global memory. That holds for the first one and whatever
// kernel stands before it in the stream, too.
__device__ __forceinline__ void follow() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_follower(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

struct PagedAppendArgs {
  PagedCache c;
  const uint16_t* new_k;
  const uint16_t* new_v;
  const int32_t* cu_q;
  const int32_t* lens;
  int batch, total_q;
  int r;                    // rotated pairs of the stored keys (0 for K=V)
  // theta_j / (2 pi) for j = 0, 8, 16, ..., and base^(-2 / d), from one pair's frequency to the next
  double freq8[32], freq_step;
};
template <bool E4M3>
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);

struct PagedGatherArgs {
  PagedCache c;
  const int32_t* starts;
  const int32_t* cu_out;
  void* out_k;
  void* out_v;
  int batch, total_out;
};
template <bool E4M3, bool F32>
cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t stream);

struct PagedAttendArgs {
  PagedCache c;
  const uint16_t* q;        // [T, Hq, d]
  const int32_t* cu_q;
  const int32_t* lens;
  void* out;                // [T, Hq, d]
  float* lse;               // [T, Hq] or null
  int out_f32;
  int batch, total_q, max_q, max_len;
  int hq, group;            // query heads, query heads per KV head
  int is_local, window;
  int r;                    // rotated pairs
  double log2_base;
  float softmax_scale;
  // short sequences: parts of cut units, two a team
  float* partial_o;         // [2 teams, unit_rows, d]
  float* partial_lse;       // [2 teams, unit_rows]
  int4* joins;              // [teams]: the unit that a team's run begins and does not end (paged_merge_kernel)
  const int* rest;          // beside chunk_of: sequences with rows that are not chunks
  int row_groups;           // most units of one KV head of a sequence
  const int* chunk_of;      // [batch], >= 0: the sequence is chunk_kernel's; null: there are none
  // set at the launch: units are cut into equal runs; teams; a run is a multiple of run_step;
  // rows of a unit (8 or 40), log2 of the keys of a block
  int cut, teams, run_step, unit_rows, unit_shift;
};

constexpr int kSms = 148;

// How a call's short sequences run.
struct PagedRowsShape {
  int tile;                 // the tensor-core kernel (paged_tile.cu), not the one below
  int unit_rows, row_groups;
  int cut;                  // units are cut into equal runs
  int parts;                // places for parts of cut units
  long long line;           // most blocks of all units together
  // row-group kernel (paged_decode.cu)
  int warp_teams;           // units go to single warps, not CTAs
  int q_rows;               // rows of the fullest group
  int nw, nsk, nsv;         // warps of a CTA; key (K=V) and value stages of a warp's ring
};
// `rows` rows per KV head and `keys` visible keys at most.
PagedRowsShape paged_rows_shape(int head_dim, bool local, int rotated, int batch, int hkv, int rows, long long keys);
cudaError_t launch_paged_rows(const PagedAttendArgs& a, const PagedRowsShape& f, bool e4m3, cudaStream_t stream);
cudaError_t launch_paged_tile(const PagedAttendArgs& a, const PagedRowsShape& f, bool e4m3, cudaStream_t stream);
cudaError_t launch_paged_merge(const PagedAttendArgs& a, cudaStream_t stream);

// Long chunks (paged_chunk.cu): the device-side plan and the buffers it names, all in the
// call's workspace.
struct ChunkPlan {
  int* header;              // [3]: entries of list, entries of merges, sequences with rows that are not chunks
  int* chunk_of;            // [batch]: index among the chunk sequences, or -1
  int* tile0;               // [batch + 1]: first 128-position tile of the side copies
  int* unit0;               // [batch + 1]: first unit
  int4* list;               // pairs {sequence, unit of it, first key tile, end}, {partial slot or -1, -, -, -}
  int4* merges;             // {sequence, unit of it, first slot, pieces}
  uint16_t* q_side;         // [T, Hq, q_cols (twice with q_lo)] rotated 64-dim chunks of the queries
  uint16_t* k_rot;          // [Hkv, rot_rows, k_cols] rotated chunks of K=V keys, every tile
  uint16_t* k_copy;         // [Hkv, copy_rows, d] bf16 rows of every tile (e4m3) or of the cut ones (bf16)
  uint16_t* v_copy;
  float* part_o;            // [slots, Hkv, rows, d]
  float* part_lse;          // [slots, Hkv, rows]
  uint32_t q_mask, k_mask;  // 64-dim chunks that come from q_side / k_rot
  int q_cols, k_cols;
  int q_lo;                 // rotated queries in two bf16 parts (ChunkCfg)
  long long rot_rows, copy_rows;
  int e4m3;
  int min_rows;             // sequences with more rows per KV head than this are chunks
  int tokens, rows;         // of a unit: tokens, and rows with their padding (128 or 256)
  int units_x;              // units of a list entry: KV heads x output parts
  int clusters;             // CTAs or pairs that walk the list
};
struct ChunkMaps {
  CUtensorMap q, qs, k, k_rot, k_copy, v, v_copy;
};
cudaError_t launch_chunk(const ChunkMaps& maps, const PagedAttendArgs& a, const ChunkPlan& p, int units_bound,
                         int slots, cudaStream_t stream);

struct DraftArgs {
  const void* target;
  const void* draft;        // null: certain drafts
  const int32_t* tokens;
  const int32_t* lens;      // null: all max_draft
  const float* uniforms;
  const float* noise;
  int32_t* accepted;
  int32_t* out;
  int batch, max_draft, vocab;
};
cudaError_t launch_draft_verify(const DraftArgs& a, bool bf16, cudaStream_t stream);

}  // namespace gattn
