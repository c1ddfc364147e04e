// paged_api.cu -- entry points of the paged-cache operators and of the draft verification:
// argument checks, workspace carving and launches.
#include "../../include/gemma_attn.h"
#include "kernels.h"
#include "paged.h"

namespace gattn {
namespace {

// Checks shared by the paged entry points; fills the kernels' view of the cache.
int paged_prepare(const gemma_attn_params* p, const gemma_attn_paged_cache* c, PagedCache* out, bool* e4m3) {
  const int rc = check_params(p);
  if (rc != GEMMA_ATTN_OK) return rc;
  if (!c) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (p->kind == GEMMA_ATTN_BIDIR) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if (p->head_dim < 64 || p->num_q_heads / p->num_kv_heads > 128) return GEMMA_ATTN_ERR_UNSUPPORTED;
  const bool global = p->kind == GEMMA_ATTN_GLOBAL;
  if (c->dtype != GEMMA_ATTN_PAGES_BF16 && c->dtype != GEMMA_ATTN_PAGES_E4M3) return GEMMA_ATTN_ERR_INVALID_ARG;
  *e4m3 = c->dtype == GEMMA_ATTN_PAGES_E4M3;
  if (!c->k_pages || !c->block_table || global != (c->v_pages == nullptr)) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (*e4m3 != (c->k_scales != nullptr) || (*e4m3 && !global) != (c->v_scales != nullptr)) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->max_blocks < 1) return GEMMA_ATTN_ERR_INVALID_ARG;
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if ((long long)c->num_pages * p->num_kv_heads > 0x7fffffffll) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if (((uintptr_t)c->k_pages | (uintptr_t)c->v_pages | (uintptr_t)c->k_scales | (uintptr_t)c->v_scales) & 15u)
    return GEMMA_ATTN_ERR_MISALIGNED;
  if ((uintptr_t)c->block_table & 3u) return GEMMA_ATTN_ERR_MISALIGNED;
  out->k = static_cast<uint8_t*>(c->k_pages);
  out->v = static_cast<uint8_t*>(c->v_pages);
  out->k_scales = c->k_scales;
  out->v_scales = c->v_scales;
  out->table = c->block_table;
  out->num_pages = c->num_pages;
  out->page_shift = shift;
  out->max_blocks = c->max_blocks;
  out->hkv = p->num_kv_heads;
  out->d = p->head_dim;
  return GEMMA_ATTN_OK;
}

// Lengths, prefixes and log-sum-exps are read and written 4 bytes at a time.
bool aligned4(const void* x, const void* y, const void* z = nullptr) {
  return (((uintptr_t)x | (uintptr_t)y | (uintptr_t)z) & 3u) == 0;
}

int launched(cudaError_t e, int launches) {
  if (e != cudaSuccess) return GEMMA_ATTN_ERR_LAUNCH;
  set_launch_count(launches);
  return GEMMA_ATTN_OK;
}

// Rows per KV head up to which a sequence takes the kernels of short sequences; with more it is a
// chunk. Up to 40 rows they are one unit there (paged_rows_shape), up to 80 two, each with all the
// keys read. Measured, us, with the border at 40, 64 and 128 rows: 16 sequences of 1k to 32k keys, K=V of
// 512 dims, 64 rows: chunks 324, units 218 in e4m3, 250 and 208 in bf16; 80 rows: 332 and 220, 258 and
// 210; 128 rows (four units): 344 and 382, 270 and 370. On a window of 1,024 with 256 dims, where a
// chunk's fixed launches weigh less than second units: 60 rows 125 and 171, 80 rows 132 and 173.
constexpr int kChunkMinRows = 64;

// How an attend call's work is cut, and what of the workspace each part takes (byte offsets).
struct AttendPlan {
  PagedRowsShape shape;             // the sequences that are not chunks
  size_t part_o, part_lse, joins;
  bool chunk;                       // some sequence may have more rows than kChunkMinRows
  bool pair;
  int tokens, units_x, clusters, slots, units, seqs;
  uint32_t q_mask, k_mask;
  bool q_lo;                        // rotated queries in two bf16 parts
  long long tiles, copy_rows;
  size_t header, chunk_of, tile0, unit0, list, merges, q_side, k_rot, k_copy, v_copy, c_part_o, c_part_lse;
  size_t total;
};

int attend_plan(const gemma_attn_params* p, bool e4m3, int batch, int total_q, int max_q, int max_cache_len, AttendPlan* L) {
  if (batch < 1 || total_q < 0 || max_q < 0 || max_cache_len < 0) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch > 65535 || (long long)max_cache_len + max_q > 0x7fffff00ll) return GEMMA_ATTN_ERR_UNSUPPORTED;
  const long long rows = (long long)total_q * p->num_q_heads;
  if (rows > 0x7fffffffll) return GEMMA_ATTN_ERR_UNSUPPORTED;
  const int d = p->head_dim, hkv = p->num_kv_heads, group = p->num_q_heads / hkv;
  const bool local = p->kind == GEMMA_ATTN_LOCAL;
  *L = AttendPlan{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  const long long keys = local ? std::min<long long>(max_cache_len, p->window) + max_q : (long long)max_cache_len + max_q;
  L->chunk = (long long)max_q * group > kChunkMinRows;
  const int r = rotated_pairs(p->rope_p, d);
  L->shape = paged_rows_shape(d, local, r, batch, hkv, L->chunk ? kChunkMinRows : std::max(1, max_q * group), keys);
  if (L->shape.line > 0x7fffffffll) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if (L->shape.cut) {
    L->part_o = take((size_t)L->shape.parts * L->shape.unit_rows * d * 4);
    L->part_lse = take((size_t)L->shape.parts * L->shape.unit_rows * 4);
    L->joins = take((size_t)L->shape.parts / 2 * sizeof(int4));
  }
  if (L->chunk) {
    L->q_mask = rotated_chunk_mask(d, r);
    L->k_mask = local ? 0u : L->q_mask;
    L->q_lo = local && d <= 256 && L->q_mask != 0;
    L->pair = d >= 128 && (long long)max_q * group > 128;
    L->tokens = 128 / group * (L->pair ? 2 : 1);
    L->units_x = hkv * (d > 256 ? d / 256 : 1);
    L->clusters = L->pair ? 74 : 148;
    // pieces of cut units: under 4 clusters / units_x (chunk_plan_kernel)
    L->slots = 4 * L->clusters / L->units_x + 1;
    // chunk sequences have at least kChunkMinRows / group + 1 tokens each
    L->seqs = std::min(batch, total_q / (kChunkMinRows / group + 1));
    L->units = total_q / L->tokens + L->seqs;
    const long long most = (long long)L->seqs * (((long long)max_cache_len + max_q + 127) / 128);
    L->tiles = most;
    if (local)  // window and chunk, and a tile that either end cuts
      L->tiles = std::min(most, ((long long)L->seqs * p->window + total_q) / 128 + 2ll * L->seqs + 1);
    L->copy_rows = e4m3 ? L->tiles * 128 : (long long)L->seqs * 256;
    if (L->tiles * 128 > 0x7fffffffll) return GEMMA_ATTN_ERR_UNSUPPORTED;
    L->header = take(12);
    L->chunk_of = take((size_t)batch * 4);
    L->tile0 = take(((size_t)batch + 1) * 4);
    L->unit0 = take(((size_t)batch + 1) * 4);
    L->list = take((size_t)(L->units + L->slots) * 32);
    L->merges = take((size_t)L->slots * 16);
    L->q_side = take((size_t)rows * __builtin_popcount(L->q_mask) * (L->q_lo ? 256 : 128));
    L->k_rot = take((size_t)L->tiles * 128 * hkv * __builtin_popcount(L->k_mask) * 128);
    L->k_copy = take((size_t)L->copy_rows * hkv * d * 2);
    L->v_copy = local ? take((size_t)L->copy_rows * hkv * d * 2) : L->k_copy;
    const size_t prow = (size_t)L->slots * hkv * (L->pair ? 256 : 128);
    L->c_part_o = take(prow * d * 4);
    L->c_part_lse = take(prow * 4);
  }
  L->total = at;
  return GEMMA_ATTN_OK;
}

// 3-D bf16 map over [n2][n1][n0] with a {64, b1, b2} box, 128-byte swizzle.
bool box_map(CUtensorMap* m, const void* base, long long n0, long long n1, long long n2, int b1, int b2) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
  cuuint64_t strides[2] = {(cuuint64_t)n0 * 2, (cuuint64_t)(n0 * n1) * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_attend_chunks(const gemma_attn_params* params, const PagedAttendArgs& a, bool e4m3, const AttendPlan& L,
                         uint8_t* ws, cudaStream_t stream) {
  ChunkPlan p{};
  p.header = reinterpret_cast<int*>(ws + L.header);
  p.chunk_of = reinterpret_cast<int*>(ws + L.chunk_of);
  p.tile0 = reinterpret_cast<int*>(ws + L.tile0);
  p.unit0 = reinterpret_cast<int*>(ws + L.unit0);
  p.list = reinterpret_cast<int4*>(ws + L.list);
  p.merges = reinterpret_cast<int4*>(ws + L.merges);
  p.q_side = reinterpret_cast<uint16_t*>(ws + L.q_side);
  p.k_rot = reinterpret_cast<uint16_t*>(ws + L.k_rot);
  p.k_copy = reinterpret_cast<uint16_t*>(ws + L.k_copy);
  p.v_copy = reinterpret_cast<uint16_t*>(ws + L.v_copy);
  p.part_o = reinterpret_cast<float*>(ws + L.c_part_o);
  p.part_lse = reinterpret_cast<float*>(ws + L.c_part_lse);
  p.q_mask = L.q_mask;
  p.k_mask = L.k_mask;
  p.q_cols = __builtin_popcount(L.q_mask) * 64;
  p.q_lo = L.q_lo ? 1 : 0;
  p.k_cols = __builtin_popcount(L.k_mask) * 64;
  p.rot_rows = L.tiles * 128;
  p.copy_rows = L.copy_rows;
  p.e4m3 = e4m3 ? 1 : 0;
  p.min_rows = kChunkMinRows;
  p.tokens = L.tokens;
  p.rows = L.pair ? 256 : 128;
  p.units_x = L.units_x;
  p.clusters = L.clusters;
  const int d = a.c.d, hkv = a.c.hkv, ps = 1 << a.c.page_shift, tpc = 128 / a.group, keys = L.pair ? 64 : 128;
  const long long planes = (long long)a.c.num_pages * hkv;
  const bool local = a.c.v != nullptr;
  ChunkMaps m;
  bool ok = box_map(&m.q, a.q, d, a.hq, a.total_q, a.group, tpc);
  m.qs = m.q;
  if (L.q_mask) ok &= box_map(&m.qs, p.q_side, L.q_lo ? 2 * p.q_cols : p.q_cols, a.hq, a.total_q, a.group, tpc);
  ok &= box_map(&m.k_copy, p.k_copy, d, p.copy_rows, hkv, keys, 1);
  ok &= box_map(&m.v_copy, p.v_copy, d, p.copy_rows, hkv, 128, 1);
  m.k = m.k_copy;
  m.v = m.v_copy;
  if (!e4m3) {
    ok &= box_map(&m.k, a.c.k, d, ps, planes, std::min(ps, keys), 1);
    ok &= box_map(&m.v, local ? a.c.v : a.c.k, d, ps, planes, std::min(ps, 128), 1);
  }
  m.k_rot = m.k_copy;
  if (L.k_mask) ok &= box_map(&m.k_rot, p.k_rot, p.k_cols, p.rot_rows, hkv, keys, 1);
  if (!ok) return GEMMA_ATTN_ERR_LAUNCH;
  const long long units = (long long)(L.units + L.slots) * L.units_x;
  return launch_chunk(m, a, p, (int)std::min<long long>(units, 1 << 20), L.slots, stream) == cudaSuccess ? GEMMA_ATTN_OK : GEMMA_ATTN_ERR_LAUNCH;
}

}  // namespace
}  // namespace gattn

extern "C" {

int gemma_attn_paged_append(const gemma_attn_params* params, const gemma_attn_paged_cache* cache,
                            const void* new_k, const void* new_v, const int32_t* cu_q,
                            const int32_t* cache_seqlens, int32_t batch, int32_t total_q, void* stream) {
  set_launch_count(0);
  PagedAppendArgs a{};
  bool e4m3;
  const int rc = paged_prepare(params, cache, &a.c, &e4m3);
  if (rc != GEMMA_ATTN_OK) return rc;
  if (batch < 1 || total_q < 0 || !cu_q || !cache_seqlens) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch > 65535) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if (total_q == 0) return GEMMA_ATTN_OK;
  if (!new_k || (new_v != nullptr) != (a.c.v != nullptr)) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (((uintptr_t)new_k | (uintptr_t)new_v) & 15u || !aligned4(cu_q, cache_seqlens)) return GEMMA_ATTN_ERR_MISALIGNED;
  a.new_k = static_cast<const uint16_t*>(new_k);
  a.new_v = static_cast<const uint16_t*>(new_v);
  a.cu_q = cu_q;
  a.lens = cache_seqlens;
  a.batch = batch;
  a.total_q = total_q;
  a.r = params->kind == GEMMA_ATTN_LOCAL ? rotated_pairs(params->rope_p, params->head_dim) : 0;
  if (a.r > 0) {
    const double log2_step = -2.0 / params->head_dim * log2((double)params->rope_base);
    for (int j = 0; j < a.r; j += 8) a.freq8[j / 8] = exp2(j * log2_step) * 0.15915494309189533577;  // 1 / (2 pi)
    a.freq_step = exp2(log2_step);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(e4m3 ? launch_paged_append<true>(a, s) : launch_paged_append<false>(a, s), 1);
}

int gemma_attn_paged_gather(const gemma_attn_params* params, const gemma_attn_paged_cache* cache,
                            const int32_t* starts, const int32_t* cu_out, void* out_k, void* out_v,
                            int32_t batch, int32_t total_out, void* stream) {
  set_launch_count(0);
  PagedGatherArgs a{};
  bool e4m3;
  const int rc = paged_prepare(params, cache, &a.c, &e4m3);
  if (rc != GEMMA_ATTN_OK) return rc;
  if (batch < 1 || total_out < 0 || !starts || !cu_out) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch > 65535) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if (total_out == 0) return GEMMA_ATTN_OK;
  if (!out_k || (out_v != nullptr) != (a.c.v != nullptr)) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (((uintptr_t)out_k | (uintptr_t)out_v) & 15u || !aligned4(starts, cu_out)) return GEMMA_ATTN_ERR_MISALIGNED;
  a.starts = starts;
  a.cu_out = cu_out;
  a.out_k = out_k;
  a.out_v = out_v;
  a.batch = batch;
  a.total_out = total_out;
  const bool f32 = params->out_dtype == GEMMA_ATTN_OUT_F32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (e4m3) e = f32 ? launch_paged_gather<true, true>(a, s) : launch_paged_gather<true, false>(a, s);
  else e = f32 ? launch_paged_gather<false, true>(a, s) : launch_paged_gather<false, false>(a, s);
  return launched(e, 1);
}

int gemma_attn_paged_workspace_size(const gemma_attn_params* params, const gemma_attn_paged_cache* cache,
                                    int32_t batch, int32_t total_q, int32_t max_q, int32_t max_cache_len,
                                    size_t* bytes) {
  PagedCache c;
  bool e4m3;
  int rc = paged_prepare(params, cache, &c, &e4m3);
  if (rc != GEMMA_ATTN_OK) return rc;
  if (!bytes) return GEMMA_ATTN_ERR_INVALID_ARG;
  AttendPlan plan;
  rc = attend_plan(params, e4m3, batch, total_q, max_q, max_cache_len, &plan);
  if (rc != GEMMA_ATTN_OK) return rc;
  *bytes = plan.total;
  return GEMMA_ATTN_OK;
}

int gemma_attn_paged_attend(const gemma_attn_params* params, const gemma_attn_paged_cache* cache,
                            const void* q, const int32_t* cu_q, const int32_t* cache_seqlens, void* out,
                            float* lse, int32_t batch, int32_t total_q, int32_t max_q,
                            int32_t max_cache_len, void* workspace, size_t workspace_bytes, void* stream) {
  set_launch_count(0);
  PagedAttendArgs a{};
  bool e4m3;
  int rc = paged_prepare(params, cache, &a.c, &e4m3);
  if (rc != GEMMA_ATTN_OK) return rc;
  AttendPlan plan;
  rc = attend_plan(params, e4m3, batch, total_q, max_q, max_cache_len, &plan);
  if (rc != GEMMA_ATTN_OK) return rc;
  if (!cu_q || !cache_seqlens) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (total_q == 0 || max_q == 0) return GEMMA_ATTN_OK;
  if (!q || !out) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)out) & 15u || !aligned4(cu_q, cache_seqlens, lse)) return GEMMA_ATTN_ERR_MISALIGNED;
  if (plan.total > 0 && (!workspace || workspace_bytes < plan.total)) return GEMMA_ATTN_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return GEMMA_ATTN_ERR_MISALIGNED;
  a.q = static_cast<const uint16_t*>(q);
  a.cu_q = cu_q;
  a.lens = cache_seqlens;
  a.out = out;
  a.lse = lse;
  a.out_f32 = params->out_dtype == GEMMA_ATTN_OUT_F32;
  a.batch = batch;
  a.total_q = total_q;
  a.max_q = max_q;
  a.max_len = max_cache_len;
  a.hq = params->num_q_heads;
  a.group = params->num_q_heads / params->num_kv_heads;
  a.is_local = params->kind == GEMMA_ATTN_LOCAL;
  a.window = a.is_local ? params->window : 0;
  a.r = rotated_pairs(params->rope_p, params->head_dim);
  a.log2_base = log2((double)params->rope_base);
  a.softmax_scale = params->softmax_scale;
  a.row_groups = plan.shape.row_groups;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.partial_o = reinterpret_cast<float*>(ws + plan.part_o);
  a.partial_lse = reinterpret_cast<float*>(ws + plan.part_lse);
  a.joins = reinterpret_cast<int4*>(ws + plan.joins);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = plan.shape.cut ? 2 : 1;
  if (plan.chunk) {
    if (plan.seqs > 0) {
      a.chunk_of = reinterpret_cast<int*>(ws + plan.chunk_of);
      a.rest = reinterpret_cast<int*>(ws + plan.header) + 2;
      rc = launch_attend_chunks(params, a, e4m3, plan, ws, s);
      if (rc != GEMMA_ATTN_OK) return rc;
      launches += 4;
    }
  }
  return launched(launch_paged_rows(a, plan.shape, e4m3, s), launches);
}

int gemma_attn_draft_verify(const void* target_probs, const void* draft_probs, int32_t prob_dtype,
                            const int32_t* draft_tokens, const int32_t* draft_lens, const float* uniforms,
                            const float* noise, int32_t batch, int32_t max_draft, int32_t vocab,
                            int32_t* num_accepted, int32_t* out_tokens, void* stream) {
  set_launch_count(0);
  if (prob_dtype != GEMMA_ATTN_PROBS_F32 && prob_dtype != GEMMA_ATTN_PROBS_BF16) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch < 0 || max_draft < 0 || vocab < 1) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch > (0x7fffffff / 8) || max_draft > (1 << 20) || vocab > (1 << 30)) return GEMMA_ATTN_ERR_UNSUPPORTED;
  if (batch == 0) return GEMMA_ATTN_OK;
  if (!target_probs || !noise || !num_accepted || !out_tokens) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (max_draft > 0 && (!draft_tokens || !uniforms)) return GEMMA_ATTN_ERR_INVALID_ARG;
  const uintptr_t probs = (uintptr_t)target_probs | (uintptr_t)draft_probs;
  if (probs & (prob_dtype == GEMMA_ATTN_PROBS_F32 ? 3u : 1u)) return GEMMA_ATTN_ERR_MISALIGNED;
  if (((uintptr_t)draft_tokens | (uintptr_t)draft_lens | (uintptr_t)uniforms | (uintptr_t)noise |
       (uintptr_t)num_accepted | (uintptr_t)out_tokens) & 3u)
    return GEMMA_ATTN_ERR_MISALIGNED;
  DraftArgs a{};
  a.target = target_probs;
  a.draft = draft_probs;
  a.tokens = draft_tokens;
  a.lens = draft_lens;
  a.uniforms = uniforms;
  a.noise = noise;
  a.accepted = num_accepted;
  a.out = out_tokens;
  a.batch = batch;
  a.max_draft = max_draft;
  a.vocab = vocab;
  return launched(launch_draft_verify(a, prob_dtype == GEMMA_ATTN_PROBS_BF16, static_cast<cudaStream_t>(stream)), 1);
}

}  // extern "C"
