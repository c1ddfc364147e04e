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

int launched(cudaError_t e, int launches) {
  if (e != cudaSuccess) return GEMMA_ATTN_ERR_LAUNCH;
  set_launch_count(launches);
  return GEMMA_ATTN_OK;
}

// Shape of an attend call: how the rows and keys are cut, and the workspace that takes.
struct AttendPlan {
  int row_groups, splits;
  size_t lse_off, total;
};

int attend_plan(const gemma_attn_params* p, int batch, int total_q, int max_q, int max_cache_len, AttendPlan* plan) {
  if (batch < 1 || total_q < 0 || max_q < 0 || max_cache_len < 0) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch > 65535 || (long long)max_cache_len + max_q > 0x7fffff00ll) return GEMMA_ATTN_ERR_UNSUPPORTED;
  const long long rows = (long long)total_q * p->num_q_heads;
  if (rows > 0x7fffffffll) return GEMMA_ATTN_ERR_UNSUPPORTED;
  const int group = p->num_q_heads / p->num_kv_heads;
  plan->row_groups = (int)(((long long)max_q * group + 7) / 8);
  const long long keys = p->kind == GEMMA_ATTN_LOCAL ? std::min<long long>(max_cache_len, p->window) + max_q
                                                     : (long long)max_cache_len + max_q;
  plan->splits = paged_rows_splits(batch, p->num_kv_heads, std::max(1, plan->row_groups), (int)keys);
  const size_t o = plan->splits > 1 ? round_up((size_t)plan->splits * rows * p->head_dim * 4, 256) : 0;
  const size_t l = plan->splits > 1 ? round_up((size_t)plan->splits * rows * 4, 256) : 0;
  plan->lse_off = o;
  plan->total = o + l;
  return GEMMA_ATTN_OK;
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
  if (((uintptr_t)new_k | (uintptr_t)new_v) & 15u) return GEMMA_ATTN_ERR_MISALIGNED;
  a.new_k = static_cast<const uint16_t*>(new_k);
  a.new_v = static_cast<const uint16_t*>(new_v);
  a.cu_q = cu_q;
  a.lens = cache_seqlens;
  a.batch = batch;
  a.total_q = total_q;
  a.r = params->kind == GEMMA_ATTN_LOCAL ? rotated_pairs(params->rope_p, params->head_dim) : 0;
  a.log2_base = log2((double)params->rope_base);
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
  if (((uintptr_t)out_k | (uintptr_t)out_v) & 15u) return GEMMA_ATTN_ERR_MISALIGNED;
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
  rc = attend_plan(params, batch, total_q, max_q, max_cache_len, &plan);
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
  rc = attend_plan(params, batch, total_q, max_q, max_cache_len, &plan);
  if (rc != GEMMA_ATTN_OK) return rc;
  if (!cu_q || !cache_seqlens) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (total_q == 0 || max_q == 0) return GEMMA_ATTN_OK;
  if (!q || !out) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)out) & 15u) return GEMMA_ATTN_ERR_MISALIGNED;
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
  a.row_groups = plan.row_groups;
  a.splits = plan.splits;
  a.partial_o = static_cast<float*>(workspace);
  a.partial_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.lse_off);
  return launched(launch_paged_rows(a, e4m3, static_cast<cudaStream_t>(stream)), plan.splits > 1 ? 2 : 1);
}

int gemma_attn_draft_verify(const void* target_probs, const void* draft_probs, int32_t prob_dtype,
                            const int32_t* draft_tokens, const int32_t* draft_lens, const float* uniforms,
                            const float* noise, int32_t batch, int32_t max_draft, int32_t vocab,
                            int32_t* num_accepted, int32_t* out_tokens, void* stream) {
  set_launch_count(0);
  if (prob_dtype != GEMMA_ATTN_PROBS_F32 && prob_dtype != GEMMA_ATTN_PROBS_BF16) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch < 0 || max_draft < 0 || vocab < 1) return GEMMA_ATTN_ERR_INVALID_ARG;
  if (batch > (0x7fffffff / 8) || max_draft > (1 << 20)) return GEMMA_ATTN_ERR_UNSUPPORTED;
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
