// draft.cu -- verification of drafted tokens from given random numbers.
//
// Drafted token i, x, is accepted iff u_i q_i(x) < p_i(x); at the first rejection the next token
// is the winner of the exponential race argmax_v w(v) / e(v) over w = max(p_i - q_i, 0), which
// draws v with probability w(v) / sum(w) when e holds unit-exponential draws; after n accepted
// drafts w = p_n. Product, difference and quotient are one correctly rounded fp32 operation
// each (no contraction, no approximate division), and a maximum has no order, so the
// outcome depends on nothing but the inputs.
//
// The race reads three rows of `vocab` once (p, q, noise): bound by HBM for a batch, by latency
// for one sequence. One cluster of 8 CTAs owns a sequence, so that a single sequence still
// draws on eight SMs' loads and the CTAs' winners meet through distributed shared memory: one
// launch, no workspace, nothing to reset. Every CTA settles the acceptance for itself (a warp
// reads the few drafted tokens' probabilities).
// A candidate is one 64-bit key, the quotient's bits above the complement of its index: quotients
// are not negative, so the keys order like (quotient, lowest index first), and 0 means none.
#include "paged.h"

namespace gattn {

namespace {

constexpr int kDraftThreads = 512;
constexpr int kDraftCluster = 8;

__device__ __forceinline__ float prob_at(const void* p, size_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16)
              : __ldg(static_cast<const float*>(p) + i);
}

__device__ __forceinline__ unsigned long long race_key(float w, float e, int v) {
  if (!(w > 0.f) || !(e > 0.f)) return 0ull;
  const float x = __fdiv_rn(w, e);
  if (!(x >= 0.f)) return 0ull;  // inf / inf
  return ((unsigned long long)__float_as_uint(x) << 32) | (uint32_t)~(uint32_t)v;
}

__device__ __forceinline__ unsigned long long shfl_max(unsigned long long k) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, m);
    if (o > k) k = o;
  }
  return k;
}

}  // namespace

template <bool BF16>
__global__ void __launch_bounds__(kDraftThreads) draft_verify_kernel(DraftArgs a) {
  __shared__ int s_stop;
  __shared__ unsigned long long s_warp[2][kDraftThreads / 32];
  __shared__ unsigned long long s_best[2];  // this CTA's winners: residual, and p alone
  const int rank = (int)cluster_ctarank();
  const int b = blockIdx.x / kDraftCluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t V = (size_t)a.vocab;
  int n = a.lens ? __ldg(a.lens + b) : a.max_draft;
  if (n < 0 || n > a.max_draft) {
    if (rank == 0 && tid == 0) atomicOr(&g_status, kStatusSeqlen);
    n = n < 0 ? 0 : a.max_draft;
  }
  const int32_t* tokens = a.tokens + (size_t)b * a.max_draft;
  const size_t prow = (size_t)b * (a.max_draft + 1), qrow = (size_t)b * a.max_draft;
  if (warp == 0) {
    int stop = n;
    for (int i0 = 0; i0 < n && stop == n; i0 += 32) {
      const int i = i0 + lane;
      bool good = true;
      if (i < n) {
        const int x = __ldg(tokens + i);
        good = x >= 0 && x < a.vocab;
        if (good) {
          const float p = prob_at(a.target, (prow + i) * V + x, BF16);
          const float q = a.draft ? prob_at(a.draft, (qrow + i) * V + x, BF16) : 1.f;
          good = __fmul_rn(__ldg(a.uniforms + (size_t)b * a.max_draft + i), q) < p;
        }
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, !good);
      if (bad) stop = i0 + __ffs(bad) - 1;
    }
    if (lane == 0) s_stop = stop;
  }
  __syncthreads();
  const int stop = s_stop;
  const bool rejected = stop < n;
  const bool dense = rejected && a.draft != nullptr;
  const int certain = rejected && a.draft == nullptr ? __ldg(tokens + stop) : -1;  // left out of the residual
  const void* pt = BF16 ? (const void*)(static_cast<const uint16_t*>(a.target) + (prow + stop) * V)
                        : (const void*)(static_cast<const float*>(a.target) + (prow + stop) * V);
  const void* qt = !dense ? nullptr
                   : BF16 ? (const void*)(static_cast<const uint16_t*>(a.draft) + (qrow + stop) * V)
                          : (const void*)(static_cast<const float*>(a.draft) + (qrow + stop) * V);
  const float* nz = a.noise + (size_t)b * V;

  unsigned long long best[2] = {0ull, 0ull};
  auto take = [&](float p, float q, float e, int v) {
    const float w = v == certain ? 0.f : dense ? __fsub_rn(p, q) : p;
    const unsigned long long k = race_key(w, e, v);
    if (k > best[0]) best[0] = k;
    if (rejected) {
      const unsigned long long kp = race_key(p, e, v);
      if (kp > best[1]) best[1] = kp;
    }
  };
  // 16-byte loads where the three rows allow them (the vocabulary need not be a multiple of 4)
  const bool vec = ((reinterpret_cast<uintptr_t>(pt) | reinterpret_cast<uintptr_t>(qt)) & (BF16 ? 7u : 15u)) == 0 &&
                   (reinterpret_cast<uintptr_t>(nz) & 15u) == 0;
  const int quads = vec ? a.vocab / 4 : 0;
  auto quad = [&](const void* base, int i) -> float4 {
    if constexpr (BF16) {
      const uint2 w = __ldg(static_cast<const uint2*>(base) + i);
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xFFFF0000u));
    } else {
      return __ldg(static_cast<const float4*>(base) + i);
    }
  };
  const int step = kDraftCluster * kDraftThreads;
#pragma unroll 4
  for (int i = rank * kDraftThreads + tid; i < quads; i += step) {
    const float4 p = quad(pt, i), e = __ldg(reinterpret_cast<const float4*>(nz) + i);
    const float4 q = dense ? quad(qt, i) : make_float4(0.f, 0.f, 0.f, 0.f);
    take(p.x, q.x, e.x, 4 * i);
    take(p.y, q.y, e.y, 4 * i + 1);
    take(p.z, q.z, e.z, 4 * i + 2);
    take(p.w, q.w, e.w, 4 * i + 3);
  }
  for (int v = 4 * quads + rank * kDraftThreads + tid; v < a.vocab; v += step)
    take(prob_at(pt, v, BF16), dense ? prob_at(qt, v, BF16) : 0.f, __ldg(nz + v), v);

#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const unsigned long long w = shfl_max(best[k]);
    if (lane == 0) s_warp[k][warp] = w;
  }
  __syncthreads();
  if (warp < 2) {
    const unsigned long long w = shfl_max(lane < kDraftThreads / 32 ? s_warp[warp][lane] : 0ull);
    if (lane == 0) s_best[warp] = w;
  }
  __syncthreads();
  __syncwarp();
  cluster_sync_all();  // every CTA's winners are in its shared memory
  if (rank == 0 && warp == 0) {
    unsigned long long k[2] = {0ull, 0ull};
    if (lane < kDraftCluster) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t addr;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(&s_best[j])), "r"(lane));
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k[j]) : "r"(addr) : "memory");
      }
    }
    k[0] = shfl_max(k[0]);
    k[1] = shfl_max(k[1]);
    const unsigned long long w = k[0] != 0ull ? k[0] : k[1];
    const int next = w != 0ull ? (int)~(uint32_t)w : -1;
    int32_t* out = a.out + (size_t)b * (a.max_draft + 1);
    for (int i = lane; i <= a.max_draft; i += 32) out[i] = i < stop ? __ldg(tokens + i) : i == stop ? next : -1;
    if (lane == 0) a.accepted[b] = stop;
  }
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while its winners may still be read
}

cudaError_t launch_draft_verify(const DraftArgs& a, bool bf16, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * kDraftCluster);
  cfg.blockDim = dim3(kDraftThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kDraftCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<true>, a)
              : cudaLaunchKernelEx(&cfg, draft_verify_kernel<false>, a);
}

}  // namespace gattn
