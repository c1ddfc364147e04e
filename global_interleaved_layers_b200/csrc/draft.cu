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
// Few candidates are divided: with x the largest quotient that the warp has seen, one whose
// w < fl(x e) (1 - 2^-21) has a quotient that rounds below x (passes()). Dividing them all, for both
// races at once, took 59 us for 64 sequences of 262,144 words in bf16; HBM would allow 20.
// The race over p alone, which only counts where no residual is left, is a second pass. Measured:
// those 64 sequences 37 us (HBM: 20), one of 262,144 words in fp32 12 us (launch, acceptance and
// three latencies; the bytes would take half a microsecond).
#include "paged.h"

namespace gattn {

namespace {

constexpr int kDraftThreads = 512;
constexpr int kDraftCluster = 8;

__device__ __forceinline__ float prob_at(const void* p, size_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16)
              : __ldg(static_cast<const float*>(p) + i);
}

__device__ __noinline__ unsigned long long race_key(float w, float e, int v) {
  if (!(w > 0.f) || !(e > 0.f)) return 0ull;
  const float x = __fdiv_rn(w, e);
  if (!(x >= 0.f)) return 0ull;  // inf / inf
  return ((unsigned long long)__float_as_uint(x) << 32) | (uint32_t)~(uint32_t)v;
}

// May w / e, rounded, be x or more? The product's rounding is 2^-24 of it while it is normal, the
// quotient's 2^-24, the bound's product 2^-24: together far under 2^-21. A product near the
// ends of fp32's range proves nothing, nor does an x whose neighbours are not 2^-23 of it away.
__device__ __forceinline__ bool passes(float w, float e, float x) {
  const float y = __fmul_rn(x, e);
  return w > 0.f && !(w < __fmul_rn(y, 1.f - 0x1p-21f) && y >= 0x1p-100f && y < INFINITY && x >= 0x1p-100f);
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
__global__ void __launch_bounds__(kDraftThreads, 2) draft_verify_kernel(DraftArgs a) {
  __shared__ int s_stop;
  __shared__ unsigned long long s_warp[kDraftThreads / 32];
  __shared__ unsigned long long s_best[2];  // this CTA's winner of either pass
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
  // The noise is read whatever the acceptance says: this CTA's eighth of it is on its way meanwhile.
  if (warp == 1 && lane == 0) {
    const size_t part = (V * 4 / kDraftCluster) & ~size_t(15);
    const char* at = reinterpret_cast<const char*>(a.noise + (size_t)b * V) + rank * part;
    at += -reinterpret_cast<uintptr_t>(at) & 15;
    if (part > 16)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"((uint32_t)(part - 16)) : "memory");
  }
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

  // 16-byte loads where the three rows allow them (the vocabulary need not be a multiple of 4)
  const bool vec = ((reinterpret_cast<uintptr_t>(pt) | reinterpret_cast<uintptr_t>(qt)) & (BF16 ? 7u : 15u)) == 0 &&
                   (reinterpret_cast<uintptr_t>(nz) & 15u) == 0;
  const int quads = vec ? a.vocab / 4 : 0;
  using Raw = typename std::conditional<BF16, uint2, float4>::type;  // four probabilities as they lie
  auto quad = [&](const Raw& w) -> float4 {
    if constexpr (BF16)
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xFFFF0000u));
    else
      return w;
  };
  const int step = kDraftCluster * kDraftThreads;
  unsigned long long win = 0ull;
  // pass 0: the residual (or p, where nothing was rejected); pass 1, if that leaves no candidate: p
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const bool sub = dense && pass == 0;
    const int out = pass == 0 ? certain : -1;
    unsigned long long best = 0ull;
    float x = 0.f;  // the largest quotient of this warp's lanes, up to a group ago
    auto take = [&](float p, float q, float e, int v) {
      const float w = v == out ? 0.f : sub ? __fsub_rn(p, q) : p;
      if (passes(w, e, x)) {
        const unsigned long long k = race_key(w, e, v);
        if (k > best) best = k;
      }
    };
    // Groups of loads in flight together; between them the warp agrees on its best quotient.
    constexpr int U = 4;
#pragma unroll 1
    for (int i0 = rank * kDraftThreads + warp * 32; i0 < quads; i0 += U * step) {
      Raw p[U], q[U];
      float4 e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * step + lane;
        const bool get = i < quads;
        p[u] = get ? __ldg(static_cast<const Raw*>(pt) + i) : Raw{};
        e[u] = get ? __ldg(reinterpret_cast<const float4*>(nz) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        q[u] = get && sub ? __ldg(static_cast<const Raw*>(qt) + i) : Raw{};
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = 4 * (i0 + u * step + lane);
        const float4 pf = quad(p[u]), qf = quad(q[u]);
        take(pf.x, qf.x, e[u].x, v);
        take(pf.y, qf.y, e[u].y, v + 1);
        take(pf.z, qf.z, e[u].z, v + 2);
        take(pf.w, qf.w, e[u].w, v + 3);
        // (quotients are not negative: their bits order like unsigned integers)
        x = __uint_as_float(__reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32)));
      }
    }
    // The rest: the last few words, or all where a row of an odd vocabulary is not aligned.
    constexpr int W = 8;
#pragma unroll 1
    for (int v0 = 4 * quads + rank * kDraftThreads + warp * 32; v0 < a.vocab; v0 += W * step) {
      float p[W], q[W], e[W];
#pragma unroll
      for (int u = 0; u < W; ++u) {
        const int v = v0 + u * step + lane;
        const bool get = v < a.vocab && v >= 0;
        p[u] = get ? prob_at(pt, v, BF16) : 0.f;
        e[u] = get ? __ldg(nz + v) : 0.f;
        q[u] = get && sub ? prob_at(qt, v, BF16) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < W; ++u) take(p[u], q[u], e[u], v0 + u * step + lane);
      x = __uint_as_float(__reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32)));
    }

    best = shfl_max(best);
    if (lane == 0) s_warp[warp] = best;
    __syncthreads();
    if (warp == 0) {
      best = shfl_max(lane < kDraftThreads / 32 ? s_warp[lane] : 0ull);
      if (lane == 0) s_best[pass] = best;
    }
    __syncthreads();
    __syncwarp();
    cluster_sync_all();  // every CTA's winner is in its shared memory
    win = 0ull;
    if (lane < kDraftCluster) {
      uint32_t addr;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(&s_best[pass])), "r"(lane));
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(win) : "r"(addr) : "memory");
    }
    win = shfl_max(win);
    if (win != 0ull || !rejected) break;  // the same in every CTA of the cluster
  }
  if (rank == 0 && warp == 0) {
    const int next = win != 0ull ? (int)~(uint32_t)win : -1;
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
