// kda_verify.cu -- verification of drafted tokens from given random numbers:
// kda_verify_drafts of kda_serving.h.
//
// Drafts are accepted in order while u q(x) < p(x); the next token is then
// the largest r / e with r = max(p - q, 0) after a refusal and r = p when
// every draft was accepted, e the given exponential noise. Every quantity
// that is compared is one fp32 operation of the inputs, so the result does
// not depend on how the vocabulary is split over threads.
//
// Bound: HBM for a batch (one row of p and e, and of q after a refusal: 8 to
// 12 bytes per vocabulary entry; the other rows are never read), latency for
// one sequence. 256 sequences of up to 5 drafts over 131072 entries take 53 us,
// 89% of the measured copy rate; one sequence takes 5. A cluster of CTAs shares
// a sequence: each finds the accepted count itself (a few gathered
// probabilities), scans its part of the row, and reads the others' best through
// distributed shared memory. So one launch does it, without scratch memory or
// counters.
#include <math.h>

#include <cooperative_groups.h>

#include "kda_internal.cuh"
#include "kda_serving.h"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kSms = 152;

struct VerifyArgs {
  const float *target, *draft, *u, *noise;
  const int32_t *x, *num;
  int32_t *tokens, *accepted;
  int* status;
  int N, T, V;
};

struct Best {
  float score;  // -1: none
  int idx;
};
__device__ __forceinline__ void take(Best& a, float score, int idx) {
  if (score > a.score || (score == a.score && idx < a.idx)) {
    a.score = score;
    a.idx = idx;
  }
}

// Largest r / e of this CTA's part of the row. Q: subtract the draft row;
// skip: the entry to leave out (a draft without a distribution), or -1.
//
// Divisions are few: an entry can only win if r >= thr e, with thr just below
// the warp's best quotient so far (by 2^-20: the rounding of the product and
// of the quotients is far smaller), so a batch without such an entry costs one
// subtraction, one product and one comparison an entry. A warp meets new
// bests about ln(entries) times.
template <bool Q, int VEC>
__device__ Best scan(const float* p, const float* q, const float* e, int V, int skip, int rank, int ranks) {
  Best best{-1.f, INT32_MAX};
  float thr = -1.f;
  constexpr int kUnroll = VEC == 4 ? 2 : 8;  // loads of a row in flight a thread: more would cost threads
  const int units = V / VEC, step = ranks * kThreads;
  const int turns = (units + step * kUnroll - 1) / (step * kUnroll);  // the same for every lane
  int i = rank * kThreads + static_cast<int>(threadIdx.x);
  for (int t = 0; t < turns; ++t, i += kUnroll * step) {
    float pv[kUnroll][VEC], qv[kUnroll][VEC], ev[kUnroll][VEC];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int at = i + j * step;
      if (at < units) {
        if constexpr (VEC == 4) {
          *reinterpret_cast<float4*>(pv[j]) = __ldcs(reinterpret_cast<const float4*>(p) + at);
          if (Q) *reinterpret_cast<float4*>(qv[j]) = __ldcs(reinterpret_cast<const float4*>(q) + at);
          *reinterpret_cast<float4*>(ev[j]) = __ldcs(reinterpret_cast<const float4*>(e) + at);
        } else {
          pv[j][0] = __ldcs(p + at);
          if (Q) qv[j][0] = __ldcs(q + at);
          ev[j][0] = __ldcs(e + at);
        }
      } else {
#pragma unroll
        for (int c = 0; c < VEC; ++c) pv[j][c] = qv[j][c] = 0.f, ev[j][c] = 1.f;
      }
    }
    bool any = false;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        if (Q) pv[j][c] -= qv[j][c];  // r from here on
        any |= pv[j][c] > 0.f && pv[j][c] >= thr * ev[j][c];
      }
    if (__any_sync(~0u, any)) {
      if (any) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            const float r = pv[j][c];
            const int idx = (i + j * step) * VEC + c;
            if (r > 0.f && r >= thr * ev[j][c] && idx != skip) take(best, r / ev[j][c], idx);
          }
      }
      // quotients are never negative, so their order is that of their bits; -1: none yet
      const uint32_t top = __reduce_max_sync(~0u, best.score < 0.f ? 0u : __float_as_uint(best.score));
      const bool some = __any_sync(~0u, best.score >= 0.f);
      thr = some ? __uint_as_float(top) * (1.f - 0x1p-20f) : -1.f;
    }
  }
  return best;
}

// Best over the cluster, the same on every thread of it.
__device__ Best over_cluster(Best b, Best* warps, Best* mine) {
  auto cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) take(b, __shfl_xor_sync(~0u, b.score, m), __shfl_xor_sync(~0u, b.idx, m));
  if (lane == 0) warps[warp] = b;
  __syncthreads();
  if (warp == 0) {
    b = lane < kThreads / 32 ? warps[lane] : Best{-1.f, INT32_MAX};
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) take(b, __shfl_xor_sync(~0u, b.score, m), __shfl_xor_sync(~0u, b.idx, m));
    if (lane == 0) *mine = b;
  }
  cluster.sync();
  b = Best{-1.f, INT32_MAX};
  for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
    const Best o = *cluster.map_shared_rank(mine, r);
    take(b, o.score, o.idx);
  }
  cluster.sync();  // every CTA has read *mine
  return b;
}

template <int VEC>
__global__ void __launch_bounds__(kThreads, 2) kda_verify_kernel(const VerifyArgs a) {
  auto cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int n = static_cast<int>(blockIdx.x) / ranks;
  __shared__ Best s_warps[kThreads / 32], s_best;
  __shared__ int s_taken;
  const int64_t V = a.V;
  int num = a.num ? a.num[n] : a.T;
  num = num < 0 ? 0 : (num > a.T ? a.T : num);
  const float* const target = a.target + static_cast<int64_t>(n) * (a.T + 1) * V;
  const int32_t* const x = a.x + static_cast<int64_t>(n) * a.T;
  if (threadIdx.x < 32) {
    int taken = num;
    for (int i0 = 0; i0 < num; i0 += 32) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      bool ok = true;
      if (i < num) {
        const int xi = x[i];
        ok = xi >= 0 && xi < a.V;
        if (!ok && rank == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
        if (ok) {
          const float p = target[i * V + xi];
          const float q = a.draft ? a.draft[(static_cast<int64_t>(n) * a.T + i) * V + xi] : 1.f;
          ok = a.u[static_cast<int64_t>(n) * a.T + i] * q < p;
        }
      }
      const unsigned refused = __ballot_sync(~0u, !ok);
      if (refused) {
        taken = i0 + __ffs(refused) - 1;
        break;
      }
    }
    if (threadIdx.x == 0) s_taken = taken;
  }
  __syncthreads();
  const int taken = s_taken;
  const float* const p = target + taken * V;
  const float* const e = a.noise + static_cast<int64_t>(n) * V;
  Best best{-1.f, INT32_MAX};
  if (taken < num) {
    if (a.draft)
      best = scan<true, VEC>(p, a.draft + (static_cast<int64_t>(n) * a.T + taken) * V, e, a.V, -1, rank, ranks);
    else
      best = scan<false, VEC>(p, nullptr, e, a.V, x[taken], rank, ranks);
    best = over_cluster(best, s_warps, &s_best);
  }
  if (best.score < 0.f) {  // every draft accepted, or nothing left of the target after the draft
    best = scan<false, VEC>(p, nullptr, e, a.V, -1, rank, ranks);
    best = over_cluster(best, s_warps, &s_best);
  }
  if (rank == 0) {
    const int next = best.score < 0.f ? 0 : best.idx;
    for (int i = static_cast<int>(threadIdx.x); i <= a.T; i += kThreads)
      a.tokens[static_cast<int64_t>(n) * (a.T + 1) + i] = i < taken ? x[i] : (i == taken ? next : -1);
    if (threadIdx.x == 0) a.accepted[n] = taken;
  }
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_verify_drafts(int32_t num_seqs, int32_t max_drafts, int32_t vocab, const float* target,
                                        const float* draft, const int32_t* draft_tokens, const int32_t* num_drafts,
                                        const float* u, const float* noise, int32_t* tokens, int32_t* accepted,
                                        int32_t* status, void* stream) {
  using namespace kda;
  if (num_seqs < 1 || num_seqs > (1 << 27)) return set_error(KDA_ERR_INVALID_ARG, "num_seqs %d out of range", num_seqs);
  if (max_drafts < 0 || max_drafts > (1 << 20))
    return set_error(KDA_ERR_INVALID_ARG, "max_drafts %d out of range", max_drafts);
  if (vocab < 1 || vocab > (1 << 30)) return set_error(KDA_ERR_INVALID_ARG, "vocab %d out of range", vocab);
  const struct { const char* name; const void* p; bool wanted; } ptrs[] = {
      {"target", target, true}, {"draft", draft, false}, {"draft_tokens", draft_tokens, max_drafts > 0},
      {"num_drafts", num_drafts, false}, {"u", u, max_drafts > 0}, {"noise", noise, true},
      {"tokens", tokens, true}, {"accepted", accepted, true}, {"status", status, false}};
  for (const auto& t : ptrs) {
    if (t.wanted && !t.p) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", t.name);
    if ((uintptr_t)t.p & 3u) return set_error(KDA_ERR_INVALID_ARG, "%s is not 4-byte aligned", t.name);
  }
  VerifyArgs a{target, draft, u, noise, draft_tokens, num_drafts, tokens, accepted, status, num_seqs, max_drafts, vocab};
  const bool vec = vocab % 4 == 0 && (((uintptr_t)target | (uintptr_t)draft | (uintptr_t)noise) & 15u) == 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  // CTAs of a sequence: at most 8, and no more than give every SM one over the
  // call (256 x 131072: 54 us with 1, 57 with 2, 64 with 4 CTAs a sequence; a
  // cluster's CTAs have to find room together).
  unsigned ranks = 8;
  while (ranks > 1 && (int64_t)num_seqs * ranks / 2 >= kSms) ranks /= 2;
  attr.val.clusterDim.x = ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)num_seqs * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      vec ? cudaLaunchKernelEx(&cfg, kda_verify_kernel<4>, a) : cudaLaunchKernelEx(&cfg, kda_verify_kernel<1>, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return set_error(KDA_ERR_CUDA, "verify launch failed: %s", cudaGetErrorString(e));
  }
  return KDA_OK;
}
