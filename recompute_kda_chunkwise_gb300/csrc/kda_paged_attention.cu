// kda_paged_attention.cu -- attention of new tokens over a paged cache.
//
// One warp per (token, query head) walks the token's keys with the running
// maximum and sum of a softmax: lanes hold D / 32 channels each.
#include "kda_paged.cuh"

namespace kda {
namespace {

template <int D>
__global__ void __launch_bounds__(128) kda_paged_attention_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (job >= a.S * a.Hq) return;
  const int64_t tok = job / a.Hq;
  const int h = static_cast<int>(job % a.Hq), hk = h / (a.Hq / a.Hkv);
  int n = 0, bad = a.cu[0] != 0 || a.cu[a.N] != a.S;
  for (int i = lane; i < a.N; i += 32) {
    n += a.cu[i + 1] <= tok;
    bad |= a.cu[i + 1] < a.cu[i];
  }
  n = __reduce_add_sync(~0u, n);
  bad = __reduce_or_sync(~0u, bad);
  __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(a.o) + job * D + lane * E;
  bool ok = !bad && n < a.N;
  int64_t keys = 0;
  if (ok) {
    keys = static_cast<int64_t>(a.lens[n]) - (a.cu[n + 1] - tok) + 1;
    ok = a.lens[n] >= 0 && a.lens[n] <= static_cast<int64_t>(a.width) * a.page;
  }
  if (!ok && lane == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) {
    q[i] = ldf(static_cast<const __nv_bfloat16*>(a.q) + job * D + lane * E + i) * a.scale;
    acc[i] = 0.f;
  }
  for (int64_t t = 0; ok && t < keys; ++t) {
    const int64_t page = a.table[static_cast<int64_t>(n) * a.width + t / a.page];
    if (page < 0 || page >= a.pages) {
      if (lane == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
      l = 0.f;
      break;
    }
    const int64_t at = ((page * a.page + t % a.page) * a.Hkv + hk) * D + lane * E;
    float s = 0.f;
    for (int i = 0; i < E; ++i) s += q[i] * ldf(static_cast<const __nv_bfloat16*>(a.k) + at + i);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = mn == m ? 1.f : expf(m - mn), p = s == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * f + p;
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + p * ldf(static_cast<const __nv_bfloat16*>(a.v) + at + i);
  }
  for (int i = 0; i < E; ++i) stf(o + i, l == 0.f ? 0.f : acc[i] / l);
}

}  // namespace

size_t paged_attention_scratch_bytes(const PagedArgs&) { return 0; }

kda_status launch_paged_attention(const PagedArgs& a, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int), s);
  const unsigned grid = static_cast<unsigned>((a.S * a.Hq + 3) / 4);
  if (e == cudaSuccess) {
    if (a.D == 128)
      kda_paged_attention_kernel<128><<<grid, 128, 0, s>>>(a);
    else
      kda_paged_attention_kernel<64><<<grid, 128, 0, s>>>(a);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

}  // namespace kda
