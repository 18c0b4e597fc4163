// kda_paged.cu -- the paged cache: appending new tokens, and the host side of
// attention over it (kda_paged_append / kda_paged_attention of kda_serving.h).
#include <math.h>

#include "kda_internal.cuh"
#include "kda_paged.cuh"
#include "kda_serving.h"

namespace kda {
namespace {

// One CTA copies one token's keys and values. The token's sequence is the
// number of sequences that end at or before it: one pass of loads over
// cu_seqlens instead of a chain of dependent ones.
// Bound: launch latency in decoding, HBM for long chunks (8 Hkv D bytes a
// token, read and written).
__global__ void __launch_bounds__(128) kda_paged_append_kernel(const PagedArgs a, const uint4* k, const uint4* v,
                                                               uint4* kp, uint4* vp, int* status) {
  const int64_t tok = blockIdx.x;
  int before = 0;
  for (int i = static_cast<int>(threadIdx.x); i < a.N; i += 128) before += a.cu[i + 1] <= tok;
  __shared__ int s[4];
  before = __reduce_add_sync(~0u, before);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = before;
  __syncthreads();
  const int n = s[0] + s[1] + s[2] + s[3];
  bool ok = n < a.N;
  int64_t at = -1;
  if (ok) {
    const int64_t pos = static_cast<int64_t>(a.lens[n]) - (a.cu[n + 1] - tok);
    // where cu_seqlens decreases, sequence n need not hold the token
    ok = tok >= a.cu[n] && tok < a.cu[n + 1] && pos >= 0 && pos / a.page < a.width;
    if (ok) {
      const int64_t page = a.table[static_cast<int64_t>(n) * a.width + pos / a.page];
      ok = page >= 0 && page < a.pages;
      at = page * a.page + pos % a.page;
    }
  }
  if (!ok) {
    if (threadIdx.x == 0) set_status(status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  const int64_t vecs = static_cast<int64_t>(a.Hkv) * a.D / 8;
  for (int64_t i = threadIdx.x; i < vecs; i += 128) {
    kp[at * vecs + i] = k[tok * vecs + i];
    vp[at * vecs + i] = v[tok * vecs + i];
  }
}

kda_status validate_paged(const kda_paged_problem* p, bool ptrs) {
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != KDA_DTYPE_BF16) return set_error(KDA_ERR_UNSUPPORTED, "dtype %d is not supported (bf16)", p->dtype);
  if (p->head_dim != 64 && p->head_dim != 128)
    return set_error(KDA_ERR_UNSUPPORTED, "head_dim %d is not supported (64 or 128)", p->head_dim);
  if (p->num_seqs < 1 || p->num_seqs > kPagedMaxSeqs)
    return set_error(KDA_ERR_INVALID_ARG, "num_seqs %d out of range (1 to %d)", p->num_seqs, kPagedMaxSeqs);
  if (p->num_kv_heads < 1 || p->num_heads < 1 || p->num_heads > 4096 || p->num_heads % p->num_kv_heads != 0)
    return set_error(KDA_ERR_INVALID_ARG, "num_heads %d must be a multiple of num_kv_heads %d (at most 4096)",
                     p->num_heads, p->num_kv_heads);
  if (p->page_size < 8 || p->page_size % 8 != 0 || p->page_size > (1 << 20))
    return set_error(KDA_ERR_UNSUPPORTED, "page_size %d is not supported (a multiple of 8)", p->page_size);
  if (p->max_pages < 1 || (int64_t)p->max_pages * p->page_size > ((int64_t)1 << 30))
    return set_error(KDA_ERR_INVALID_ARG, "max_pages %d out of range", p->max_pages);
  if (p->num_pages < 1 || p->num_pages > INT32_MAX)
    return set_error(KDA_ERR_INVALID_ARG, "num_pages %lld out of range", (long long)p->num_pages);
  if (p->total_tokens < 0 || p->total_tokens > ((int64_t)1 << 30) / (p->num_heads / p->num_kv_heads))
    return set_error(KDA_ERR_INVALID_ARG, "total_tokens %lld out of range", (long long)p->total_tokens);
  if (!isfinite(p->scale)) return set_error(KDA_ERR_INVALID_ARG, "scale must be finite");
  if (!ptrs) return KDA_OK;
  const struct { const char* name; const void* q; } dev[] = {
      {"cu_seqlens", p->cu_seqlens}, {"page_table", p->page_table}, {"kv_lens", p->kv_lens}};
  for (const auto& t : dev) {
    if (!t.q) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", t.name);
    if ((uintptr_t)t.q & 3u) return set_error(KDA_ERR_INVALID_ARG, "%s is not 4-byte aligned", t.name);
  }
  return KDA_OK;
}

kda_status tensor(const char* name, const void* p) {
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p & 15u) return set_error(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return KDA_OK;
}

PagedArgs args_of(const kda_paged_problem* p) {
  PagedArgs a{};
  a.cu = p->cu_seqlens; a.table = p->page_table; a.lens = p->kv_lens;
  a.S = p->total_tokens; a.pages = p->num_pages;
  a.N = p->num_seqs; a.Hq = p->num_heads; a.Hkv = p->num_kv_heads; a.D = p->head_dim;
  a.page = p->page_size; a.width = p->max_pages; a.scale = p->scale;
  return a;
}

#define PAGED_TRY(x)               \
  do {                             \
    const kda_status st_ = (x);    \
    if (st_ != KDA_OK) return st_; \
  } while (0)

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_paged_append(const kda_paged_problem* p, const void* k, const void* v, void* k_pages, void* v_pages,
                            int32_t* status, void* stream) {
  using namespace kda;
  PAGED_TRY(validate_paged(p, true));
  if (p->total_tokens == 0) return KDA_OK;
  PAGED_TRY(tensor("k", k));
  PAGED_TRY(tensor("v", v));
  PAGED_TRY(tensor("k_pages", k_pages));
  PAGED_TRY(tensor("v_pages", v_pages));
  if ((uintptr_t)status & 3u) return set_error(KDA_ERR_INVALID_ARG, "status is not 4-byte aligned");
  kda_paged_append_kernel<<<(unsigned)p->total_tokens, 128, 0, (cudaStream_t)stream>>>(
      args_of(p), (const uint4*)k, (const uint4*)v, (uint4*)k_pages, (uint4*)v_pages, status);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "append launch failed: %s", cudaGetErrorString(e));
}

size_t kda_paged_attention_workspace_bytes(const kda_paged_problem* p) {
  using namespace kda;
  return validate_paged(p, false) == KDA_OK ? kHeaderBytes + paged_attention_scratch_bytes(args_of(p)) : 0;
}

kda_status kda_paged_attention(const kda_paged_problem* p, const void* q, const void* k_pages, const void* v_pages,
                               void* o, void* workspace, void* stream) {
  using namespace kda;
  PAGED_TRY(validate_paged(p, true));
  PAGED_TRY(tensor("workspace", workspace));
  cudaStream_t s = (cudaStream_t)stream;
  if (p->total_tokens == 0) {
    if (cudaMemsetAsync(workspace, 0, sizeof(int), s) != cudaSuccess)
      return set_error(KDA_ERR_CUDA, "status reset failed: %s", cudaGetErrorString(cudaGetLastError()));
    return KDA_OK;
  }
  PAGED_TRY(tensor("q", q));
  PAGED_TRY(tensor("k_pages", k_pages));
  PAGED_TRY(tensor("v_pages", v_pages));
  PAGED_TRY(tensor("o", o));
  PagedArgs a = args_of(p);
  a.q = q; a.k = k_pages; a.v = v_pages; a.o = o;
  a.status = (int*)workspace;
  a.scratch = (char*)workspace + kHeaderBytes;
  return launch_paged_attention(a, s);
}

}  // extern "C"
