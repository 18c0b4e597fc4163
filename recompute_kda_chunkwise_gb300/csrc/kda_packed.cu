// kda_packed.cu -- host side of causal attention over packed sequences
// (kda_attention_fwd / kda_attention_bwd of kda_blocks.h), and the list of its
// row tiles.
#include <math.h>

#include "kda_packed.cuh"

namespace kda {
namespace {

constexpr int kBuckets = 1024;

// The tiles of all sequences, heaviest first (above 1024 different weights, by
// buckets of neighbouring ones): one CTA counts the weights, sums the counts
// from the top, and places each tile. The order within a bucket is left open:
// it decides when a tile is worked on, not what comes out.
__global__ void __launch_bounds__(1024) kda_packed_list_kernel(const int32_t* cu, int N, int64_t S, int rows, int* list,
                                                               int* head, int* status) {
  __shared__ int count[kBuckets], sums[32], s_most;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  before_kernel();
  if (tid < kClearBytes / 4) head[tid] = 0;
  int bad = 0, most = 0;
  for (int n = tid; n < N; n += 1024) {
    const int lo = cu[n], hi = cu[n + 1];
    if (lo < 0 || hi < lo || hi > S || (n == 0 && lo != 0) || (n == N - 1 && hi != S)) {
      bad = 1;
      break;
    }
    most = max(most, (hi - lo + rows - 1) / rows);
  }
  if (tid == 0) s_most = 0;
  count[tid] = 0;
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0) {
      set_status(status, KDA_ERR_DEVICE_CHECK);
      list[0] = 0;
    }
    return;
  }
  most = __reduce_max_sync(~0u, most);
  if (lane == 0) atomicMax(&s_most, most);
  __syncthreads();
  most = s_most;
  // heaviest: bucket 0
  auto bucket = [&](int w) {
    const int below = most - w;
    return most <= kBuckets ? below : static_cast<int>(static_cast<int64_t>(below) * kBuckets / most);
  };
  for (int n = warp; n < N; n += 32) {
    const int tiles = (cu[n + 1] - cu[n] + rows - 1) / rows;
    for (int w = 1 + lane; w <= tiles; w += 32) atomicAdd(&count[bucket(w)], 1);
  }
  __syncthreads();
  // exclusive sums of the counts
  const int mine = count[tid];
  int x = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += sums[i];
  if (tid == 1023) list[0] = before + x;
  count[tid] = before + x - mine;
  __syncthreads();
  int4* const out = reinterpret_cast<int4*>(list + 4);
  for (int n = warp; n < N; n += 32) {
    const int lo = cu[n], L = cu[n + 1] - lo, tiles = (L + rows - 1) / rows;
    for (int w = 1 + lane; w <= tiles; w += 32) out[atomicAdd(&count[bucket(w)], 1)] = make_int4(lo, L, w, n);
  }
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
// Bytes of the list of tiles: none for one sequence.
size_t list_bytes(const kda_attention_problem* p, int rows) {
  return p->num_seqs == 1 ? 0 : up(16 + 16 * (static_cast<size_t>(p->total_tokens) / rows + p->num_seqs));
}
// Parts that a head group is cut into for dk and dv: twice the SMs in items if
// the group allows, since the longest item is then a small part of the call.
int split_of(const kda_attention_problem* p) {
  const int group = p->num_heads / p->num_kv_heads;
  const int64_t items = (p->total_tokens / 128 + 1) * p->num_kv_heads;
  int split = 1;
  for (int s = 1; s <= group; ++s)
    if (group % s == 0) {
      split = s;
      if (items * s >= 2 * kPackedMaxCtas) break;
    }
  return split;
}
size_t delta_bytes(const kda_attention_problem* p) { return up(sizeof(float) * p->total_tokens * p->num_heads); }
int64_t stat_tiles(const kda_attention_problem* p) { return p->total_tokens / 128 + p->num_seqs + 1; }
size_t stat_bytes(const kda_attention_problem* p) { return static_cast<size_t>(1024) * stat_tiles(p) * p->num_heads; }
size_t part_bytes(const kda_attention_problem* p) {
  const int split = split_of(p);
  return split == 1 ? 0 : sizeof(float) * 2 * split * p->total_tokens * p->num_kv_heads * p->head_dim;
}

kda_status tensor(const char* name, const void* p, unsigned align = 15u) {
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p & align) return set_error(KDA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align + 1);
  return KDA_OK;
}

#define TRY(x)                     \
  do {                             \
    const kda_status st_ = (x);    \
    if (st_ != KDA_OK) return st_; \
  } while (0)

kda_status validate(const kda_attention_problem* p, bool ptrs) {
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != KDA_DTYPE_BF16) return set_error(KDA_ERR_UNSUPPORTED, "dtype %d is not supported (bf16)", p->dtype);
  if (p->head_dim != 64 && p->head_dim != 128)
    return set_error(KDA_ERR_UNSUPPORTED, "head_dim %d is not supported (64 or 128)", p->head_dim);
  if (p->num_seqs < 1 || p->num_seqs > kPackedMaxSeqs)
    return set_error(KDA_ERR_INVALID_ARG, "num_seqs %d out of range (1 to %d)", p->num_seqs, kPackedMaxSeqs);
  if (p->num_kv_heads < 1 || p->num_heads < 1 || p->num_heads > 4096 || p->num_heads % p->num_kv_heads != 0)
    return set_error(KDA_ERR_INVALID_ARG, "num_heads %d must be a multiple of num_kv_heads %d (at most 4096)", p->num_heads,
                     p->num_kv_heads);
  if (p->total_tokens < 0 || p->total_tokens > ((int64_t)1 << 30))
    return set_error(KDA_ERR_INVALID_ARG, "total_tokens %lld out of range", (long long)p->total_tokens);
  if (!(p->scale > 0.f) || !isfinite(p->scale)) return set_error(KDA_ERR_INVALID_ARG, "scale must be positive and finite");
  const struct { const char* name; int64_t n, heads; } strides[] = {{"q_stride", p->q_stride, p->num_heads},
                                                                    {"k_stride", p->k_stride, p->num_kv_heads},
                                                                    {"v_stride", p->v_stride, p->num_kv_heads}};
  for (const auto& t : strides)
    if (t.n < t.heads * p->head_dim || t.n % 8 != 0 || t.n >= ((int64_t)1 << 38))
      return set_error(KDA_ERR_INVALID_ARG, "%s %lld must be at least heads * head_dim and a multiple of 8", t.name,
                       (long long)t.n);
  return ptrs ? tensor("cu_seqlens", p->cu_seqlens, 3u) : KDA_OK;
}

struct Maps {
  CUtensorMap q, k, v, d_o;
};

kda_status maps_of(const kda_attention_problem* p, const void* q, const void* k, const void* v, const void* d_o, Maps* m) {
  const bool made = in_context(reinterpret_cast<const void*>(&kda_packed_list_kernel), [&]() {
    return rows_map(&m->q, q, p->total_tokens, p->num_heads, p->head_dim, p->q_stride) &&
           rows_map(&m->k, k, p->total_tokens, p->num_kv_heads, p->head_dim, p->k_stride) &&
           rows_map(&m->v, v, p->total_tokens, p->num_kv_heads, p->head_dim, p->v_stride) &&
           (!d_o || rows_map(&m->d_o, d_o, p->total_tokens, p->num_heads, p->head_dim, (int64_t)p->num_heads * p->head_dim));
  });
  return made ? KDA_OK : set_error(KDA_ERR_CUDA, "the tensor maps of q, k, v and d_o could not be made");
}

// Status word and list of tiles; the arguments that forward and backward share.
kda_status begin(const kda_attention_problem* p, int rows, void* workspace, int32_t* status, PackedArgs* a, cudaStream_t s) {
  *a = PackedArgs{};
  a->cu = p->cu_seqlens;
  a->head = static_cast<int*>(workspace);
  a->status = status ? status : a->head;
  a->tickets = a->head + 4;
  a->S = p->total_tokens;
  a->N = p->num_seqs;
  a->Hq = p->num_heads;
  a->Hkv = p->num_kv_heads;
  a->D = p->head_dim;
  a->scale = p->scale;
  a->split = 1;
  // The header is cleared by the call's first kernel: the list's; without a list,
  // the backward's sums; or the forward's where it hands out nothing.
  static PerDevice kept;
  int64_t sms = 0;
  cudaError_t e = kept.get(&sms, [](int dev, int64_t* n) {
    int count = 0;
    const cudaError_t got = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
    *n = count;
    return got;
  });
  if (e != cudaSuccess) return set_error(KDA_ERR_CUDA, "attention set-up failed: %s", cudaGetErrorString(e));
  a->clears = rows == 256 && a->N == 1 && a->S > 0 && (a->S + 255) / 256 * a->Hq <= (sms < kPackedMaxCtas ? sms : kPackedMaxCtas);
  if (a->S == 0 || (a->N == 1 && rows == 256 && !a->clears)) {
    e = cudaMemsetAsync(workspace, 0, kClearBytes, s);
  } else if (a->N > 1) {
    int* const list = reinterpret_cast<int*>(static_cast<char*>(workspace) + kHeaderBytes);
    kda_packed_list_kernel<<<1, 1024, 0, s>>>(a->cu, a->N, a->S, rows, list, a->head, a->status);
    e = cudaGetLastError();
    a->list = list;
  }
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "attention set-up failed: %s", cudaGetErrorString(e));
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_attention_fwd_workspace_bytes(const kda_attention_problem* p) {
  using namespace kda;
  return validate(p, false) == KDA_OK ? kHeaderBytes + list_bytes(p, 256) : 0;
}

kda_status kda_attention_fwd_fresh(const kda_attention_problem* p, const void* q, const void* k, const void* v, void* o,
                                   float* lse, void* workspace, int32_t fresh, int32_t* status, void* stream) {
  using namespace kda;
  TRY(validate(p, true));
  TRY(tensor("workspace", workspace));
  if (fresh & ~3) return set_error(KDA_ERR_INVALID_ARG, "fresh %d is not 0 .. 3", fresh);
  if ((uintptr_t)status & 3u) return set_error(KDA_ERR_INVALID_ARG, "status is not 4-byte aligned");
  if (p->total_tokens > 0) {
    TRY(tensor("q", q));
    TRY(tensor("k", k));
    TRY(tensor("v", v));
    TRY(tensor("o", o));
    TRY(tensor("lse", lse, 3u));
  }
  cudaStream_t s = (cudaStream_t)stream;
  PackedArgs a;
  Maps m;
  if (p->total_tokens > 0) TRY(maps_of(p, q, k, v, nullptr, &m));
  TRY(begin(p, 256, workspace, status, &a, s));
  if (p->total_tokens == 0) return KDA_OK;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.fresh = fresh;
  const cudaError_t e = launch_packed_fwd(a, m.q, m.k, m.v, s);
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

kda_status kda_attention_fwd(const kda_attention_problem* p, const void* q, const void* k, const void* v, void* o, float* lse,
                             void* workspace, void* stream) {
  return kda_attention_fwd_fresh(p, q, k, v, o, lse, workspace, 0, nullptr, stream);
}

size_t kda_attention_bwd_workspace_bytes(const kda_attention_problem* p) {
  using namespace kda;
  return validate(p, false) == KDA_OK ? kHeaderBytes + list_bytes(p, 128) + delta_bytes(p) + stat_bytes(p) + part_bytes(p) : 0;
}

kda_status kda_attention_bwd_fresh(const kda_attention_problem* p, const void* q, const void* k, const void* v, const void* o,
                                   const float* lse, const void* d_o, void* dq, void* dk, void* dv, void* workspace,
                                   int32_t fresh, int32_t* status, void* stream) {
  using namespace kda;
  TRY(validate(p, true));
  TRY(tensor("workspace", workspace));
  if (fresh & ~1) return set_error(KDA_ERR_INVALID_ARG, "fresh %d is not 0 or 1", fresh);
  if ((uintptr_t)status & 3u) return set_error(KDA_ERR_INVALID_ARG, "status is not 4-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  PackedArgs a;
  Maps m;
  if (p->total_tokens > 0) {
    const struct { const char* name; const void* t; } all[] = {{"q", q},     {"k", k},   {"v", v},   {"o", o},
                                                               {"d_o", d_o}, {"dq", dq}, {"dk", dk}, {"dv", dv}};
    for (const auto& t : all) TRY(tensor(t.name, t.t));
    TRY(tensor("lse", lse, 3u));
    TRY(maps_of(p, q, k, v, d_o, &m));
  }
  TRY(begin(p, 128, workspace, status, &a, s));
  if (p->total_tokens == 0) return KDA_OK;
  a.fresh = fresh;
  a.o_in = static_cast<const __nv_bfloat16*>(o);
  a.d_o = static_cast<const __nv_bfloat16*>(d_o);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.lse = const_cast<float*>(lse);
  char* at = static_cast<char*>(workspace) + kHeaderBytes + list_bytes(p, 128);
  a.delta = reinterpret_cast<float*>(at);
  a.stats = reinterpret_cast<float*>(at + delta_bytes(p));
  a.stat_tiles = stat_tiles(p);
  a.part = reinterpret_cast<float*>(at + delta_bytes(p) + stat_bytes(p));
  a.split = split_of(p);
  const cudaError_t e = launch_packed_bwd(a, m.q, m.k, m.v, m.d_o, s);
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

kda_status kda_attention_bwd(const kda_attention_problem* p, const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* d_o, void* dq, void* dk, void* dv, void* workspace, void* stream) {
  return kda_attention_bwd_fresh(p, q, k, v, o, lse, d_o, dq, dk, dv, workspace, 0, nullptr, stream);
}

}  // extern "C"
