// kda_step.cu -- the recurrent form of the gated delta rule (KDA and GDN-2)
// over a pool of fp32 states: kda_step / kda_gdn2_step of kda_serving.h.
//
// Per token, with P = diag(e^g) S:
//     r = w*v - P^T (b*kh)      S' = P + kh r^T
//     o = S'^T qh = P^T qh + (kh . qh) r
// so both products with the state are of P and can be formed in one sweep
// before r is known: one reduction over the key channels per token instead
// of two, and the state stays in registers from the load to the store.
//
// Bound: HBM. One token moves 2 * 4 D^2 bytes of state per sequence and head
// and needs 7 D^2 flops; the fp32 pipes would allow about ten tokens per
// state in the time that its load and store take.
//
// Split: a value column of the state depends on no other, so a CTA takes 32
// columns (128 bytes of each state row: whole lines) of one (sequence, head)
// with 128 threads: each thread four columns (one 16-byte load) of every
// 16th row, 8 loads in flight at D = 128. Small CTAs keep many loads of
// other items in flight on the SM while one waits for its reduction; four
// CTAs per state also give one-sequence calls four times the SMs.
#include <math.h>

#include "kda_internal.cuh"
#include "kda_serving.h"

namespace kda {
namespace {

constexpr int kCols = 32;     // value columns of a CTA
constexpr int kThreads = 128;
constexpr int kBatch = 4;     // tokens whose channel vectors are staged at once

struct StepArgs {
  const void *q, *k, *v, *g, *b, *w;
  const float *A_log, *dt_bias;
  float* states;
  const int32_t *index, *commit, *cu;
  void* o;
  int* status;
  int64_t S, slots;
  int N, H;
  float scale, lower, eps;
};

// D / 32 consecutive channels of one row, a warp across the row.
template <int E>
__device__ __forceinline__ void load_row(const float* p, int lane, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 t = *reinterpret_cast<const float2*>(p + lane * E + i);
    x[i] = t.x;
    x[i + 1] = t.y;
  }
}
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, int lane, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + lane * E + i));
    x[i] = t.x;
    x[i + 1] = t.y;
  }
}

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

// CG: GDN-2's channel gates (b: erase on key channels, w: write on value
// channels); otherwise beta scales r.
template <typename T, int D, bool CG>
__global__ void __launch_bounds__(kThreads) kda_step_kernel(const StepArgs a) {
  constexpr int R = D / 16;        // rows of a thread
  constexpr int E = D / 32;        // channels of a lane in the staged vectors
  constexpr int kSplit = D / kCols;
  __shared__ float s_q[kBatch][D], s_k[kBatch][D], s_a[kBatch][D], s_b[CG ? kBatch : 1][D];
  __shared__ __align__(16) float s_v[kBatch][kCols];
  __shared__ float s_beta[kBatch];
  __shared__ __align__(16) float4 s_pk[2][4][8], s_pq[2][4][8];
  __shared__ float s_kq[2][4];

  const int cb = static_cast<int>(blockIdx.x) % kSplit;
  const int item = static_cast<int>(blockIdx.x) / kSplit;
  const int n = item / a.H, h = item % a.H;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int cg = lane & 7, row0 = warp * 4 + (lane >> 3);

  const int64_t lo = a.cu[n], hi = a.cu[n + 1];
  const int64_t slot = a.index ? a.index[n] : n;
  const int32_t upto = a.commit ? a.commit[n] : INT32_MAX;
  if (lo < 0 || hi < lo || hi > a.S || slot >= a.slots || upto < 0 || (n == 0 && lo != 0) ||
      (n == a.N - 1 && hi != a.S)) {
    if (tid == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  const int64_t count = hi - lo;
  if (count == 0) return;
  const int64_t kept = upto < count ? upto : count;

  T* const o = static_cast<T*>(a.o) + (lo * a.H + h) * D + cb * kCols;
  const int64_t tok = static_cast<int64_t>(a.H) * D;  // elements from one token to the next
  if (slot < 0) {  // inactive sequence
    for (int64_t i = tid; i < count * kCols; i += kThreads) stf(o + i / kCols * tok + i % kCols, 0.f);
    return;
  }
  float* const state = a.states + ((slot * a.H + h) * D + row0) * D + cb * kCols + cg * 4;
  float4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i) S[i] = *reinterpret_cast<const float4*>(state + i * 16 * D);

  const int64_t base = (lo * a.H + h) * D;
  const T* const q = static_cast<const T*>(a.q) + base;
  const T* const k = static_cast<const T*>(a.k) + base;
  const T* const v = static_cast<const T*>(a.v) + base + cb * kCols;
  const T* const g = static_cast<const T*>(a.g) + base;
  const T* const er = static_cast<const T*>(a.b) + (CG ? base : 0);
  const T* const wr = CG ? static_cast<const T*>(a.w) + base + cb * kCols : nullptr;
  const float rate = expf(a.A_log[h]);

  for (int64_t t0 = 0; t0 < count; t0 += kBatch) {
    const int nb = static_cast<int>(count - t0 < kBatch ? count - t0 : kBatch);
    // Channel vectors of the next nb tokens: one warp normalises the queries,
    // one the keys, one forms the decays, one the values and gates.
    for (int t = 0; t < nb; ++t) {
      const int64_t at = (t0 + t) * tok;
      if (warp == 0 || warp == 1) {
        float x[E], e[E];
        load_row<E>((warp == 0 ? q : k) + at, lane, x);
        if (CG && warp == 1) load_row<E>(er + at, lane, e);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss += x[i] * x[i];
        const float inv = rsqrtf(warp_sum(ss) + a.eps) * (warp == 0 ? a.scale : 1.f);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float y = x[i] * inv;
          (warp == 0 ? s_q : s_k)[t][lane * E + i] = y;
          if (CG && warp == 1) s_b[t][lane * E + i] = y * sigmoidf_(e[i]);
        }
      } else if (warp == 2) {
        float x[E], bias[E];
        load_row<E>(g + at, lane, x);
        load_row<E>(a.dt_bias + h * D, lane, bias);
#pragma unroll
        for (int i = 0; i < E; ++i)
          s_a[t][lane * E + i] = expf(a.lower * sigmoidf_(rate * (x[i] + bias[i])));
      } else {
        float x = ldf(v + at + lane);
        if (CG)
          x *= sigmoidf_(ldf(wr + at + lane));
        else if (lane == 0)
          s_beta[t] = sigmoidf_(ldf(static_cast<const T*>(a.b) + (lo + t0 + t) * a.H + h));
        s_v[t][lane] = x;
      }
    }
    __syncthreads();

    for (int t = 0; t < nb; ++t) {
      float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
      float kq = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = row0 + i * 16;
        const float al = s_a[t][row], kr = s_k[t][row], qr = s_q[t][row];
        const float br = CG ? s_b[CG ? t : 0][row] : kr;
        S[i].x *= al; S[i].y *= al; S[i].z *= al; S[i].w *= al;
        pk.x = fmaf(S[i].x, br, pk.x); pk.y = fmaf(S[i].y, br, pk.y);
        pk.z = fmaf(S[i].z, br, pk.z); pk.w = fmaf(S[i].w, br, pk.w);
        pq.x = fmaf(S[i].x, qr, pq.x); pq.y = fmaf(S[i].y, qr, pq.y);
        pq.z = fmaf(S[i].z, qr, pq.z); pq.w = fmaf(S[i].w, qr, pq.w);
        kq = fmaf(kr, qr, kq);
      }
      // Sum over the 4 row lanes of the warp, then over the 4 warps; two
      // buffers, so that one barrier a token is enough.
#pragma unroll
      for (int m = 8; m <= 16; m <<= 1) {
        pk.x += __shfl_xor_sync(~0u, pk.x, m); pk.y += __shfl_xor_sync(~0u, pk.y, m);
        pk.z += __shfl_xor_sync(~0u, pk.z, m); pk.w += __shfl_xor_sync(~0u, pk.w, m);
        pq.x += __shfl_xor_sync(~0u, pq.x, m); pq.y += __shfl_xor_sync(~0u, pq.y, m);
        pq.z += __shfl_xor_sync(~0u, pq.z, m); pq.w += __shfl_xor_sync(~0u, pq.w, m);
        kq += __shfl_xor_sync(~0u, kq, m);
      }
      const int buf = t & 1;
      if (lane < 8) {
        s_pk[buf][warp][cg] = pk;
        s_pq[buf][warp][cg] = pq;
        if (lane == 0) s_kq[buf][warp] = kq;
      }
      __syncthreads();
      pk = s_pk[buf][0][cg];
      pq = s_pq[buf][0][cg];
      kq = s_kq[buf][0];
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        const float4 x = s_pk[buf][j][cg], y = s_pq[buf][j][cg];
        pk.x += x.x; pk.y += x.y; pk.z += x.z; pk.w += x.w;
        pq.x += y.x; pq.y += y.y; pq.z += y.z; pq.w += y.w;
        kq += s_kq[buf][j];
      }
      const float4 x = *reinterpret_cast<const float4*>(&s_v[t][cg * 4]);
      const float beta = CG ? 1.f : s_beta[t];
      const float4 r = make_float4(beta * (x.x - pk.x), beta * (x.y - pk.y), beta * (x.z - pk.z), beta * (x.w - pk.w));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float kr = s_k[t][row0 + i * 16];
        S[i].x = fmaf(kr, r.x, S[i].x); S[i].y = fmaf(kr, r.y, S[i].y);
        S[i].z = fmaf(kr, r.z, S[i].z); S[i].w = fmaf(kr, r.w, S[i].w);
      }
      if (row0 == 0)
        store4(o + (t0 + t) * tok + cg * 4, make_float4(fmaf(kq, r.x, pq.x), fmaf(kq, r.y, pq.y), fmaf(kq, r.z, pq.z),
                                                        fmaf(kq, r.w, pq.w)));
      if (t0 + t + 1 == kept) {
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(state + i * 16 * D) = S[i];
      }
    }
    __syncthreads();  // the staged vectors are read: the next batch may replace them
  }
}

template <typename T, int D>
void launch(const StepArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.N) * static_cast<unsigned>(a.H) * (D / kCols);
  if (a.w)
    kda_step_kernel<T, D, true><<<grid, kThreads, 0, s>>>(a);
  else
    kda_step_kernel<T, D, false><<<grid, kThreads, 0, s>>>(a);
}

bool bad_ptr(const char* name, const void* p, bool optional = false) {
  if (!p && !optional) {
    set_error(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    return true;
  }
  if ((uintptr_t)p & 15u) {
    set_error(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return true;
  }
  return false;
}

kda_status step(const kda_problem* p, const void* q, const void* k, const void* v, const void* g_raw, const void* b,
                const void* w, bool channel, const float* A_log, const float* dt_bias, float* states, int64_t num_slots,
                const int32_t* state_index, const int32_t* commit, void* o, int32_t* status, void* stream) {
  const kda_status st = validate_problem(p);
  if (st != KDA_OK) return st;
  if (p->flags != (channel ? KDA_FLAG_CHANNEL_GATES : 0))
    return set_error(KDA_ERR_INVALID_ARG, channel ? "kda_gdn2_step needs flags = KDA_FLAG_CHANNEL_GATES (got 0x%x)"
                                                  : "kda_step needs flags = 0 (got 0x%x)", p->flags);
  if ((int64_t)p->num_seqs * p->num_heads > (1 << 28))
    return set_error(KDA_ERR_INVALID_ARG, "too many sequences x heads for one step");
  if (num_slots < 1 || (!state_index && num_slots < p->num_seqs))
    return set_error(KDA_ERR_INVALID_ARG, "num_slots %lld is too small", (long long)num_slots);
  if (num_slots > ((int64_t)1 << 46) / ((int64_t)p->num_heads * p->head_dim * p->head_dim))
    return set_error(KDA_ERR_INVALID_ARG, "num_slots %lld is too large", (long long)num_slots);
  if (p->total_tokens == 0) return KDA_OK;
  if (bad_ptr("q", q) || bad_ptr("k", k) || bad_ptr("v", v) || bad_ptr("g_raw", g_raw) ||
      bad_ptr(channel ? "erase_raw" : "beta_raw", b) || (channel && bad_ptr("write_raw", w)) ||
      bad_ptr("A_log", A_log) || bad_ptr("dt_bias", dt_bias) || bad_ptr("states", states) || bad_ptr("o", o))
    return KDA_ERR_INVALID_ARG;
  if (((uintptr_t)state_index | (uintptr_t)commit | (uintptr_t)status) & 3u)
    return set_error(KDA_ERR_INVALID_ARG, "state_index, commit and status must be 4-byte aligned");
  StepArgs a{q, k, v, g_raw, b, channel ? w : nullptr, A_log, dt_bias, states, state_index, commit, p->cu_seqlens, o,
             status, p->total_tokens, num_slots, p->num_seqs, p->num_heads, p->scale, p->gate_lower_bound, p->l2_eps};
  cudaStream_t s = (cudaStream_t)stream;
  if (p->dtype == KDA_DTYPE_BF16)
    p->head_dim == 128 ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 64>(a, s);
  else
    p->head_dim == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "step launch failed: %s", cudaGetErrorString(e));
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_step(const kda_problem* p, const void* q, const void* k, const void* v, const void* g_raw,
                    const void* beta_raw, const float* A_log, const float* dt_bias, float* states, int64_t num_slots,
                    const int32_t* state_index, const int32_t* commit, void* o, int32_t* status, void* stream) {
  return kda::step(p, q, k, v, g_raw, beta_raw, nullptr, false, A_log, dt_bias, states, num_slots, state_index, commit,
                   o, status, stream);
}

kda_status kda_gdn2_step(const kda_problem* p, const void* q, const void* k, const void* v, const void* g_raw,
                         const void* erase_raw, const void* write_raw, const float* A_log, const float* dt_bias,
                         float* states, int64_t num_slots, const int32_t* state_index, const int32_t* commit, void* o,
                         int32_t* status, void* stream) {
  return kda::step(p, q, k, v, g_raw, erase_raw, write_raw, true, A_log, dt_bias, states, num_slots, state_index,
                   commit, o, status, stream);
}

}  // extern "C"
