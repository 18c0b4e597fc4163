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
// and needs 7 D^2 flops. 128 x 96 states of 128 with one token each take 246
// us, 97% of the measured copy rate (GDN-2: 262). Several tokens a state are
// bound by the latency from barrier to barrier of a token (about 2000 cycles
// with 16 warps an SM): 48 x 16 states of 128 with up to six tokens take 35 us
// (GDN-2; KDA 32), 2.4 times what their bytes take.
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

// Exponentials and quotients of the gates from the hardware's approximations
// (each within 2^-22 of the value): one warp forms them for a token's 128
// channels before the others can go on, and the full-precision functions made
// that the longest part of a token.
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_(float x) {  // 0 and 1 in the limits: 1 / inf, 1 / 1
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + exp2_(x * -1.4426950408889634f)));
  return y;
}

// Four columns as two pairs of fp32 values: one instruction works on a pair.
struct alignas(16) F4 {
  uint64_t a, b;
};
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t add(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ F4 add(F4 x, F4 y) { return {add(x.a, y.a), add(x.b, y.b)}; }
__device__ __forceinline__ F4 mul(F4 x, float y) {
  const uint64_t t = twice(y);
  F4 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.a) : "l"(x.a), "l"(t));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(x.b), "l"(t));
  return r;
}
__device__ __forceinline__ F4 fma(F4 x, float y, F4 z) {
  const uint64_t t = twice(y);
  F4 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.a) : "l"(x.a), "l"(t), "l"(z.a));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(x.b), "l"(t), "l"(z.b));
  return r;
}
__device__ __forceinline__ float4 values(F4 x) {
  float4 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.a));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.z), "=f"(r.w) : "l"(x.b));
  return r;
}

// CG: GDN-2's channel gates (b: erase on key channels, w: write on value
// channels); otherwise beta scales r.
template <typename T, int D, bool CG>
__global__ void __launch_bounds__(kThreads) kda_step_kernel(const StepArgs a) {
  constexpr int R = D / 16;        // rows of a thread
  constexpr int E = D / 32;        // channels of a lane in the staged vectors
  constexpr int kSplit = D / kCols;
  // Per key channel: decay, key, query, and the key under GDN-2's erase gate,
  // at place(channel): a lane writes E consecutive channels and reads rows four
  // apart, and neither falls on a few banks only.
  constexpr int kSkew = 32 + 8 / E;
  __shared__ float4 s_c[kBatch][E * kSkew];
  auto place = [](int c) { return c / E + c % E * kSkew; };
  __shared__ __align__(16) float s_v[kBatch][kCols];
  __shared__ float s_beta[kBatch];
  __shared__ __align__(16) float s_pk[2][4][kCols], s_pq[2][4][kCols];
  // kh . qh: of each staged token by one warp, or a part of every warp's sums.
  // Each is the faster way where it is taken: with one token for 128 x 96 states
  // of 128, once a token takes KDA 247 us against 261, but GDN-2
  // 269 against 263, and states of 64 lose a tenth by it.
  constexpr bool kOnce = !CG && D == 128;
  __shared__ float s_kq[kOnce ? 1 : 2][4];

  const int cb = static_cast<int>(blockIdx.x) % kSplit;
  const int item = static_cast<int>(blockIdx.x) / kSplit;
  const int n = item / a.H, h = item % a.H;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int cg = lane & 7, row0 = warp * 4 + (lane >> 3), at0 = place(row0);

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
  F4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i) S[i] = *reinterpret_cast<const F4*>(state + i * 16 * D);

  const int64_t base = (lo * a.H + h) * D;
  const T* const q = static_cast<const T*>(a.q) + base;
  const T* const k = static_cast<const T*>(a.k) + base;
  const T* const v = static_cast<const T*>(a.v) + base + cb * kCols;
  const T* const g = static_cast<const T*>(a.g) + base;
  const T* const er = static_cast<const T*>(a.b) + (CG ? base : 0);
  const T* const wr = CG ? static_cast<const T*>(a.w) + base + cb * kCols : nullptr;
  const float rate = expf(a.A_log[h]), lower2 = a.lower * 1.4426950408889634f;

  for (int64_t t0 = 0; t0 < count; t0 += kBatch) {
    const int nb = static_cast<int>(count - t0 < kBatch ? count - t0 : kBatch);
    // Channel vectors of the next nb tokens. A single token is shared out: one
    // warp normalises the query, one the key, one forms the decays, one the
    // values and gates. Of several, each warp takes a token, so that the loads
    // of all of them are in flight together.
    const bool shared_out = nb == 1;
    const int t = shared_out ? 0 : warp;
    if (t < nb) {
      const int64_t at = (t0 + t) * tok;
      float xq[E], xk[E], xe[E], xg[E], bias[E], xv = 0.f, xw = 0.f;
      const bool do_q = !shared_out || warp == 0, do_k = !shared_out || warp == 1, do_g = !shared_out || warp == 2,
                 do_v = !shared_out || warp == 3;
      if (do_q) load_row<E>(q + at, lane, xq);
      if (do_k) {
        load_row<E>(k + at, lane, xk);
        if (CG) load_row<E>(er + at, lane, xe);
      }
      if (do_g) {
        load_row<E>(g + at, lane, xg);
        load_row<E>(a.dt_bias + h * D, lane, bias);
      }
      if (do_v) {
        xv = ldf(v + at + lane);
        xw = CG ? ldf(wr + at + lane) : ldf(static_cast<const T*>(a.b) + (lo + t0 + t) * a.H + h);
      }
      if (do_q) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss += xq[i] * xq[i];
        const float inv = rsqrtf(warp_sum(ss) + a.eps) * a.scale;
#pragma unroll
        for (int i = 0; i < E; ++i) s_c[t][lane + i * kSkew].z = xq[i] * inv;
      }
      if (do_k) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss += xk[i] * xk[i];
        const float inv = rsqrtf(warp_sum(ss) + a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          s_c[t][lane + i * kSkew].y = xk[i] * inv;
          if (CG) s_c[t][lane + i * kSkew].w = xk[i] * inv * sigmoid_(xe[i]);
        }
      }
      if (do_g) {
#pragma unroll
        for (int i = 0; i < E; ++i) s_c[t][lane + i * kSkew].x = exp2_(lower2 * sigmoid_(rate * (xg[i] + bias[i])));
      }
      if (do_v) {
        const float w = sigmoid_(xw);
        s_v[t][lane] = CG ? xv * w : xv;
        if (!CG && lane == 0) s_beta[t] = w;
      }
    }
    __syncthreads();
    if (kOnce && warp < nb) {  // read after the next barrier
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float4 c = s_c[warp][lane + i * kSkew];
        ss = fmaf(c.y, c.z, ss);
      }
      ss = warp_sum(ss);
      if (lane == 0) s_kq[0][warp] = ss;
    }

    for (int t = 0; t < nb; ++t) {
      F4 pk = {0, 0}, pq = {0, 0};
      float kq = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float4 c = s_c[t][at0 + i * (16 / E)];
        S[i] = mul(S[i], c.x);
        pk = fma(S[i], CG ? c.w : c.y, pk);
        pq = fma(S[i], c.z, pq);
        if (!kOnce) kq = fmaf(c.y, c.z, kq);
      }
      // Sums over the 4 row lanes of the warp: a lane passes on what its
      // partner keeps, pk against pq, then one pair of columns against the
      // other, so that lane 8 j + cg ends with pair j % 2 of pk (j < 2) or pq.
      const bool hi = lane & 16, odd = lane & 8;
      const F4 keep = hi ? pq : pk, give = hi ? pk : pq;
      F4 w;
      w.a = add(keep.a, __shfl_xor_sync(~0u, give.a, 16));
      w.b = add(keep.b, __shfl_xor_sync(~0u, give.b, 16));
      const uint64_t pair = add(odd ? w.b : w.a, __shfl_xor_sync(~0u, odd ? w.a : w.b, 8));
      if (!kOnce) {
        kq += __shfl_xor_sync(~0u, kq, 8);
        kq += __shfl_xor_sync(~0u, kq, 16);
      }
      // then over the 4 warps; two buffers, so that one barrier a token is enough
      const int buf = t & 1;
      *reinterpret_cast<uint64_t*>(&(hi ? s_pq : s_pk)[buf][warp][cg * 4 + (odd ? 2 : 0)]) = pair;
      if (!kOnce && lane == 0) s_kq[buf][warp] = kq;
      __syncthreads();
      pk = *reinterpret_cast<const F4*>(&s_pk[buf][0][cg * 4]);
#pragma unroll
      for (int j = 1; j < 4; ++j) pk = add(pk, *reinterpret_cast<const F4*>(&s_pk[buf][j][cg * 4]));
      // r = w v - pk (KDA: beta (v - pk))
      const float beta = CG ? 1.f : s_beta[t];
      const F4 r = mul(fma(pk, -1.f, *reinterpret_cast<const F4*>(&s_v[t][cg * 4])), beta);
#pragma unroll
      for (int i = 0; i < R; ++i) S[i] = fma(r, s_c[t][at0 + i * (16 / E)].y, S[i]);
      if (row0 == 0) {
        pq = *reinterpret_cast<const F4*>(&s_pq[buf][0][cg * 4]);
        kq = kOnce ? s_kq[0][t] : s_kq[buf][0];
#pragma unroll
        for (int j = 1; j < 4; ++j) {
          pq = add(pq, *reinterpret_cast<const F4*>(&s_pq[buf][j][cg * 4]));
          if (!kOnce) kq += s_kq[buf][j];
        }
        store4(o + (t0 + t) * tok + cg * 4, values(fma(r, kq, pq)));
      }
      if (t0 + t + 1 == kept) {
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<F4*>(state + i * 16 * D) = S[i];
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
