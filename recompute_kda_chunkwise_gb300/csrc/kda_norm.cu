// kda_norm.cu -- the norm between blocks, forward and backward:
// kda_block_norm_fwd / kda_block_norm_bwd of kda_serving.h.
//
// Per row of D elements, with ry = 1 / sqrt(mean(y^2) + eps), yn = y ry,
// s = sigmoid(z):
//     h' = a h + b w_post yn s        rh = 1 / sqrt(mean(h'^2) + eps), hn = h' rh
//     n  = w_pre hn
// and backwards, with d = dn w_pre:
//     D  = dh_out + rh (d - hn mean(d hn))     dw_pre = sum_rows dn hn
//     dh = a D      du = b D      dz = du yn w_post s (1 - s)
//     t  = du s     dw_post = sum_rows t yn    dy = ry (t w_post - yn mean(t w_post yn))
// The backward forms yn, s and h' again from y, z and h: it reads those rows
// anyway, and needs no statistics or h' from the forward.
//
// Bound: HBM; each tensor is read or written once. A row stays at hand between
// its reductions. A group of G threads takes a row; a thread holds NV 16-byte
// vectors of it. Forward and backward together, bf16: head norms of 128 with a
// gate take 254 us, 93% of the measured copy rate; 8192 rows of 4096 with the
// next norm 162 us, 79%. There a row is spread over a CTA and its reductions
// are barriers: between them the SM waits for the slowest warp, and the weight
// gradients' registers leave room for one CTA.
//
// Rows of an odd width start anywhere within 16 bytes. There a group works on
// the aligned vectors that cover its row, `shift` elements before its start;
// what lies outside the row is set to zero as it is read and not written. The
// rows of a group are a multiple of the vector's elements apart, so its shift
// is the same for all of them, and with it a thread's columns: weights and
// their gradients stay in registers as for other widths.
//
// x - xn mean(x xn) takes x's part along the row out. In a row of one element
// that is all of x but the share eps r^2 that eps keeps, far below the
// rounding of the two terms: width 1 multiplies by that share instead.
#include <math.h>

#include "kda_device.cuh"
#include "kda_internal.cuh"
#include "kda_serving.h"

namespace kda {
namespace {

constexpr int kMaxWidth = 8192;
constexpr int kMaxCtas = 152 * 8;  // of a backward: rows of its workspace's partial weight gradients

struct NormArgs {
  const void *y, *z, *h, *dho, *dn;
  const float *wpost, *wpre;
  void *ho, *n, *dy, *dz, *dh;
  float* part;  // [2][ctas][width] partial weight gradients (post, then pre)
  int64_t rows;
  int width;
  float a, b, eps;
};

// kVec consecutive elements as loaded.
template <typename T, int V>
struct Raw;
template <>
struct alignas(16) Raw<__nv_bfloat16, 8> {
  uint4 u;
};
template <>
struct alignas(16) Raw<float, 4> {
  float4 u;
};
// Arithmetic on the values of a vector: pairs where V is even (one
// instruction for two fp32 operations), single values otherwise.
struct F2 {
  uint64_t u;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 both(F2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.u));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ float sum(F2 a) { return both(a).x + both(a).y; }
__device__ __forceinline__ F2 all(float x) { return f2(x, x); }

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 8>& r, F2 (&x)[4]) {
  const uint32_t u[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, F2 (&x)[2]) {
  x[0] = f2(r.u.x, r.u.y);
  x[1] = f2(r.u.z, r.u.w);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const F2 (&x)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 t = __float22bfloat162_rn(both(x[i]));
    u[i] = *reinterpret_cast<uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void put(float* p, const F2 (&x)[2]) {
  const float2 a = both(x[0]), b = both(x[1]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
// A thread's vectors of a row: vector j starts at column at(j). ODD: rows
// start `shift` elements into an aligned vector, and the first and last one
// may reach over the row's ends.
template <int V, int G, bool ODD>
struct Span {
  int c0, width;
  __device__ __forceinline__ Span(int lane, int64_t row, int w)
      : c0(lane * V - (ODD ? static_cast<int>(row % V * (w % V) % V) : 0)), width(w) {}
  __device__ __forceinline__ int at(int j) const { return c0 + j * G * V; }
  __device__ __forceinline__ bool any(int j) const { return at(j) < width; }
  __device__ __forceinline__ bool whole(int j) const { return !ODD || (at(j) >= 0 && at(j) + V <= width); }
  // x's values outside the row set to zero
  template <int N>
  __device__ __forceinline__ void clip(int j, F2 (&x)[N]) const {
    if (whole(j)) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 t = both(x[i]);
      const int c = at(j) + 2 * i;
      x[i] = f2(c >= 0 && c < width ? t.x : 0.f, c >= -1 && c + 1 < width ? t.y : 0.f);
    }
  }
  template <typename T, int N>
  __device__ __forceinline__ void store(T* row, int j, const F2 (&x)[N]) const {
    if (whole(j)) {
      put(row + at(j), x);
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 t = both(x[i]);
      const int c = at(j) + 2 * i;
      if (c >= 0 && c < width) stf(row + c, t.x);
      if (c >= -1 && c + 1 < width) stf(row + c + 1, t.y);
    }
  }
  // weights of vector j (1 without weights)
  template <int N>
  __device__ __forceinline__ void weights(const float* w, int j, F2 (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float t[4] = {1.f, 1.f, 1.f, 1.f};
      const int c = at(j) + 2 * i;
      if (w != nullptr) {
        if constexpr (ODD) {
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = c + k >= 0 && c + k < width ? w[c + k] : 0.f;
        } else {
          *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(w + c);
        }
      }
      x[i] = f2(t[0], t[1]);
      x[i + 1] = f2(t[2], t[3]);
    }
  }
};

// A thread's weights: in registers for all its rows where it holds one vector
// of a row (read every row they cost the L1 more than the row itself: 4 bytes
// an element against 2), from L1 each time where it holds more.
template <int V, int NV, int G, bool ODD>
struct Weights {
  static constexpr int N = V / 2;
  static constexpr bool kKept = NV == 1;
  const float* w;
  const Span<V, G, ODD>& span;
  F2 kept[kKept ? N : 1];
  __device__ __forceinline__ Weights(const float* p, const Span<V, G, ODD>& sp) : w(p), span(sp) {
    if constexpr (kKept) {
      if (span.any(0)) span.weights(w, 0, kept);
    }
  }
  __device__ __forceinline__ void get(int j, F2 (&x)[N]) const {
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = kept[i];
    } else {
      span.weights(w, j, x);
    }
  }
};

// Sums of N values over a group of G threads (G <= 32: lanes; else the whole
// CTA of G threads, through `sh`, whose halves alternate so that one barrier
// a reduction is enough).
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float* sh, int& turn) {
  constexpr int L = G < 32 ? G : 32;
#pragma unroll
  for (int m = L / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(~0u, x[i], m);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    float* const s = sh + turn * 3 * 32;
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i * 32 + warp] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = s[i * 32 + lane % W];
#pragma unroll
      for (int m = W / 2; m > 0; m >>= 1) t += __shfl_xor_sync(~0u, t, m);
      x[i] = t;
    }
  }
}

// s = sigmoid(z) = 1 / (1 + e) and n = sigmoid(-z) = e s with e = exp(-z), so
// that neither is a difference that cancels. e stops at 2^127, where 1 + e is
// still finite and its reciprocal, below fp32's normal numbers, is 0: from
// z = -87.4 down to -inf the gate is shut, and the gradient through it is 0.
__device__ __forceinline__ F2 gate_exp(F2 z) {
  const float2 t = both(mul(z, all(-1.4426950408889634f)));
  float ex, ey;
  asm("{.reg .f32 t;\n min.NaN.f32 t, %1, 0f42FE0000;\n ex2.approx.ftz.f32 %0, t;\n}" : "=f"(ex) : "f"(t.x));
  asm("{.reg .f32 t;\n min.NaN.f32 t, %1, 0f42FE0000;\n ex2.approx.ftz.f32 %0, t;\n}" : "=f"(ey) : "f"(t.y));
  return f2(ex, ey);
}
__device__ __forceinline__ F2 gate_of(F2 e) {
  const float2 d = both(add(e, all(1.f)));
  float x, y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d.y));
  return f2(x, y);
}

// How a thread gets its share of its group's rows: 16-byte vectors by
// asynchronous copies, one or two rows ahead, into a ring of shared memory in
// which a thread reads only what it copied itself. The rows ahead hold no
// registers and need no barrier. More of them do not pay: head norms of 128 in
// training take 254 us with one row ahead, 264 with two, 275 with three, and
// rows of 4096 163, 164 and 173 with two, three and four. Tensors that are
// absent are not read.
// FILL: the ring holds zeros in their place (the gate's: infinities, whose
// sigmoid is 1), and whoever reads it need not ask which there are.
enum Which { kY, kZ, kDho, kH, kDn };  // a backward without the next norm has no kH, kDn; a forward the first two and kH
template <typename T>
__device__ __forceinline__ uint4 infinities() {
  const uint32_t u = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u;
  return make_uint4(u, u, u, u);
}
template <typename T, int V, int NV, int G, int NT, bool ODD, int SLOTS, bool FILL>
struct Rows {
  static constexpr int kStage = SLOTS * NV * NT * 16;  // bytes
  static constexpr int kFit = 200 * 1024 / kStage;
  static constexpr int kWant = G > 32 ? 3 : 2;
  static constexpr int kDepth = kFit < kWant ? kFit : kWant;
  static constexpr size_t kBytes = static_cast<size_t>(kDepth) * kStage;
  // The next row is at hand too: where a reduction is a barrier of the CTA,
  // its first one shares the last one of the row before.
  static constexpr bool kNext = G > 32 && kDepth >= 3;
  static_assert(kDepth >= 1, "");
  const NormArgs& a;
  const Span<V, G, ODD>& span;
  const void* const (&from)[SLOTS];
  uint8_t* ring;
  int64_t step, ahead;  // rows between two turns; the next row to copy
  int in, out;          // ring positions

  __device__ __forceinline__ Rows(const NormArgs& args, const Span<V, G, ODD>& sp, const void* const (&f)[SLOTS],
                                  uint8_t* sm, int64_t row, int64_t st)
      : a(args), span(sp), from(f), ring(sm), step(st), ahead(row), in(0), out(kDepth - 1) {
    if constexpr (FILL) {
#pragma unroll
      for (int s = 0; s < SLOTS; ++s)
        if (!from[s])
          for (int i = 0; i < kDepth * NV; ++i)
            *reinterpret_cast<uint4*>(slot(i / NV, s, i % NV)) = s == kZ ? infinities<T>() : make_uint4(0, 0, 0, 0);
    }
    for (int i = 0; i + 1 < kDepth; ++i) copy();
  }
  __device__ __forceinline__ uint8_t* slot(int stage, int s, int j) const {
    return ring + stage * kStage + ((s * NV + j) * NT + threadIdx.x) * 16;
  }
  __device__ __forceinline__ void copy() {
    if (ahead < a.rows) {
      const int64_t base = ahead * a.width;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (span.any(j)) {
          int bytes = 16;
          if constexpr (ODD) {  // the last vector of the tensor may be short
            const int64_t left = (a.rows * a.width - base - span.at(j)) * static_cast<int64_t>(sizeof(T));
            if (left < 16) bytes = static_cast<int>(left);
          }
#pragma unroll
          for (int s = 0; s < SLOTS; ++s)
            if (from[s])
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                               static_cast<uint32_t>(__cvta_generic_to_shared(slot(in, s, j)))),
                           "l"(static_cast<const T*>(from[s]) + base + span.at(j)), "r"(bytes)
                           : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += step;
    if (++in == kDepth) in = 0;
  }
  // The next row of this group (kNext: and the one after it) is at hand afterwards.
  __device__ __forceinline__ void turn() {
    copy();
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - (kNext ? 2 : 1)) : "memory");
    if (++out == kDepth) out = 0;
  }
  __device__ __forceinline__ void get(int s, int j, F2 (&x)[V / 2], bool next = false) const {
    const int stage = !next ? out : out + 1 == kDepth ? 0 : out + 1;
    unpack(*reinterpret_cast<const Raw<T, V>*>(slot(stage, s, j)), x);
    span.clip(j, x);
  }
  // This thread's share of the sum of y^2 over `row`, the one at hand or the next.
  __device__ __forceinline__ float squares(int64_t row, bool next) const {
    F2 t = all(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (row < a.rows && span.any(j)) {
        F2 y[V / 2];
        get(kY, j, y, next);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) t = fma(y[i], y[i], t);
      }
    return sum(t);
  }
};

template <typename T, int V, int NV, int G, int NT, bool ODD>
__global__ void __launch_bounds__(NT) norm_fwd_kernel(const NormArgs a) {
  using F = F2;
  constexpr int kGroups = NT / G, NP = V / 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sh[2 * 3 * 32];
  int turn = 0;
  const int lane = static_cast<int>(threadIdx.x) % G;
  const float inv = 1.f / static_cast<float>(a.width);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / G;
  const Span<V, G, ODD> span(lane, row, a.width);
  const Weights<V, NV, G, ODD> wpost(a.wpost, span), wpre(a.wpre, span);
  const void* const from[3] = {a.y, a.z, a.h};
  Rows<T, V, NV, G, NT, ODD, 3, false> in(a, span, from, ring, row, step);
  constexpr bool kNext = in.kNext;
  float yy[1];
  if constexpr (kNext) {
    in.turn();
    yy[0] = in.squares(row, false);
    group_sum<G>(yy, sh, turn);
  }
  // every group of a CTA makes the same number of turns (the reductions are collective)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups; r0 < a.rows; r0 += step, row += step) {
    if constexpr (!kNext) in.turn();
    const bool live = row < a.rows;
    const int64_t base = row * a.width;
    auto here = [&](int j) { return live && span.any(j); };
    F x[NV][NP], hh = all(0.f);
    if constexpr (!kNext) {
      yy[0] = in.squares(row, false);
      group_sum<G>(yy, sh, turn);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (here(j)) in.get(kY, j, x[j]);
    const F scale = all(rsqrtf(yy[0] * inv + a.eps) * a.b), keep = all(a.a);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (here(j)) {
        F w[NP], t[NP];
        wpost.get(j, w);
#pragma unroll
        for (int i = 0; i < NP; ++i) x[j][i] = mul(x[j][i], mul(scale, w[i]));
        if (a.z) {
          in.get(kZ, j, t);
#pragma unroll
          for (int i = 0; i < NP; ++i) x[j][i] = mul(x[j][i], gate_of(gate_exp(t[i])));
        }
        if (a.h) {
          in.get(2, j, t);
#pragma unroll
          for (int i = 0; i < NP; ++i) x[j][i] = fma(keep, t[i], x[j][i]);
        }
        span.store(static_cast<T*>(a.ho) + base, j, x[j]);
#pragma unroll
        for (int i = 0; i < NP; ++i) hh = fma(x[j][i], x[j][i], hh);
      }
    }
    if (a.n) {
      float two[kNext ? 2 : 1] = {sum(hh)};
      if constexpr (kNext) two[1] = in.squares(row + step, true);
      group_sum<G>(two, sh, turn);
      if constexpr (kNext) yy[0] = two[1];
      const F r = all(rsqrtf(two[0] * inv + a.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (here(j)) {
          F w[NP];
          wpre.get(j, w);
#pragma unroll
          for (int i = 0; i < NP; ++i) x[j][i] = mul(x[j][i], mul(r, w[i]));
          span.store(static_cast<T*>(a.n) + base, j, x[j]);
        }
      }
    } else if constexpr (kNext) {
      yy[0] = in.squares(row + step, true);
      group_sum<G>(yy, sh, turn);
    }
    if constexpr (kNext) in.turn();
  }
}

// PRE: the next norm takes part (dn and w_pre are given).
template <typename T, int V, int NV, int G, int NT, bool ODD, bool PRE>
__global__ void __launch_bounds__(NT, NT == 256 ? (PRE ? 2 : 3) : 1) norm_bwd_kernel(const NormArgs a) {
  using F = F2;
  constexpr int kGroups = NT / G, NP = V / 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sh[2 * 3 * 32];
  int turn = 0;
  const int lane = static_cast<int>(threadIdx.x) % G, group = static_cast<int>(threadIdx.x) / G;
  const float inv = 1.f / static_cast<float>(a.width);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const bool one = a.width == 1;
  F gpost[NV][NP], gpre[PRE ? NV : 1][NP];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < NP; ++i) gpost[j][i] = gpre[PRE ? j : 0][i] = all(0.f);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const Span<V, G, ODD> span(lane, row, a.width);
  const Weights<V, NV, G, ODD> wpost(a.wpost, span), wpre(PRE ? a.wpre : nullptr, span);
  constexpr int kSlots = PRE ? 5 : 3;
  const void* const five[5] = {a.y, a.z, a.dho, a.h, a.dn};
  const void* const(&from)[kSlots] = reinterpret_cast<const void* const(&)[kSlots]>(five);
  Rows<T, V, NV, G, NT, ODD, kSlots, PRE> in(a, span, from, ring, row, step);
  constexpr bool kNext = in.kNext;
  float yy[1];
  if constexpr (kNext) {
    in.turn();
    yy[0] = in.squares(row, false);
    group_sum<G>(yy, sh, turn);
  }
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups; r0 < a.rows; r0 += step, row += step) {
    if constexpr (!kNext) in.turn();
    const bool live = row < a.rows;
    const int64_t base = row * a.width;
    auto here = [&](int j) { return live && span.any(j); };
    if constexpr (!kNext) {
      yy[0] = in.squares(row, false);
      group_sum<G>(yy, sh, turn);
    }
    const float iy = rsqrtf(yy[0] * inv + a.eps);
    // yn and d are formed again in each stage from the row at hand: registers,
    // not instructions, limit the warps here.
    F hp[PRE ? NV : 1][NP];  // h'
    F q[NV][NP];             // exp(-z) of the gate, then the gradient of yn, until dy is formed
    F hh = all(0.f), hd = all(0.f);
    if constexpr (PRE) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (here(j)) {
          F t[NP], w[NP];
          in.get(kY, j, t);
          wpost.get(j, w);
#pragma unroll
          for (int i = 0; i < NP; ++i) hp[j][i] = mul(mul(t[i], all(iy * a.b)), w[i]);
          {
            in.get(kZ, j, t);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              q[j][i] = gate_exp(t[i]);
              hp[j][i] = mul(hp[j][i], gate_of(q[j][i]));
            }
          }
          {
            in.get(kH, j, t);
#pragma unroll
            for (int i = 0; i < NP; ++i) hp[j][i] = fma(all(a.a), t[i], hp[j][i]);
          }
          in.get(kDn, j, t);
          wpre.get(j, w);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            hh = fma(hp[j][i], hp[j][i], hh);
            hd = fma(hp[j][i], mul(t[i], w[i]), hd);
          }
        }
      }
    }
    F ih = all(0.f), dk = ih, dp = ih;  // dh' = dh_out + dk d - dp h'
    if constexpr (PRE) {
      float two[2] = {sum(hh), sum(hd)};
      group_sum<G>(two, sh, turn);
      const float r = rsqrtf(two[0] * inv + a.eps);
      ih = all(r);
      // r^3 alone leaves fp32's range long before r^2 mean(d hn) does: r times each factor in turn
      dk = all(r * (one ? a.eps * r * r : 1.f));
      dp = all(one ? 0.f : -r * (r * (r * (two[1] * inv))));
    }
    F ty = all(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (here(j)) {
        F d[NP], w[NP], t[NP];
        if (PRE || a.dho)
          in.get(kDho, j, d);
        else
#pragma unroll
          for (int i = 0; i < NP; ++i) d[i] = all(0.f);
        if constexpr (PRE) {
          in.get(kDn, j, t);
          wpre.get(j, w);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            gpre[j][i] = fma(t[i], mul(hp[j][i], ih), gpre[j][i]);
            d[i] = fma(hp[j][i], dp, fma(mul(t[i], w[i]), dk, d[i]));
          }
        }
        if (a.dh) {
#pragma unroll
          for (int i = 0; i < NP; ++i) t[i] = mul(all(a.a), d[i]);
          span.store(static_cast<T*>(a.dh) + base, j, t);
        }
        F yn[NP];
        in.get(kY, j, yn);
        wpost.get(j, w);
        F z[NP];
        if constexpr (!PRE) {
          if (a.z) {
            in.get(kZ, j, z);
#pragma unroll
            for (int i = 0; i < NP; ++i) q[j][i] = gate_exp(z[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          F sg = all(1.f), sn = sg;
          if (PRE || a.z) {
            sg = gate_of(q[j][i]);
            sn = mul(q[j][i], sg);
          }
          yn[i] = mul(yn[i], all(iy));
          const F du = mul(d[i], mul(sg, all(a.b)));
          gpost[j][i] = fma(du, yn[i], gpost[j][i]);
          q[j][i] = mul(du, w[i]);
          ty = fma(q[j][i], yn[i], ty);
          z[i] = mul(mul(q[j][i], yn[i]), sn);
        }
        if (a.z) span.store(static_cast<T*>(a.dz) + base, j, z);
      }
    }
    float two[kNext ? 2 : 1] = {sum(ty)};
    if constexpr (kNext) two[1] = in.squares(row + step, true);
    group_sum<G>(two, sh, turn);
    if constexpr (kNext) yy[0] = two[1];
    const F yk = all(iy * (one ? a.eps * iy * iy : 1.f)), yp = all(one ? 0.f : -iy * iy * (two[0] * inv));
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (here(j)) {
        F y[NP];
        in.get(kY, j, y);
#pragma unroll
        for (int i = 0; i < NP; ++i) q[j][i] = fma(y[i], yp, mul(q[j][i], yk));
        span.store(static_cast<T*>(a.dy) + base, j, q[j]);
      }
    if constexpr (kNext) in.turn();
  }
  // This CTA's share of the weight gradients: its groups' sums, in order.
  // (Without dn, w_pre's gradient is zero: gpre was never added to.)
  if (!a.part) return;
  float* const acc = reinterpret_cast<float*>(ring);  // [groups][G * NV * V], where a CTA has several groups
  if constexpr (kGroups > 1) __syncthreads();         // every group is done with the ring
  const int64_t half = static_cast<int64_t>(gridDim.x) * a.width;
  float* const out = a.part + static_cast<int64_t>(blockIdx.x) * a.width;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.wpost : a.wpre) == nullptr) continue;
    constexpr int W = G * NV * V;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 t = both(which == 0 ? gpost[j][i / 2] : gpre[PRE ? j : 0][i / 2]);
        const float v = i % 2 ? t.y : t.x;
        const int c = span.at(j) + i;
        if constexpr (kGroups > 1)
          acc[group * W + (j * G + lane) * V + i] = v;
        else if (c >= 0 && c < a.width)
          out[which * half + c] = v;
      }
    }
    if constexpr (kGroups > 1) {
      __syncthreads();
      for (int c = static_cast<int>(threadIdx.x); c < a.width; c += NT) {
        float t = 0.f;
        for (int g = 0; g < kGroups; ++g)
          t += acc[g * W + c - Span<V, G, ODD>(0, static_cast<int64_t>(blockIdx.x) * kGroups + g, a.width).at(0)];
        out[which * half + c] = t;
      }
      __syncthreads();
    }
  }
}

// Sums the CTAs' shares in a fixed order: 32 columns a CTA, 32 rows of threads.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* part, int ctas, int width, float* dpost,
                                                           float* dpre) {
  __shared__ float s[32][33];
  const float* const p = part + static_cast<int64_t>(blockIdx.y) * ctas * width;
  float* const out = blockIdx.y == 0 ? dpost : dpre;
  if (out == nullptr) return;
  const int c = static_cast<int>(blockIdx.x) * 32 + threadIdx.x;
  float t = 0.f;
  if (c < width)
    for (int r = static_cast<int>(threadIdx.y); r < ctas; r += 32) t += p[static_cast<int64_t>(r) * width + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int col = static_cast<int>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < width) out[col] = t;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs that a device's SMs hold at once (a launch's loop takes the rest of the rows), at most `most`.
template <typename K>
cudaError_t resident(K kernel, int threads, size_t smem, int most, int dev, int64_t* ctas) {
  int sms = 0, per = 0;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  const int fit = (sms < 8 ? 8 : sms) * (per < 1 ? 1 : per);
  *ctas = (fit < most ? fit : most) / 8 * 8;  // a group's rows are a multiple of the vector's elements apart
  return e;
}

template <typename T, int V, int NV, int G, int NT, bool ODD, bool PRE>
cudaError_t run_bwd(const NormArgs& a, int64_t blocks, float* dpost, float* dpre, cudaStream_t s) {
  auto k = norm_bwd_kernel<T, V, NV, G, NT, ODD, PRE>;
  constexpr size_t rows = Rows<T, V, NV, G, NT, ODD, PRE ? 5 : 3, PRE>::kBytes;
  constexpr size_t sums = NT / G > 1 ? sizeof(float) * NT * NV * V : 0;
  constexpr size_t smem = rows > sums ? rows : sums;
  static PerDevice kept;
  int64_t fit = 0;
  const cudaError_t e =
      kept.get(&fit, [&](int dev, int64_t* n) { return resident(k, NT, smem, kMaxCtas, dev, n); });
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(blocks < fit ? blocks : fit);
  k<<<grid, NT, smem, s>>>(a);
  if (a.part)
    norm_weight_kernel<<<dim3((a.width + 31) / 32, 2), dim3(32, 32), 0, s>>>(a.part, grid, a.width, dpost, dpre);
  return cudaGetLastError();
}

template <typename T, int V, int NV, int G, int NT, bool ODD>
cudaError_t run_fwd(const NormArgs& a, int64_t blocks, cudaStream_t s) {
  auto k = norm_fwd_kernel<T, V, NV, G, NT, ODD>;
  constexpr size_t smem = Rows<T, V, NV, G, NT, ODD, 3, false>::kBytes;
  static PerDevice kept;
  int64_t fit = 0;
  const cudaError_t e = kept.get(&fit, [&](int dev, int64_t* n) { return resident(k, NT, smem, 1 << 30, dev, n); });
  if (e != cudaSuccess) return e;
  k<<<static_cast<int>(blocks < fit ? blocks : fit), NT, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int V, int NV, int G, int NT, bool ODD>
kda_status run(const NormArgs& a, bool bwd, float* dpost, float* dpre, cudaStream_t s) {
  const int64_t blocks = ceil_div(a.rows, NT / G);
  const cudaError_t e = !bwd  ? run_fwd<T, V, NV, G, NT, ODD>(a, blocks, s)
                        : a.dn ? run_bwd<T, V, NV, G, NT, ODD, true>(a, blocks, dpost, dpre, s)
                               : run_bwd<T, V, NV, G, NT, ODD, false>(a, blocks, dpost, dpre, s);
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "block norm launch failed: %s", cudaGetErrorString(e));
}

// The smallest group that holds a row (with the elements before its start, where they may be any number).
template <typename T, int V, bool ODD>
kda_status dispatch(const NormArgs& a, bool bwd, float* dpost, float* dpre, cudaStream_t s) {
  const int vecs = (a.width + (ODD ? V - 1 : 0) + V - 1) / V;
  if (vecs <= 8) return run<T, V, 1, 8, 256, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 16) return run<T, V, 1, 16, 256, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 32) return run<T, V, 1, 32, 256, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 64) return run<T, V, 1, 64, 64, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 128) return run<T, V, 1, 128, 128, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 256) return run<T, V, 1, 256, 256, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 512) return run<T, V, 1, 512, 512, ODD>(a, bwd, dpost, dpre, s);
  if (vecs <= 1024) return run<T, V, 2, 512, 512, ODD>(a, bwd, dpost, dpre, s);
  if constexpr (V == 4) {
    if (vecs <= 2048) return run<T, V, 4, 512, 512, ODD>(a, bwd, dpost, dpre, s);
  }
  // widths from 8186 (fp32: 8190), whose first elements need one vector more
  if constexpr (ODD) return run<T, V, V == 4 ? 5 : 3, 512, 512, ODD>(a, bwd, dpost, dpre, s);
  return set_error(KDA_ERR_UNSUPPORTED, "width %d", a.width);
}

kda_status launch_norm(const kda_norm_problem* p, const NormArgs& a, bool bwd, float* dpost, float* dpre,
                       cudaStream_t s) {
  if (p->dtype == KDA_DTYPE_BF16)
    return p->width % 8 == 0 ? dispatch<__nv_bfloat16, 8, false>(a, bwd, dpost, dpre, s)
                             : dispatch<__nv_bfloat16, 8, true>(a, bwd, dpost, dpre, s);
  return p->width % 4 == 0 ? dispatch<float, 4, false>(a, bwd, dpost, dpre, s)
                           : dispatch<float, 4, true>(a, bwd, dpost, dpre, s);
}

kda_status validate_norm(const kda_norm_problem* p) {
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != KDA_DTYPE_BF16 && p->dtype != KDA_DTYPE_F32)
    return set_error(KDA_ERR_UNSUPPORTED, "dtype %d is not supported", p->dtype);
  if (p->width < 1 || p->width > kMaxWidth)
    return set_error(KDA_ERR_UNSUPPORTED, "width %d is not supported (1 to %d)", p->width, kMaxWidth);
  if (p->rows < 0 || p->rows > ((int64_t)1 << 45) / p->width)
    return set_error(KDA_ERR_INVALID_ARG, "rows %lld out of range", (long long)p->rows);
  if (!isfinite(p->residual_scale) || !isfinite(p->block_scale))
    return set_error(KDA_ERR_INVALID_ARG, "the scales must be finite");
  if (!(p->eps >= 0.f) || !isfinite(p->eps)) return set_error(KDA_ERR_INVALID_ARG, "eps must be >= 0");
  return KDA_OK;
}

kda_status need(const char* name, const void* p, bool wanted) {
  if (wanted && !p) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!wanted && p) return set_error(KDA_ERR_INVALID_ARG, "%s is given without the tensor it belongs to", name);
  if ((uintptr_t)p & 15u) return set_error(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return KDA_OK;
}
kda_status optional(const char* name, const void* p) { return need(name, p, p != nullptr); }

#define NORM_TRY(x)                   \
  do {                                \
    const kda_status st_ = (x);       \
    if (st_ != KDA_OK) return st_;    \
  } while (0)

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_block_norm_fwd(const kda_norm_problem* p, const void* y, const void* z, const void* h,
                              const float* w_post, const float* w_pre, void* h_out, void* n, void* stream) {
  using namespace kda;
  NORM_TRY(validate_norm(p));
  if (p->rows == 0) return KDA_OK;
  NORM_TRY(need("y", y, true));
  NORM_TRY(optional("z", z));
  NORM_TRY(optional("h", h));
  NORM_TRY(optional("w_post", w_post));
  NORM_TRY(optional("w_pre", w_pre));
  NORM_TRY(need("h_out", h_out, true));
  NORM_TRY(need("n", n, w_pre != nullptr));
  NormArgs a{};
  a.y = y; a.z = z; a.h = h; a.wpost = w_post; a.wpre = w_pre; a.ho = h_out; a.n = n;
  a.rows = p->rows; a.width = p->width; a.a = p->residual_scale; a.b = p->block_scale; a.eps = p->eps;
  return launch_norm(p, a, false, nullptr, nullptr, (cudaStream_t)stream);
}

size_t kda_block_norm_workspace_bytes(const kda_norm_problem* p, int32_t has_w_post, int32_t has_w_pre) {
  if (kda::validate_norm(p) != KDA_OK || !(has_w_post || has_w_pre)) return 0;
  const int64_t ctas = p->rows < kda::kMaxCtas ? (p->rows < 1 ? 1 : p->rows) : kda::kMaxCtas;
  return sizeof(float) * 2 * (size_t)ctas * (size_t)p->width;
}

kda_status kda_block_norm_bwd(const kda_norm_problem* p, const void* y, const void* z, const void* h,
                              const float* w_post, const float* w_pre, const void* dh_out, const void* dn, void* dy,
                              void* dz, void* dh, float* dw_post, float* dw_pre, void* workspace, void* stream) {
  using namespace kda;
  NORM_TRY(validate_norm(p));
  NORM_TRY(optional("w_post", w_post));
  NORM_TRY(optional("w_pre", w_pre));
  NORM_TRY(need("dw_post", dw_post, w_post != nullptr));
  NORM_TRY(need("dw_pre", dw_pre, w_pre != nullptr));
  cudaStream_t s = (cudaStream_t)stream;
  if (p->rows == 0) {
    for (float* g : {dw_post, dw_pre})
      if (g && cudaMemsetAsync(g, 0, sizeof(float) * p->width, s) != cudaSuccess)
        return set_error(KDA_ERR_CUDA, "memset failed: %s", cudaGetErrorString(cudaGetLastError()));
    return KDA_OK;
  }
  NORM_TRY(need("y", y, true));
  NORM_TRY(optional("z", z));
  NORM_TRY(optional("h", h));
  NORM_TRY(optional("dh_out", dh_out));
  if (dn && !w_pre) return set_error(KDA_ERR_INVALID_ARG, "dn is given without w_pre");
  NORM_TRY(optional("dn", dn));
  NORM_TRY(need("dy", dy, true));
  NORM_TRY(need("dz", dz, z != nullptr));
  NORM_TRY(need("dh", dh, h != nullptr));
  const bool weights = w_post != nullptr || w_pre != nullptr;  // without them a workspace is not used
  if (weights) NORM_TRY(need("workspace", workspace, true));
  NormArgs a{};
  a.y = y; a.z = z; a.h = h; a.wpost = w_post; a.wpre = w_pre; a.dho = dh_out; a.dn = dn;
  a.dy = dy; a.dz = dz; a.dh = dh; a.part = weights ? (float*)workspace : nullptr;
  a.rows = p->rows; a.width = p->width; a.a = p->residual_scale; a.b = p->block_scale; a.eps = p->eps;
  return launch_norm(p, a, true, dw_post, dw_pre, s);
}

}  // extern "C"
