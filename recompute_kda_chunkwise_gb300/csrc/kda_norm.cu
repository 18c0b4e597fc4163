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
// Bound: HBM; each tensor is read or written once. A row stays in registers
// between its reductions. A group of kGroup threads takes a row; a thread
// holds kVecs vectors of kVec elements (16 bytes where width and dtype allow,
// one element otherwise: rows of an odd width start unaligned).
//
// x - xn mean(x xn) takes x's part along the row out. In a row of one element
// that is all of x but the share eps r^2 that eps keeps, far below the
// rounding of the two terms: width 1 multiplies by that share instead.
#include <math.h>

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
struct Raw {
  T x[V];
};
template <>
struct alignas(16) Raw<__nv_bfloat16, 8> {
  uint4 u;
};
template <>
struct alignas(16) Raw<float, 4> {
  float4 u;
};
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = ldf(&r.x[i]);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 8>& r, float (&x)[8]) {
  const uint32_t u[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float (&x)[4]) {
  x[0] = r.u.x; x[1] = r.u.y; x[2] = r.u.z; x[3] = r.u.w;
}
template <typename T, int V>
__device__ __forceinline__ void put(T* p, const float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) stf(p + i, x[i]);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void put(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <int V>
__device__ __forceinline__ void weights(const float* w, int c, int width, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = (w && c < width) ? w[c + i] : 1.f;
}

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
      float t = lane < W ? s[i * 32 + lane] : 0.f;
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) t += __shfl_xor_sync(~0u, t, m);
      x[i] = t;
    }
  }
}

template <typename T, int V, int NV, int G, int NT>
__global__ void __launch_bounds__(NT) norm_fwd_kernel(const NormArgs a) {
  constexpr int kGroups = NT / G;
  __shared__ float sh[2 * 3 * 32];
  int turn = 0;
  const int lane = static_cast<int>(threadIdx.x) % G;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / G;
  const float inv = 1.f / static_cast<float>(a.width);
  // every group of a CTA makes the same number of turns (the reductions are collective)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups; r0 < a.rows;
       r0 += static_cast<int64_t>(gridDim.x) * kGroups) {
    const int64_t row = r0 + (first - static_cast<int64_t>(blockIdx.x) * kGroups);
    const bool live = row < a.rows;
    const int64_t base = row * a.width;
    Raw<T, V> ry[NV], rz[NV], rh[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + lane) * V;
      if (live && c < a.width) {
        ry[j] = *reinterpret_cast<const Raw<T, V>*>(static_cast<const T*>(a.y) + base + c);
        if (a.z) rz[j] = *reinterpret_cast<const Raw<T, V>*>(static_cast<const T*>(a.z) + base + c);
        if (a.h) rh[j] = *reinterpret_cast<const Raw<T, V>*>(static_cast<const T*>(a.h) + base + c);
      }
    }
    float x[NV][V], sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = live && (j * G + lane) * V < a.width;
      if (in) unpack(ry[j], x[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!in) x[j][i] = 0.f;
        sum[0] += x[j][i] * x[j][i];
      }
    }
    group_sum<G>(sum, sh, turn);
    const float scale = rsqrtf(sum[0] * inv + a.eps) * a.b;
    sum[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + lane) * V;
      if (live && c < a.width) {
        float w[V], t[V];
        weights(a.wpost, c, a.width, w);
#pragma unroll
        for (int i = 0; i < V; ++i) x[j][i] *= scale * w[i];
        if (a.z) {
          unpack(rz[j], t);
#pragma unroll
          for (int i = 0; i < V; ++i) x[j][i] *= sigmoidf_(t[i]);
        }
        if (a.h) {
          unpack(rh[j], t);
#pragma unroll
          for (int i = 0; i < V; ++i) x[j][i] = fmaf(a.a, t[i], x[j][i]);
        }
        put(static_cast<T*>(a.ho) + base + c, x[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += x[j][i] * x[j][i];
      }
    }
    if (a.n) {
      group_sum<G>(sum, sh, turn);
      const float r = rsqrtf(sum[0] * inv + a.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * G + lane) * V;
        if (live && c < a.width) {
          float w[V];
          weights(a.wpre, c, a.width, w);
#pragma unroll
          for (int i = 0; i < V; ++i) x[j][i] *= r * w[i];
          put(static_cast<T*>(a.n) + base + c, x[j]);
        }
      }
    }
  }
}

template <typename T, int V, int NV, int G, int NT>
__global__ void __launch_bounds__(NT) norm_bwd_kernel(const NormArgs a) {
  constexpr int kGroups = NT / G;
  __shared__ float sh[2 * 3 * 32];
  int turn = 0;
  const int lane = static_cast<int>(threadIdx.x) % G, group = static_cast<int>(threadIdx.x) / G;
  const float inv = 1.f / static_cast<float>(a.width);
  float gpost[NV][V], gpre[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) gpost[j][i] = gpre[j][i] = 0.f;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups; r0 < a.rows;
       r0 += static_cast<int64_t>(gridDim.x) * kGroups) {
    const int64_t row = r0 + group;
    const bool live = row < a.rows;
    const int64_t base = row * a.width;
    Raw<T, V> ry[NV], rz[NV], rh[NV], ro[NV], rn[NV];
    auto load = [&](const void* p, int c) {
      return *reinterpret_cast<const Raw<T, V>*>(static_cast<const T*>(p) + base + c);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + lane) * V;
      if (live && c < a.width) {
        ry[j] = load(a.y, c);
        if (a.z) rz[j] = load(a.z, c);
        if (a.h) rh[j] = load(a.h, c);
        if (a.dho) ro[j] = load(a.dho, c);
        if (a.dn) rn[j] = load(a.dn, c);
      }
    }
    float s1[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (live && (j * G + lane) * V < a.width) {
        float y[V];
        unpack(ry[j], y);
#pragma unroll
        for (int i = 0; i < V; ++i) s1[0] += y[i] * y[i];
      }
    group_sum<G>(s1, sh, turn);
    const float iy = rsqrtf(s1[0] * inv + a.eps);
    float ih = 0.f, proj = 0.f;
    auto hidden = [&](int j, int c, float (&hp)[V]) {  // h' of this thread's vector j
      float t[V], w[V];
      unpack(ry[j], hp);
      weights(a.wpost, c, a.width, w);
#pragma unroll
      for (int i = 0; i < V; ++i) hp[i] *= iy * a.b * w[i];
      if (a.z) {
        unpack(rz[j], t);
#pragma unroll
        for (int i = 0; i < V; ++i) hp[i] *= sigmoidf_(t[i]);
      }
      if (a.h) {
        unpack(rh[j], t);
#pragma unroll
        for (int i = 0; i < V; ++i) hp[i] = fmaf(a.a, t[i], hp[i]);
      }
    };
    if (a.dn) {
      float s2[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * G + lane) * V;
        if (live && c < a.width) {
          float hp[V], d[V], w[V];
          hidden(j, c, hp);
          unpack(rn[j], d);
          weights(a.wpre, c, a.width, w);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            s2[0] += hp[i] * hp[i];
            s2[1] += hp[i] * d[i] * w[i];
          }
        }
      }
      group_sum<G>(s2, sh, turn);
      ih = rsqrtf(s2[0] * inv + a.eps);
      proj = s2[1] * inv * ih * ih;  // mean(d hn) rh
    }
    float s3[1] = {0.f};
    float q[NV][V];  // du, the gradient of u, until dy is formed
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + lane) * V;
      if (live && c < a.width) {
        float D[V], y[V], w[V];
        if (a.dho)
          unpack(ro[j], D);
        else
#pragma unroll
          for (int i = 0; i < V; ++i) D[i] = 0.f;
        if (a.dn) {
          float hp[V], d[V];
          hidden(j, c, hp);
          unpack(rn[j], d);
          weights(a.wpre, c, a.width, w);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            gpre[j][i] += d[i] * hp[i] * ih;
            const float dw = d[i] * w[i];
            D[i] += ih * (a.width == 1 ? dw * (a.eps * ih * ih) : dw - hp[i] * proj);
          }
        }
        if (a.dh) {
          float t[V];
#pragma unroll
          for (int i = 0; i < V; ++i) t[i] = a.a * D[i];
          put(static_cast<T*>(a.dh) + base + c, t);
        }
        unpack(ry[j], y);
        weights(a.wpost, c, a.width, w);
        if (a.z) {
          float z[V], t[V];
          unpack(rz[j], z);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float sg = sigmoidf_(z[i]), du = a.b * D[i];
            t[i] = du * (y[i] * iy) * w[i] * (sg * sigmoidf_(-z[i]));
            q[j][i] = du * sg;
          }
          put(static_cast<T*>(a.dz) + base + c, t);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) q[j][i] = a.b * D[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          gpost[j][i] += q[j][i] * (y[i] * iy);
          q[j][i] *= w[i];
          s3[0] += q[j][i] * (y[i] * iy);
        }
      }
    }
    group_sum<G>(s3, sh, turn);
    const float m = s3[0] * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + lane) * V;
      if (live && c < a.width) {
        float y[V];
        unpack(ry[j], y);
#pragma unroll
        for (int i = 0; i < V; ++i) q[j][i] = iy * (a.width == 1 ? q[j][i] * (a.eps * iy * iy) : q[j][i] - (y[i] * iy) * m);
        put(static_cast<T*>(a.dy) + base + c, q[j]);
      }
    }
  }
  // This CTA's share of the weight gradients: its groups' sums, in order.
  if (!a.part) return;
  extern __shared__ float acc[];  // [groups][G * NV * V], only where a CTA has several groups
  const int64_t half = static_cast<int64_t>(gridDim.x) * a.width;
  float* const out = a.part + static_cast<int64_t>(blockIdx.x) * a.width;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.wpost : a.wpre) == nullptr) continue;
    if constexpr (kGroups == 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = (j * G + lane) * V + i;
          if (c < a.width) out[which * half + c] = which == 0 ? gpost[j][i] : gpre[j][i];
        }
    } else {
      constexpr int W = G * NV * V;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          acc[group * W + (j * G + lane) * V + i] = which == 0 ? gpost[j][i] : gpre[j][i];
      __syncthreads();
      for (int c = static_cast<int>(threadIdx.x); c < a.width; c += NT) {
        float t = 0.f;
        for (int g = 0; g < kGroups; ++g) t += acc[g * W + c];
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

// CTAs of a launch: what the SMs hold at once (the loop takes the rest).
template <typename K>
int grid_of(K kernel, int threads, size_t smem, int64_t blocks, int most) {
  int dev = 0, sms = 0, per = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  const int64_t fit = static_cast<int64_t>(sms) * (per < 1 ? 1 : per);
  return static_cast<int>(blocks < fit ? blocks : (fit < most ? fit : most));
}

template <typename T, int V, int NV, int G, int NT>
kda_status run(const NormArgs& a, bool bwd, float* dpost, float* dpre, cudaStream_t s) {
  const int64_t blocks = ceil_div(a.rows, NT / G);
  if (!bwd) {
    auto k = norm_fwd_kernel<T, V, NV, G, NT>;
    k<<<grid_of(k, NT, 0, blocks, 1 << 30), NT, 0, s>>>(a);
  } else {
    auto k = norm_bwd_kernel<T, V, NV, G, NT>;
    const size_t smem = NT / G > 1 && a.part ? sizeof(float) * NT * NV * V : 0;
    const int grid = grid_of(k, NT, smem, blocks, kMaxCtas);
    k<<<grid, NT, smem, s>>>(a);
    if (a.part)
      norm_weight_kernel<<<dim3((a.width + 31) / 32, 2), dim3(32, 32), 0, s>>>(a.part, grid, a.width, dpost, dpre);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "block norm launch failed: %s", cudaGetErrorString(e));
}

// The smallest group that holds a row.
template <typename T, int V>
kda_status dispatch(const NormArgs& a, bool bwd, float* dpost, float* dpre, cudaStream_t s) {
  const int vecs = (a.width + V - 1) / V;
  if (vecs <= 8) return run<T, V, 1, 8, 256>(a, bwd, dpost, dpre, s);
  if (vecs <= 16) return run<T, V, 1, 16, 256>(a, bwd, dpost, dpre, s);
  if (vecs <= 32) return run<T, V, 1, 32, 256>(a, bwd, dpost, dpre, s);
  if (vecs <= 64) return run<T, V, 1, 64, 64>(a, bwd, dpost, dpre, s);
  if (vecs <= 128) return run<T, V, 1, 128, 128>(a, bwd, dpost, dpre, s);
  if (vecs <= 256) return run<T, V, 1, 256, 256>(a, bwd, dpost, dpre, s);
  if (vecs <= 512) return run<T, V, 1, 512, 512>(a, bwd, dpost, dpre, s);
  if (vecs <= 1024) return run<T, V, 2, 512, 512>(a, bwd, dpost, dpre, s);
  if constexpr (V <= 4) {
    if (vecs <= 2048) return run<T, V, 4, 512, 512>(a, bwd, dpost, dpre, s);
  }
  if constexpr (V == 1) {
    if (vecs <= 4096) return run<T, V, 8, 512, 512>(a, bwd, dpost, dpre, s);
    return run<T, V, 16, 512, 512>(a, bwd, dpost, dpre, s);
  }
  return set_error(KDA_ERR_UNSUPPORTED, "width %d", a.width);
}

kda_status launch_norm(const kda_norm_problem* p, const NormArgs& a, bool bwd, float* dpost, float* dpre,
                       cudaStream_t s) {
  if (p->dtype == KDA_DTYPE_BF16)
    return p->width % 8 == 0 ? dispatch<__nv_bfloat16, 8>(a, bwd, dpost, dpre, s)
                             : dispatch<__nv_bfloat16, 1>(a, bwd, dpost, dpre, s);
  return p->width % 4 == 0 ? dispatch<float, 4>(a, bwd, dpost, dpre, s) : dispatch<float, 1>(a, bwd, dpost, dpre, s);
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
  NORM_TRY(need("workspace", workspace, w_post != nullptr || w_pre != nullptr));
  NormArgs a{};
  a.y = y; a.z = z; a.h = h; a.wpost = w_post; a.wpre = w_pre; a.dho = dh_out; a.dn = dn;
  a.dy = dy; a.dz = dz; a.dh = dh; a.part = (float*)workspace;
  a.rows = p->rows; a.width = p->width; a.a = p->residual_scale; a.b = p->block_scale; a.eps = p->eps;
  return launch_norm(p, a, true, dw_post, dw_pre, s);
}

}  // extern "C"
