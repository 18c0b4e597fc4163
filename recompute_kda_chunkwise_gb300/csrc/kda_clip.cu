// kda_clip.cu -- the global norm of many gradients, and clipping by it:
// kda_grad_norm / kda_clip_grads of kda_blocks.h.
//
//   norm = sqrt(sum g^2),   out = g min(1, max_norm / norm)
//
// Two launches over all tensors, however many: the tensors' addresses and
// sizes are parameters of the launch (up to 1000 of them; above that, one
// launch for every 1000), so there is no table to copy first and a captured
// graph holds its own. The tensors are cut into chunks of 8192 elements, and
// each CTA takes every grid-th chunk: the sum of squares of each CTA's chunks
// goes to the workspace in fp64. The second launch's CTAs each add those sums
// up, in the same order, and scale their chunks, last ones first, while part
// of what was read last is still in L2.
//
// Range. 32 elements of a thread are squared and summed in fp32 where the
// largest of them is between 2^-40 and 2^40 (their sum then neither overflows
// nor loses what matters beside the largest), else in fp64; sums above 32
// elements are fp64. One fp64 addition for 32 elements is a sixth of what the
// SM's slow fp64 unit could do in the time that memory takes.
//
// Bound: HBM. The gradients are read twice where they do not fit L2.
#include <math.h>

#include "kda_blocks.h"
#include "kda_device.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32 * kThreads;  // elements
constexpr int kMaxCtas = 1024;
constexpr int kTable = 1000;           // tensors of a launch

struct Tensor {
  const void* g;
  void* out;
  int64_t n;
  bool bf16_in, bf16_out;
};
// A tensor as the launch carries it: 1000 of them fit the 32764 bytes that parameters may take.
struct Packed {
  const void* g;
  void* out;
  uint64_t n_types;  // 4 * elements + 2 * bf16_out + bf16_in
  __device__ __forceinline__ Tensor get() const {
    return {g, out, static_cast<int64_t>(n_types >> 2), (n_types & 1) != 0, (n_types & 2) != 0};
  }
};
template <int N>
struct Table {
  Packed t[N];
  int32_t first[N + 1];  // first chunk of each tensor
  int32_t num;
};

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& tb, int chunk) {
  int lo = 0, hi = tb.num - 1;  // the last tensor whose first chunk is not past this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tb.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void widen(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Elements [at, at + 8) of a tensor, zeros past its end; `whole`: all eight are there and aligned.
__device__ __forceinline__ void load8(const Tensor& t, int64_t at, bool whole, float (&x)[8]) {
  if (t.bf16_in) {
    const __nv_bfloat16* const p = static_cast<const __nv_bfloat16*>(t.g) + at;
    if (whole) {
      widen(*reinterpret_cast<const uint4*>(p), x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = at + i < t.n ? ldf(p + i) : 0.f;
    }
  } else {
    const float* const p = static_cast<const float*>(t.g) + at;
    if (whole) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = at + i < t.n ? p[i] : 0.f;
    }
  }
}
__device__ __forceinline__ void store8(const Tensor& t, int64_t at, bool whole, const float (&x)[8]) {
  if (t.bf16_out) {
    __nv_bfloat16* const p = static_cast<__nv_bfloat16*>(t.out) + at;
    if (whole) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < t.n) stf(p + i, x[i]);
    }
  } else {
    float* const p = static_cast<float*>(t.out) + at;
    if (whole) {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < t.n) p[i] = x[i];
    }
  }
}

// Sum over the CTA's threads in a fixed order, at thread 0.
__device__ __forceinline__ double cta_sum(double x, double* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_down_sync(~0u, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kThreads / 32; ++i) x += s[i];
  return x;
}

template <int N>
__global__ void __launch_bounds__(kThreads) kda_squares_kernel(const __grid_constant__ Table<N> tb, double* sums) {
  __shared__ double s[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x);
  double all = 0;
  for (int chunk = static_cast<int>(blockIdx.x); chunk < tb.first[tb.num]; chunk += static_cast<int>(gridDim.x)) {
    const int i = tensor_of(tb, chunk);
    const Tensor t = tb.t[i].get();
    const int64_t at0 = static_cast<int64_t>(chunk - tb.first[i]) * kChunk + tid * 8;
    const bool aligned = (reinterpret_cast<uintptr_t>(t.g) & 15) == 0;
    float x[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = at0 + j * (8 * kThreads);
      load8(t, at, aligned && at + 8 <= t.n, x[j]);
    }
    float top = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        top = fmaxf(top, fabsf(x[j][c]));
        sum[c & 3] = fmaf(x[j][c], x[j][c], sum[c & 3]);
      }
    if (top == 0.f || (top > 0x1p-40f && top < 0x1p40f)) {  // a NaN is in the sum
      all += static_cast<double>((sum[0] + sum[1]) + (sum[2] + sum[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) all = fma(static_cast<double>(x[j][c]), static_cast<double>(x[j][c]), all);
    }
  }
  all = cta_sum(all, s);
  if (tid == 0) sums[blockIdx.x] = all;
}

// The norm from every CTA's sum, the same in each CTA that asks.
__device__ __forceinline__ double norm_of(const double* sums, int num, double* s) {
  double x = 0;
  for (int i = static_cast<int>(threadIdx.x); i < num; i += kThreads) x += sums[i];
  x = cta_sum(x, s);
  if (threadIdx.x == 0) s[0] = sqrt(x);
  __syncthreads();
  return s[0];
}

__global__ void __launch_bounds__(kThreads) kda_norm_of_sums_kernel(const double* sums, int num, float* norm) {
  __shared__ double s[kThreads / 32];
  const double n = norm_of(sums, num, s);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

template <int N>
__global__ void __launch_bounds__(kThreads) kda_scale_kernel(const __grid_constant__ Table<N> tb, const double* sums, int num,
                                                             double most, float* norm) {
  __shared__ double s[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x);
  const double n = norm_of(sums, num, s);
  if (norm && blockIdx.x == 0 && tid == 0) *norm = static_cast<float>(n);
  // what the caller sees as not finite (fp32) clips nothing
  const bool clip = n > most && isfinite(static_cast<float>(n));
  const double f = clip ? most / n : 1.0;
  // In two parts where the factor alone would lose digits in fp32's subnormals.
  const float f1 = f < 0x1p-100 ? 0x1p-100f : 1.f;
  const float f2 = static_cast<float>(f < 0x1p-100 ? f * 0x1p100 : f);
  const int chunks = tb.first[tb.num];
  for (int c = static_cast<int>(blockIdx.x); c < chunks; c += static_cast<int>(gridDim.x)) {
    const int chunk = chunks - 1 - c;
    const int i = tensor_of(tb, chunk);
    const Tensor t = tb.t[i].get();
    if (!clip && t.out == t.g) continue;
    const int64_t at0 = static_cast<int64_t>(chunk - tb.first[i]) * kChunk + tid * 8;
    const bool aligned = ((reinterpret_cast<uintptr_t>(t.g) | reinterpret_cast<uintptr_t>(t.out)) & 15) == 0;
    float x[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = at0 + j * (8 * kThreads);
      load8(t, at, aligned && at + 8 <= t.n, x[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = x[j][e] * f1 * f2;
      const int64_t at = at0 + j * (8 * kThreads);
      store8(t, at, aligned && at + 8 <= t.n, x[j]);
    }
  }
}

int grid_of(int64_t chunks, int64_t sms) {
  const int64_t most = sms * 4 < kMaxCtas ? sms * 4 : kMaxCtas;
  return static_cast<int>(chunks < 1 ? 1 : chunks < most ? chunks : most);
}

// Tensors [i0, i0 + num) of the call.
template <int N>
void fill(Table<N>& tb, int i0, int num, const void* const* g, const int64_t* sizes, const int32_t* dtypes, void* const* outs,
          const int32_t* out_dtypes) {
  int64_t chunks = 0;
  tb.num = num;
  for (int i = 0; i < num; ++i) {
    const int j = i0 + i;
    const uint64_t in = dtypes[j] == KDA_DTYPE_BF16, out = outs && out_dtypes[j] == KDA_DTYPE_BF16;
    tb.t[i] = {g[j], outs ? outs[j] : nullptr, 4 * static_cast<uint64_t>(sizes[j]) + 2 * out + in};
    tb.first[i] = static_cast<int32_t>(chunks);
    chunks += (sizes[j] + kChunk - 1) / kChunk;
  }
  tb.first[num] = static_cast<int32_t>(chunks);
}

struct Call {
  int num;
  const void* const* g;
  const int64_t* sizes;
  const int32_t* dtypes;
  void* const* outs;
  const int32_t* out_dtypes;
  double most;
  float* norm;
  double* sums;
  int64_t sms;
  cudaStream_t s;
};

// Both passes with tables of N tensors.
template <int N>
kda_status run(const Call& c) {
  Table<N> tb;
  int sums = 0;
  for (int i0 = 0; i0 == 0 || i0 < c.num; i0 += N) {
    fill(tb, i0, c.num - i0 < N ? c.num - i0 : N, c.g, c.sizes, c.dtypes, nullptr, nullptr);
    const int grid = grid_of(tb.first[tb.num], c.sms);
    kda_squares_kernel<N><<<grid, kThreads, 0, c.s>>>(tb, c.sums + sums);
    sums += grid;
  }
  if (!c.outs) {
    kda_norm_of_sums_kernel<<<1, kThreads, 0, c.s>>>(c.sums, sums, c.norm);
  } else {
    for (int i0 = c.num <= N ? 0 : (c.num - 1) / N * N; i0 >= 0; i0 -= N) {  // last ones first
      fill(tb, i0, c.num - i0 < N ? c.num - i0 : N, c.g, c.sizes, c.dtypes, c.outs, c.out_dtypes);
      kda_scale_kernel<N><<<grid_of(tb.first[tb.num], c.sms), kThreads, 0, c.s>>>(tb, c.sums, sums, c.most,
                                                                                  i0 == 0 ? c.norm : nullptr);
    }
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "gradient norm launch failed: %s", cudaGetErrorString(e));
}

kda_status call(Call c, void* workspace) {
  if (c.num < 0 || c.num > (1 << 20)) return set_error(KDA_ERR_INVALID_ARG, "num %d out of range", c.num);
  if (c.num && (!c.g || !c.sizes || !c.dtypes)) return set_error(KDA_ERR_INVALID_ARG, "grads, sizes or dtypes is NULL");
  constexpr int64_t kMost = (int64_t)1 << 42;  // elements of a call: chunks are counted in 32 bits
  int64_t all = 0;
  for (int i = 0; i < c.num; ++i) {
    if (c.sizes[i] < 0 || c.sizes[i] > kMost - all)
      return set_error(KDA_ERR_INVALID_ARG, "size %lld of tensor %d out of range", (long long)c.sizes[i], i);
    all += c.sizes[i];
    for (const int32_t* dt : {c.dtypes, c.out_dtypes})
      if (dt && dt[i] != KDA_DTYPE_BF16 && dt[i] != KDA_DTYPE_F32)
        return set_error(KDA_ERR_UNSUPPORTED, "dtype %d of tensor %d is not supported", dt[i], i);
    if (c.sizes[i] == 0) continue;
    if (!c.g[i] || (c.outs && !c.outs[i])) return set_error(KDA_ERR_INVALID_ARG, "tensor %d is NULL", i);
    if ((uintptr_t)c.g[i] % (c.dtypes[i] == KDA_DTYPE_BF16 ? 2 : 4) ||
        (c.outs && (uintptr_t)c.outs[i] % (c.out_dtypes[i] == KDA_DTYPE_BF16 ? 2 : 4)))
      return set_error(KDA_ERR_INVALID_ARG, "tensor %d is not aligned to its elements", i);
    if (c.outs && c.outs[i] == c.g[i] && c.out_dtypes[i] != c.dtypes[i])
      return set_error(KDA_ERR_INVALID_ARG, "tensor %d is clipped in place into another dtype", i);
  }
  if (!c.norm || (uintptr_t)c.norm & 3u) return set_error(KDA_ERR_INVALID_ARG, "norm must be 4-byte aligned and not NULL");
  if (!workspace || (uintptr_t)workspace & 15u)
    return set_error(KDA_ERR_INVALID_ARG, "workspace must be 16-byte aligned and not NULL");
  c.sums = static_cast<double*>(workspace);
  static PerDevice kept;
  const cudaError_t e = kept.get(&c.sms, [](int dev, int64_t* n) {
    int count = 0;
    const cudaError_t got = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
    *n = count;
    return got;
  });
  if (e != cudaSuccess) return set_error(KDA_ERR_CUDA, "gradient norm set-up failed: %s", cudaGetErrorString(e));
  // a launch carries its whole table: small calls carry a small one
  return c.num <= 32 ? run<32>(c) : c.num <= 120 ? run<120>(c) : run<kTable>(c);
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_grad_norm_workspace_bytes(int32_t num) {
  using namespace kda;
  return num < 0 ? 0 : sizeof(double) * kMaxCtas * (num <= kTable ? 1 : (num + kTable - 1) / kTable);
}

kda_status kda_grad_norm(int32_t num, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, float* norm,
                         void* workspace, void* stream) {
  return kda::call({num, grads, sizes, dtypes, nullptr, nullptr, 0, norm, nullptr, 0, (cudaStream_t)stream}, workspace);
}

kda_status kda_clip_grads(int32_t num, const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                          void* const* outs, const int32_t* out_dtypes, double max_norm, float* norm, void* workspace,
                          void* stream) {
  if (!(max_norm >= 0)) return kda::set_error(KDA_ERR_INVALID_ARG, "max_norm must not be negative or NaN");
  static void* const none[1] = {nullptr};
  static const int32_t none_dtype[1] = {KDA_DTYPE_F32};
  if (num > 0 && (!outs || !out_dtypes)) return kda::set_error(KDA_ERR_INVALID_ARG, "outs or out_dtypes is NULL");
  return kda::call({num, grads, sizes, dtypes, num > 0 ? outs : none, num > 0 ? out_dtypes : none_dtype, max_norm, norm,
                    nullptr, 0, (cudaStream_t)stream}, workspace);
}

}  // extern "C"
