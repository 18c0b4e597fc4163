// kda_clip.cu -- the global norm of many gradients, and clipping by it:
// kda_grad_norm / kda_clip_grads of kda_blocks.h.
//
//   norm = sqrt(sum g^2),   out = g min(1, max_norm / norm)
//
// Two launches over all tensors, however many: the tensors' addresses and
// sizes are parameters of the launch (up to 1000 of them; above that, one
// launch for every 1000), so there is no table to copy first and a captured
// graph holds its own. The tensors are cut into chunks of 16 KB, and each CTA
// takes every grid-th chunk: the sum of squares of each CTA's chunks
// goes to the workspace in fp64. The second launch's CTAs each add those sums
// up, in the same order, and scale their chunks, last ones first, while part
// of what was read last is still in L2.
//
// Range. A thread's 32 elements of a chunk (16 in fp32) are squared and summed in
// fp32, and where that sum is outside 2^-70 .. 2^100 again in fp64: inside, it has
// neither overflowed nor lost what matters beside its largest square. Sums above
// that are fp64: one addition for 32 elements is a sixth of what the SM's slow
// fp64 unit could do in the time that memory takes.
//
// Bound: HBM. The gradients are read twice where they do not fit L2.
#include <math.h>

#include "kda_blocks.h"
#include "kda_device.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 64 * kThreads;  // of a gradient: four 16-byte vectors a thread
constexpr int kCtasPerSm = 6;         // of the pass that only reads
constexpr int kScaleCtas = 3;         // of the one that writes: 948 us of both for 0.74e9 elements, bf16 into fp32; two 915, but
                                      // fp32 in place 1482 (three 1322), six 1103 and 1374
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

// Vector i (16 bytes) of a tensor, zeros past its end.
__device__ __forceinline__ uint4 load16(const Tensor& t, int64_t i, bool aligned) {
  const int per = t.bf16_in ? 8 : 4;
  const int64_t at = i * per;
  if (aligned && at + per <= t.n) return reinterpret_cast<const uint4*>(t.g)[i];
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (e >= per || at + e >= t.n) continue;
    if (t.bf16_in)
      w[e / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(t.g)[at + e]) << (16 * (e & 1));
    else
      w[e & 3] = static_cast<const uint32_t*>(t.g)[at + e];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight (four) values to elements at .. of the output.
template <int N>
__device__ __forceinline__ void store(const Tensor& t, int64_t at, bool aligned, const float (&x)[N]) {
  const bool whole = aligned && at + N <= t.n;
  if (t.bf16_out) {
    __nv_bfloat16* const p = static_cast<__nv_bfloat16*>(t.out) + at;
    if (whole) {
      uint32_t w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (N == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2 % (N / 2)], w[3 % (N / 2)]);
      else
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at + i < t.n) stf(p + i, x[i]);
    }
  } else {
    float* const p = static_cast<float*>(t.out) + at;
    if (whole) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
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
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kda_squares_kernel(const __grid_constant__ Table<N> tb, double* sums) {
  __shared__ double s[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x);
  before_kernel();
  double all = 0;
  for (int chunk = static_cast<int>(blockIdx.x); chunk < tb.first[tb.num]; chunk += static_cast<int>(gridDim.x)) {
    const int i = tensor_of(tb, chunk);
    const Tensor t = tb.t[i].get();
    const int64_t at = static_cast<int64_t>(chunk - tb.first[i]) * (4 * kThreads) + tid;
    const bool aligned = (reinterpret_cast<uintptr_t>(t.g) & 15) == 0;
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = load16(t, at + j * kThreads, aligned);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        any |= w[e];
        if (t.bf16_in) {
          sum[e] = fmaf(low(w[e]), low(w[e]), sum[e]);
          sum[e] = fmaf(high(w[e]), high(w[e]), sum[e]);
        } else {
          sum[e] = fmaf(__uint_as_float(w[e]), __uint_as_float(w[e]), sum[e]);
        }
      }
    }
    const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if (total > 0x1p-70f && total < 0x1p100f) {
      all += static_cast<double>(total);
    } else if (any & (t.bf16_in ? 0x7fff7fffu : 0x7fffffffu)) {  // out of fp32's range, or not finite; zeros of either sign add nothing
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const uint4 y = j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3];
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double u = t.bf16_in ? low(w[e]) : __uint_as_float(w[e]), v = t.bf16_in ? high(w[e]) : 0.f;
          all = fma(u, u, fma(v, v, all));
        }
      }
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
  after_kernel();
  const double n = norm_of(sums, num, s);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kScaleCtas) kda_scale_kernel(const __grid_constant__ Table<N> tb, const double* sums, int num,
                                                             double most, float* norm) {
  __shared__ double s[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x);
  after_kernel();
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
    const int64_t at = static_cast<int64_t>(chunk - tb.first[i]) * (4 * kThreads);  // 16-byte vectors of the gradient
    const bool aligned = ((reinterpret_cast<uintptr_t>(t.g) | reinterpret_cast<uintptr_t>(t.out)) & 15) == 0;
    if (t.bf16_in && !t.bf16_out && aligned && (at + 4 * kThreads) * 8 <= t.n) {
      // bf16 into fp32: four elements at a time, so that a warp's stores are whole lines
      uint2 x[8];
      const uint2* const src = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(t.g) + at * 8) + tid;
      float4* const dst = reinterpret_cast<float4*>(static_cast<float*>(t.out) + at * 8) + tid;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = src[j * kThreads];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dst[j * kThreads] = make_float4(low(x[j].x) * f1 * f2, high(x[j].x) * f1 * f2, low(x[j].y) * f1 * f2,
                                        high(x[j].y) * f1 * f2);
      continue;
    }
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = load16(t, at + tid + j * kThreads, aligned);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      const int64_t to = at + tid + j * kThreads;
      if (t.bf16_in) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = low(w[e]) * f1 * f2;
          y[2 * e + 1] = high(w[e]) * f1 * f2;
        }
        store(t, to * 8, aligned, y);
      } else {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __uint_as_float(w[e]) * f1 * f2;
        store(t, to * 4, aligned, y);
      }
    }
  }
}

int grid_of(int64_t chunks, int64_t sms, int per_sm) {
  const int64_t most = sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
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
    const int64_t per = kChunkBytes / (in ? 2 : 4);
    chunks += (sizes[j] + per - 1) / per;
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
    const int grid = grid_of(tb.first[tb.num], c.sms, kCtasPerSm);
    kda_squares_kernel<N><<<grid, kThreads, 0, c.s>>>(tb, c.sums + sums);
    sums += grid;
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && !c.outs)
    e = launch_after(kda_norm_of_sums_kernel, 1, kThreads, 0, c.s, static_cast<const double*>(c.sums), sums, c.norm);
  for (int i0 = c.num <= N ? 0 : (c.num - 1) / N * N; e == cudaSuccess && c.outs && i0 >= 0; i0 -= N) {  // last ones first
    fill(tb, i0, c.num - i0 < N ? c.num - i0 : N, c.g, c.sizes, c.dtypes, c.outs, c.out_dtypes);
    e = launch_after(kda_scale_kernel<N>, grid_of(tb.first[tb.num], c.sms, kScaleCtas), kThreads, 0, c.s, tb,
                     static_cast<const double*>(c.sums), sums, c.most, i0 == 0 ? c.norm : nullptr);
  }
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
