// kda_rotary.cu -- rotary positions (kda_rotary of kda_blocks.h) and the paged
// append that rotates on the way (kda_paged_append_rotary).
//
//   (a, b) -> magnitude * (a cos x - b sin x, a sin x + b cos x),  x = position * frequency
//
// Angles. A frequency is held as turns per position in units of 2^-64 of a
// turn. The 64-bit product with a position, modulo 2^64, is the angle's
// fraction of a turn: whole turns drop out without a rounding, where an fp32
// product is off by 0.06 rad at position 10^6. Its upper 32 bits go to the
// nearest quarter turn, whose rest is exact in fp32 to 2^-34 of a turn.
//
// Bound: HBM, each element read and written once. 72 heads of 128 of 8192
// tokens in bf16 (151 MB each way), rotated and, for the gradient, rotated back:
// 105 us, 86% of the measured copy rate; in fp32 40 heads, 6.0 TB/s. Interleaved
// pairs, whose items are half as long: 54 us a pass, 84%. Pairs that no vector
// divides (21 of 128 channels) go element by element: 160 us.
//
// Split. A CTA takes a tile of tokens with all their heads. A token's sines
// and cosines are formed once, in shared memory, for all of its heads (each
// costs some 40 instructions: formed anew for every head they would take as
// long as the memory). Its threads take 16-byte vectors, both ends of eight
// (fp32: four) pairs each; the first loads are under way while the tile's
// positions are looked up and its angles formed, and each later one while the
// vectors before it are worked on. bf16 is bound by instructions as much as by
// memory: a thread keeps its place in the heads and its sines in registers, steps
// through heads without a division, and works on words of two values (171 us
// before). Five CTAs an SM hold that; pairs and single elements do better with
// eight.
#include <math.h>

#include "kda_blocks.h"
#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 32;          // tokens of a CTA, at most: one warp looks them up
constexpr int64_t kMaxStride = 1 << 25;  // elements from a token to the next
static_assert(kMaxStride * kMaxTile <= 1 << 30, "");
constexpr int kTableBytes = 32768;    // sines and cosines of a tile
constexpr int kTileVectors = 2048;    // 16-byte vectors of a CTA, about
constexpr int kMinCtas = 608;

struct RotaryArgs {
  const void *q, *k, *v;   // v: paged form only
  void *qo, *ko, *vo;      // ko, vo: the pages in the paged form
  int64_t qs, ks, vs;      // elements from a token to the next
  const int64_t* freqs;
  const int32_t *positions, *cu, *table, *lens;
  int* status;
  int64_t S, pages;
  int N, Hq, Hk, D, R, tile, page, width;
  float mag;
  int inverse;
};

// Number of sequences that end at or before token t, by a whole warp: every
// step looks at 32 places of what is left.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, int64_t t, int lane) {
  int base = 0, left = N;
  while (left > 0) {
    const int step = (left + 31) / 32, at = (lane + 1) * step;
    const bool before = at <= left && cu[base + at] <= t;
    const int n = __popc(__ballot_sync(~0u, before));
    base += n * step;
    left = min(step - 1, left - n * step);
  }
  return base;
}

// A 16-byte vector's pairs, turned in words: two bf16 values or one fp32 value each.
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void turn_pair(float& a, float& b, float2 w) {
  const float x = a;
  a = fmaf(x, w.x, -b * w.y);
  b = fmaf(x, w.y, b * w.x);
}
// a and b hold the first and second channels of the pairs of `w`.
template <bool BF16>
__device__ __forceinline__ void turn_halves(uint32_t& a, uint32_t& b, const float2* w) {
  if (BF16) {
    float a0 = __uint_as_float(a << 16), a1 = __uint_as_float(a & 0xffff0000u);
    float b0 = __uint_as_float(b << 16), b1 = __uint_as_float(b & 0xffff0000u);
    turn_pair(a0, b0, w[0]);
    turn_pair(a1, b1, w[1]);
    a = round2(a0, a1);
    b = round2(b0, b1);
  } else {
    float x = __uint_as_float(a), y = __uint_as_float(b);
    turn_pair(x, y, w[0]);
    a = __float_as_uint(x);
    b = __float_as_uint(y);
  }
}

// How a head's channels are cut into items of work.
enum Layout {
  kHalf,    // pairs (i, i + R/2), both halves whole vectors: an item is a vector of either, or one that passes
  kPairs,   // pairs (2i, 2i + 1): an item is a vector
  kSingle,  // pairs (i, i + R/2) that no vector divides: an item is a pair, or an element that passes
};

template <typename T, int LAYOUT, bool PAGED>
__global__ void __launch_bounds__(kThreads, LAYOUT == kHalf || sizeof(T) == 4 ? 5 : 8) kda_rotary_kernel(const RotaryArgs a) {
  constexpr int V = 16 / sizeof(T);
  constexpr bool kBf16 = sizeof(T) == 2;
  // Items of a thread that are loaded together, while as many more are worked on.
  constexpr int kBatch = LAYOUT == kSingle ? 4 : 1;
  extern __shared__ float2 turn[];  // [tile][R / 2]: magnitude * (cos, sin)
  __shared__ int32_t s_pos[kMaxTile];
  __shared__ int64_t s_row[kMaxTile];  // paged: elements before the token's row of the pages; negative: the token is skipped
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  const int nt = static_cast<int>(a.S - t0 < a.tile ? a.S - t0 : a.tile);
  const int half = a.R / 2;
  const int per_head = LAYOUT == kHalf ? half / V + (a.D - a.R) / V : LAYOUT == kPairs ? a.D / V : half + a.D - a.R;
  const int turned = a.Hq + a.Hk, heads = turned + (PAGED ? a.Hk : 0);  // the paged form's values are copied beside them

  // A thread keeps its place within the heads, and goes over the tokens' heads
  // `slots` at a time; places past one for each thread (long heads that are cut
  // into single elements) are taken in another round.
  const int slots = per_head < kThreads ? kThreads / per_head : 1;
  const int first = per_head < kThreads ? tid / per_head : 0;
  const int step_t = slots / heads, step_h = slots % heads;
  struct At {
    int t, h;
  };
  auto advance = [&](At& x) {
    x.t += step_t;
    x.h += step_h;
    if (x.h >= heads) {
      x.h -= heads;
      ++x.t;
    }
  };
  int c = per_head < kThreads ? tid - first * per_head : tid;
  int off, pair;  // the place's first channel; its first pair, -1: it passes
  auto place = [&]() {
    if (LAYOUT == kHalf) {
      const bool pass = c >= half / V;
      off = pass ? a.R + (c - half / V) * V : c * V;
      pair = pass ? -1 : off;
    } else if (LAYOUT == kPairs) {
      off = c * V;
      pair = off < a.R ? off / 2 : -1;
    } else {
      off = c < half ? c : half + c;
      pair = c < half ? c : -1;
    }
  };
  // within a CTA's tile offsets fit 32 bits (kMaxStride)
  const T* const q = static_cast<const T*>(a.q) + t0 * a.qs;
  const T* const k = static_cast<const T*>(a.k) + t0 * a.ks;
  const T* const v = static_cast<const T*>(a.v) + t0 * a.vs;
  T* const qo = static_cast<T*>(a.qo) + t0 * a.Hq * a.D;
  T* const ko = static_cast<T*>(a.ko) + (PAGED ? 0 : t0 * a.Hk * a.D);
  T* const vo = static_cast<T*>(a.vo);
  const int qs = static_cast<int>(a.qs), ks = static_cast<int>(a.ks), vs = static_cast<int>(a.vs);
  auto source = [&](const At& x) {
    if (x.h < a.Hq) return q + (x.t * qs + x.h * a.D + off);
    if (!PAGED || x.h < turned) return k + (x.t * ks + (x.h - a.Hq) * a.D + off);
    return v + (x.t * vs + (x.h - turned) * a.D + off);
  };
  auto target = [&](const At& x) {
    if (x.h < a.Hq) return qo + ((x.t * a.Hq + x.h) * a.D + off);
    const int h = x.h - (!PAGED || x.h < turned ? a.Hq : turned);
    if (!PAGED) return ko + ((x.t * a.Hk + h) * a.D + off);
    return (x.h < turned ? ko : vo) + s_row[x.t] + (h * a.D + off);
  };
  struct Batch {
    uint4 a[kBatch], b[kBatch];
  };
  auto load = [&](Batch& r, At& x) {  // from x on, which moves past them
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (x.t < nt) {
        const T* const src = source(x);
        if (LAYOUT == kSingle) {
          r.a[u].x = kBf16 ? *reinterpret_cast<const uint16_t*>(src) : *reinterpret_cast<const uint32_t*>(src);
          if (pair >= 0)
            r.b[u].x = kBf16 ? *reinterpret_cast<const uint16_t*>(src + half) : *reinterpret_cast<const uint32_t*>(src + half);
        } else {
          r.a[u] = *reinterpret_cast<const uint4*>(src);
          if (LAYOUT == kHalf && pair >= 0) r.b[u] = *reinterpret_cast<const uint4*>(src + half);
        }
      }
      advance(x);
    }
  };
  // Sines and cosines of this place's pairs for token `held`: read from shared
  // memory once a token, since lanes 64 bytes apart fall on few banks.
  constexpr int kPairsOf = LAYOUT == kHalf ? V : LAYOUT == kPairs ? V / 2 : 1;
  float2 w[LAYOUT == kSingle ? 2 : kPairsOf] = {};
  int held = -1;
  auto finish = [&](Batch& r, At& x) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (x.t < nt && s_row[x.t] >= 0) {
        T* const dst = target(x);
        const bool turns = pair >= 0 && (!PAGED || x.h < turned);
        if (turns && x.t != held) {
          held = x.t;
          const float2* const from = turn + x.t * half + pair;
#pragma unroll
          for (int j = 0; j < kPairsOf; ++j)
            if (LAYOUT != kPairs || pair + j < half) w[j] = from[j];
        }
        if constexpr (LAYOUT == kSingle) {
          if (turns) turn_halves<kBf16>(r.a[u].x, r.b[u].x, w);  // bf16: the upper halves are not used
          if (kBf16) {
            *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(r.a[u].x);
            if (pair >= 0) *reinterpret_cast<uint16_t*>(dst + half) = static_cast<uint16_t>(r.b[u].x);
          } else {
            *reinterpret_cast<uint32_t*>(dst) = r.a[u].x;
            if (pair >= 0) *reinterpret_cast<uint32_t*>(dst + half) = r.b[u].x;
          }
        } else if constexpr (LAYOUT == kHalf) {
          constexpr int e = kBf16 ? 2 : 1;
          if (turns) {
            turn_halves<kBf16>(r.a[u].x, r.b[u].x, w);
            turn_halves<kBf16>(r.a[u].y, r.b[u].y, w + e);
            turn_halves<kBf16>(r.a[u].z, r.b[u].z, w + 2 * e);
            turn_halves<kBf16>(r.a[u].w, r.b[u].w, w + 3 * e);
          }
          *reinterpret_cast<uint4*>(dst) = r.a[u];
          if (pair >= 0) *reinterpret_cast<uint4*>(dst + half) = r.b[u];
        } else {
          if (turns) {
            uint32_t* const words[4] = {&r.a[u].x, &r.a[u].y, &r.a[u].z, &r.a[u].w};
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
              if (pair + j >= half) continue;  // a vector may reach past the channels that turn
              if (kBf16) {
                float x0 = __uint_as_float(*words[j] << 16), x1 = __uint_as_float(*words[j] & 0xffff0000u);
                turn_pair(x0, x1, w[j]);
                *words[j] = round2(x0, x1);
              } else {
                float x0 = __uint_as_float(*words[(2 * j) & 3]), x1 = __uint_as_float(*words[(2 * j + 1) & 3]);
                turn_pair(x0, x1, w[j]);
                *words[(2 * j) & 3] = __float_as_uint(x0);
                *words[(2 * j + 1) & 3] = __float_as_uint(x1);
              }
            }
          }
          *reinterpret_cast<uint4*>(dst) = r.a[u];
        }
      }
      advance(x);
    }
  };
  const At none{nt, 0};
  const At begin = first < slots ? At{first / heads, first % heads} : none;
  Batch even, odd;
  At next = begin, done = begin;
  place();
  load(even, next);

  if (warp == 0) {  // a lane for each token of the tile
    const bool here = lane < nt;
    const int64_t tok = t0 + lane;
    int64_t row = 0;
    int pos = 0;
    if (!PAGED && a.positions) {
      if (here) pos = a.positions[tok];
    } else {
      // the first token's sequence, by the whole warp; tokens past its end look among those behind it
      int n = sequence_of(a.cu, a.N, t0, lane);
      if (here && n < a.N && a.cu[n + 1] <= tok) {
        int lo = n + 1, hi = a.N;  // sequences lo .. end at or before tok, as far as it goes
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (a.cu[mid + 1] <= tok) lo = mid + 1;
          else hi = mid;
        }
        n = lo;
      }
      // where cu_seqlens decreases, sequence n need not hold the token
      bool ok = here && n < a.N && tok >= a.cu[n] && tok < a.cu[n + 1];
      if (ok) {
        if (PAGED) {
          const int64_t p = static_cast<int64_t>(a.lens[n]) - (a.cu[n + 1] - tok);
          ok = p >= 0 && p / a.page < a.width;
          if (ok) {
            const int64_t page = a.table[static_cast<int64_t>(n) * a.width + p / a.page];
            ok = page >= 0 && page < a.pages;
            row = (page * a.page + p % a.page) * a.Hk * a.D;
            pos = static_cast<int>(p);
          }
        } else {
          pos = static_cast<int>(tok - a.cu[n]);
        }
      }
      if (!ok) {
        row = -1;
        if (here) set_status(a.status, KDA_ERR_DEVICE_CHECK);
      }
    }
    s_pos[lane] = pos;
    s_row[lane] = row;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const uint64_t x = static_cast<uint64_t>(static_cast<int64_t>(s_pos[t])) * static_cast<uint64_t>(a.freqs[f]);
    const uint32_t u = static_cast<uint32_t>(x >> 32);
    const uint32_t quarter = (u + (1u << 29)) >> 30;
    const float rest = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 0x1p-31f;  // half turns
    float sn, cs;
    sincospif(rest, &sn, &cs);
    const bool swap = quarter & 1;
    float x0 = swap ? sn : cs, x1 = swap ? cs : sn;
    if ((quarter + 1) & 2) x0 = -x0;
    if (quarter & 2) x1 = -x1;
    if (a.inverse) x1 = -x1;
    turn[i] = make_float2(a.mag * x0, a.mag * x1);
  }
  __syncthreads();

  for (;;) {
    while (done.t < nt) {
      load(odd, next);
      finish(even, done);
      load(even, next);
      finish(odd, done);
    }
    c += kThreads;
    if (per_head < kThreads || c >= per_head) break;
    place();
    held = -1;
    next = done = begin;
    load(even, next);
  }
}

template <typename T, bool PAGED>
cudaError_t launch(RotaryArgs a, bool pairs, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int layout = pairs ? kPairs : a.R / 2 % V == 0 ? kHalf : kSingle;
  // Tokens of a CTA: enough for a few rounds of its threads, but no fewer CTAs
  // than four an SM; the table of a tile within its bytes.
  const int64_t vectors = static_cast<int64_t>(a.Hq + a.Hk * (PAGED ? 2 : 1)) * a.D / V;
  int64_t tile = (kTileVectors + vectors - 1) / vectors;
  if (tile > a.S / kMinCtas) tile = a.S / kMinCtas;
  if (tile > kTableBytes / (a.R / 2 * 8)) tile = kTableBytes / (a.R / 2 * 8);
  a.tile = static_cast<int>(tile < 1 ? 1 : tile > kMaxTile ? kMaxTile : tile);
  const unsigned grid = static_cast<unsigned>((a.S + a.tile - 1) / a.tile);
  const size_t smem = static_cast<size_t>(a.tile) * (a.R / 2) * sizeof(float2);
  if (layout == kPairs)
    kda_rotary_kernel<T, kPairs, PAGED><<<grid, kThreads, smem, s>>>(a);
  else if (layout == kHalf)
    kda_rotary_kernel<T, kHalf, PAGED><<<grid, kThreads, smem, s>>>(a);
  else
    kda_rotary_kernel<T, kSingle, PAGED><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

kda_status tensor(const char* name, const void* p, unsigned align = 15u) {
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p & align) return set_error(KDA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align + 1);
  return KDA_OK;
}
kda_status stride(const char* name, int64_t n, int64_t wide, int elt) {
  if (n < wide || n * elt % 16 != 0 || n > kMaxStride)
    return set_error(KDA_ERR_INVALID_ARG, "%s %lld must be at least %lld, at most %lld and a multiple of 16 bytes", name,
                     (long long)n, (long long)wide, (long long)kMaxStride);
  return KDA_OK;
}

#define TRY(x)                     \
  do {                             \
    const kda_status st_ = (x);    \
    if (st_ != KDA_OK) return st_; \
  } while (0)

// what both forms ask of the rotation itself
kda_status validate_turn(const kda_rotary_problem* p, int D) {
  if (p->rotary_dim < 2 || p->rotary_dim > D || p->rotary_dim % 2 != 0)
    return set_error(KDA_ERR_INVALID_ARG, "rotary_dim %d must be even and within 2 .. head_dim %d", p->rotary_dim, D);
  if (!isfinite(p->magnitude)) return set_error(KDA_ERR_INVALID_ARG, "magnitude must be finite");
  if ((p->interleaved | p->inverse) & ~1) return set_error(KDA_ERR_INVALID_ARG, "interleaved and inverse are 0 or 1");
  return tensor("freqs", p->freqs, 7u);
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_rotary(const kda_rotary_problem* p, const void* q, const void* k, void* q_out, void* k_out, int32_t* status,
                      void* stream) {
  using namespace kda;
  if (!p) return set_error(KDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->dtype != KDA_DTYPE_BF16 && p->dtype != KDA_DTYPE_F32)
    return set_error(KDA_ERR_UNSUPPORTED, "dtype %d is not supported", p->dtype);
  const int e = p->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  if (p->head_dim < 8 || p->head_dim % 8 != 0 || p->head_dim > 512)
    return set_error(KDA_ERR_UNSUPPORTED, "head_dim %d is not supported (a multiple of 8, up to 512)", p->head_dim);
  if (p->num_heads < 1 || p->num_kv_heads < 0 || p->num_heads > 4096 || p->num_kv_heads > 4096)
    return set_error(KDA_ERR_INVALID_ARG, "num_heads %d and num_kv_heads %d out of range", p->num_heads, p->num_kv_heads);
  if (p->total_tokens < 0 || p->total_tokens > INT32_MAX)
    return set_error(KDA_ERR_INVALID_ARG, "total_tokens %lld out of range", (long long)p->total_tokens);
  TRY(validate_turn(p, p->head_dim));
  TRY(stride("q_stride", p->q_stride, (int64_t)p->num_heads * p->head_dim, e));
  if (p->num_kv_heads) TRY(stride("k_stride", p->k_stride, (int64_t)p->num_kv_heads * p->head_dim, e));
  if (p->positions) {
    TRY(tensor("positions", p->positions, 3u));
  } else {
    if (p->num_seqs < 1) return set_error(KDA_ERR_INVALID_ARG, "num_seqs %d out of range", p->num_seqs);
    TRY(tensor("cu_seqlens", p->cu_seqlens, 3u));
  }
  if ((uintptr_t)status & 3u) return set_error(KDA_ERR_INVALID_ARG, "status is not 4-byte aligned");
  if (p->total_tokens == 0) return KDA_OK;
  TRY(tensor("q", q));
  TRY(tensor("q_out", q_out));
  if (q_out == q && p->q_stride != (int64_t)p->num_heads * p->head_dim)
    return set_error(KDA_ERR_INVALID_ARG, "q_out may be q only where q is contiguous");
  if (p->num_kv_heads) {
    TRY(tensor("k", k));
    TRY(tensor("k_out", k_out));
    if (k_out == k && p->k_stride != (int64_t)p->num_kv_heads * p->head_dim)
      return set_error(KDA_ERR_INVALID_ARG, "k_out may be k only where k is contiguous");
  }
  RotaryArgs a{};
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out; a.qs = p->q_stride; a.ks = p->k_stride;
  a.freqs = p->freqs; a.positions = p->positions; a.cu = p->cu_seqlens; a.status = status;
  a.S = p->total_tokens; a.N = p->num_seqs; a.Hq = p->num_heads; a.Hk = p->num_kv_heads; a.D = p->head_dim;
  a.R = p->rotary_dim; a.mag = p->magnitude; a.inverse = p->inverse;
  const cudaError_t r = e == 2 ? launch<__nv_bfloat16, false>(a, p->interleaved, (cudaStream_t)stream)
                               : launch<float, false>(a, p->interleaved, (cudaStream_t)stream);
  return r == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "rotary launch failed: %s", cudaGetErrorString(r));
}

kda_status kda_paged_append_rotary(const kda_paged_problem* p, const kda_rotary_problem* r, int64_t v_stride, const void* q,
                                   const void* k, const void* v, void* q_out, void* k_pages, void* v_pages, int32_t* status,
                                   void* stream) {
  using namespace kda;
  TRY(validate_paged(p, true));
  if (!r) return set_error(KDA_ERR_INVALID_ARG, "rotary problem is NULL");
  TRY(validate_turn(r, p->head_dim));
  if (r->inverse) return set_error(KDA_ERR_INVALID_ARG, "an append has no inverse rotation");
  if (!q != !q_out) return set_error(KDA_ERR_INVALID_ARG, "q and q_out are given together or not at all");
  if (q) TRY(stride("q_stride", r->q_stride, (int64_t)p->num_heads * p->head_dim, 2));
  TRY(stride("k_stride", r->k_stride, (int64_t)p->num_kv_heads * p->head_dim, 2));
  TRY(stride("v_stride", v_stride, (int64_t)p->num_kv_heads * p->head_dim, 2));
  if ((uintptr_t)status & 3u) return set_error(KDA_ERR_INVALID_ARG, "status is not 4-byte aligned");
  if (p->total_tokens == 0) return KDA_OK;
  if (q) {
    TRY(tensor("q", q));
    TRY(tensor("q_out", q_out));
    if (q_out == q && r->q_stride != (int64_t)p->num_heads * p->head_dim)
      return set_error(KDA_ERR_INVALID_ARG, "q_out may be q only where q is contiguous");
  }
  TRY(tensor("k", k));
  TRY(tensor("v", v));
  TRY(tensor("k_pages", k_pages));
  TRY(tensor("v_pages", v_pages));
  RotaryArgs a{};
  a.q = q; a.k = k; a.v = v; a.qo = q_out; a.ko = k_pages; a.vo = v_pages;
  a.qs = r->q_stride; a.ks = r->k_stride; a.vs = v_stride;
  a.freqs = r->freqs; a.cu = p->cu_seqlens; a.table = p->page_table; a.lens = p->kv_lens; a.status = status;
  a.S = p->total_tokens; a.pages = p->num_pages; a.N = p->num_seqs; a.Hq = q ? p->num_heads : 0; a.Hk = p->num_kv_heads;
  a.D = p->head_dim; a.R = r->rotary_dim; a.page = p->page_size; a.width = p->max_pages; a.mag = r->magnitude;
  const cudaError_t st = launch<__nv_bfloat16, true>(a, r->interleaved, (cudaStream_t)stream);
  return st == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "append launch failed: %s", cudaGetErrorString(st));
}

}  // extern "C"
