// kda_rotary.cu -- rotary positions (kda_rotary of kda_blocks.h) and the paged
// append that rotates on the way (kda_paged_append_rotary).
//
//   (a, b) -> magnitude * (a cos x - b sin x, a sin x + b cos x),  x = position * frequency
//
// Angles. A frequency is held as turns per position in units of 2^-64 of a
// turn. The 64-bit product with a position, modulo 2^64, is the angle's
// fraction of a turn: whole turns drop out without a rounding, where an fp32
// product is off by 0.06 rad at position 10^6. Its upper 32 bits (the rest, less
// than 2^-32 of a turn, is cut off) go to the nearest quarter turn; what is left,
// up to an eighth of a turn, is rounded to fp32: by 2^-28 of a turn at most, 2^-24 of
// itself, which is what its sine is rounded by too.
//
// Bound: HBM, each element read and written once. 72 heads of 128 of 8192
// tokens in bf16 (151 MB each way), rotated and, for the gradient, rotated back:
// 101 us, 90% of the measured copy rate; in fp32 40 heads, 6.2 TB/s. Interleaved
// pairs, whose items are half as long: 52 us a pass, 87%. Halves that no vector
// divides go by what does, the channels behind them by vectors: 40 of 128 channels
// (four at a time) 60 us, 44 (two) 67, 42 (one) 88; all of them one at a time 160.
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
// before). Ten CTAs of 128 threads an SM hold that (104 us with five of 256, pairs 55
// instead of 52, one head of 64 a token 83 instead of 68; 103, 53 and 64 with 64
// threads), twelve half vectors and pairs of fp32 (8192 tokens, 40 heads of 128, both
// ways 118 us, 127 with ten; 1777 tokens, 12 + 3 heads of 64, 9.6 and 11.7, in a graph);
// other pairs and shorter items do better with sixteen.
#include <math.h>

#include "kda_blocks.h"
#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxTile = 32;          // tokens of a CTA, at most: one warp looks them up
constexpr int64_t kMaxStride = 1 << 25;  // elements from a token to the next
static_assert(kMaxStride * kMaxTile <= 1 << 30, "");
constexpr int kTableBytes = 32768;    // sines and cosines of a tile
constexpr int kTileVectors = 1024;    // 16-byte vectors of a CTA, about
constexpr int kSms = 152;

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
  int inverse, fresh;
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

// BYTES of a tensor in the lower words of a vector.
template <int BYTES>
__device__ __forceinline__ uint4 load_words(const void* p) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (BYTES == 16) {
    r = *static_cast<const uint4*>(p);
  } else if constexpr (BYTES == 8) {
    const uint2 x = *static_cast<const uint2*>(p);
    r.x = x.x;
    r.y = x.y;
  } else if constexpr (BYTES == 4) {
    r.x = *static_cast<const uint32_t*>(p);
  } else {
    r.x = *static_cast<const uint16_t*>(p);
  }
  return r;
}
template <int BYTES>
__device__ __forceinline__ void store_words(void* p, const uint4& r) {
  if constexpr (BYTES == 16)
    *static_cast<uint4*>(p) = r;
  else if constexpr (BYTES == 8)
    *static_cast<uint2*>(p) = make_uint2(r.x, r.y);
  else if constexpr (BYTES == 4)
    *static_cast<uint32_t*>(p) = r.x;
  else
    *static_cast<uint16_t*>(p) = static_cast<uint16_t>(r.x);
}

// Zeros in n elements, whole vectors.
template <typename T>
__device__ __forceinline__ void zero_row(T* p, int n) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll 1
  for (int i = 0; i < n; i += V) *reinterpret_cast<uint4*>(p + i) = make_uint4(0u, 0u, 0u, 0u);
}

// How a head's channels are cut into items of work. PAIRS, channels (2i, 2i + 1)
// turn together: an item is a 16-byte vector. Else, channels (i, i + R/2): W, the
// largest power of two up to a vector that divides R/2, elements of either half;
// of the channels that pass, a vector, W elements only up to the first vector.
template <typename T, int W, bool PAIRS>
constexpr int kCtasPerSm = sizeof(T) == 4 ? PAIRS ? 12 : 10 : W == 8 && !PAIRS ? 10 : W == 4 ? 12 : 16;

template <typename T, int W, bool PAIRS, bool PAGED>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<T, W, PAIRS>)
    kda_rotary_kernel(const RotaryArgs a) {
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int kBytes = W * sizeof(T);
  extern __shared__ float2 turn[];  // [tile][R / 2]: magnitude * (cos, sin)
  __shared__ int32_t s_pos[kMaxTile];
  __shared__ int64_t s_row[kMaxTile];  // paged: elements before the token's row of the pages; negative: the token is skipped
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  const int nt = static_cast<int>(a.S - t0 < a.tile ? a.S - t0 : a.tile);
  const int half = a.R / 2;
  constexpr int V = 16 / sizeof(T);
  const int lead = (V - a.R % V) % V / W;  // items between the channels that turn and the next vector's
  const int per_head = PAIRS ? a.D / W : half / W + lead + (a.D - a.R - lead * W) / V;
  const int turned = a.Hq + a.Hk, heads = turned + (PAGED ? a.Hk : 0);  // the paged form's values are copied beside them

  // A thread keeps its place within the heads, and goes over the tokens' heads
  // `slots` at a time; places past one for each thread (long heads that are cut
  // into short items) are taken in another round.
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
  bool wide = true;  // a vector
  auto place = [&]() {
    if (PAIRS) {
      off = c * W;
      pair = off < a.R ? off / 2 : -1;
    } else {
      const int passing = c - half / W;
      wide = W == V || passing >= lead;
      off = passing < 0 ? c * W : a.R + (passing < lead ? passing * W : lead * W + (passing - lead) * V);
      pair = passing < 0 ? off : -1;
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
  struct Item {
    uint4 a, b;
  };
  auto load = [&](Item& r, At& x) {  // x moves past it
    if (x.t < nt) {
      const T* const src = source(x);
      r.a = wide ? load_words<16>(src) : load_words<kBytes>(src);
      if (!PAIRS && pair >= 0) r.b = load_words<kBytes>(src + half);
    }
    advance(x);
  };
  // Sines and cosines of this place's pairs for token `held`: read from shared
  // memory once a token, since lanes 64 bytes apart fall on few banks.
  constexpr int kPairsOf = PAIRS ? W / 2 : W;
  float2 w[kPairsOf < 2 ? 2 : kPairsOf] = {};
  int held = -1;
  auto finish = [&](Item& r, At& x) {
    if (x.t < nt && s_row[x.t] >= 0) {
      T* const dst = target(x);
      const bool turns = pair >= 0 && (!PAGED || x.h < turned);
      if (turns && x.t != held) {
        held = x.t;
        const float2* const from = turn + x.t * half + pair;
#pragma unroll
        for (int j = 0; j < kPairsOf; ++j)
          if (!PAIRS || pair + j < half) w[j] = from[j];
      }
      uint32_t* const words[4] = {&r.a.x, &r.a.y, &r.a.z, &r.a.w};
      if constexpr (PAIRS) {
        if (turns) {
#pragma unroll
          for (int j = 0; j < W / 2; ++j) {
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
      } else {
        uint32_t* const others[4] = {&r.b.x, &r.b.y, &r.b.z, &r.b.w};
        constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4, e = kBf16 ? 2 : 1;  // a single bf16: the upper half is not used
        if (turns) {
#pragma unroll
          for (int j = 0; j < kWords; ++j) turn_halves<kBf16>(*words[j], *others[j], w + e * j);
        }
        if (pair >= 0) store_words<kBytes>(dst + half, r.b);
      }
      if (wide) store_words<16>(dst, r.a);
      else store_words<kBytes>(dst, r.a);
    }
    advance(x);
  };
  const At none{nt, 0};
  const At begin = first < slots ? At{first / heads, first % heads} : none;
  Item even, odd;
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
        if (here) {  // a fresh row by its own lane: behind the tile's loop zeros cost every call (96.7 -> 99.1 us, append 41 -> 43)
          set_status(a.status, KDA_ERR_DEVICE_CHECK);
          if (a.fresh & 1) zero_row(static_cast<T*>(a.qo) + tok * a.Hq * a.D, a.Hq * a.D);
          if (!PAGED && (a.fresh & 2)) zero_row(static_cast<T*>(a.ko) + tok * a.Hk * a.D, a.Hk * a.D);
        }
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

template <typename T, int W, bool PAIRS, bool PAGED>
cudaError_t launch_as(RotaryArgs a, cudaStream_t s) {
  // Tokens of a CTA: enough for a few rounds of its threads, but of a call that all CTAs
  // take at once no more than that needs (1777 tokens, 12 + 3 heads of 64, both ways: halves
  // in bf16 8.3 us, where 1777 CTAs of one token take 11.1; fp32 pairs, of which 1824 CTAs
  // fit, 9.6, and 10.3 with two tokens); the table of a tile within its bytes.
  constexpr int V = 16 / sizeof(T), kWave = kSms * kCtasPerSm<T, W, PAIRS>;
  const int64_t vectors = static_cast<int64_t>(a.Hq + a.Hk * (PAGED ? 2 : 1)) * a.D / V;
  int64_t tile = (kTileVectors + vectors - 1) / vectors;
  if (tile > (a.S + kWave - 1) / kWave) tile = (a.S + kWave - 1) / kWave;
  if (tile > kTableBytes / (a.R / 2 * 8)) tile = kTableBytes / (a.R / 2 * 8);
  a.tile = static_cast<int>(tile < 1 ? 1 : tile > kMaxTile ? kMaxTile : tile);
  const unsigned grid = static_cast<unsigned>((a.S + a.tile - 1) / a.tile);
  const size_t smem = static_cast<size_t>(a.tile) * (a.R / 2) * sizeof(float2);
  kda_rotary_kernel<T, W, PAIRS, PAGED><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool PAGED>
cudaError_t launch(const RotaryArgs& a, bool pairs, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int half = a.R / 2;
  if (pairs) return launch_as<T, V, true, PAGED>(a, s);
  if (half % V == 0) return launch_as<T, V, false, PAGED>(a, s);
  if constexpr (V == 8)
    if (half % 4 == 0) return launch_as<T, 4, false, PAGED>(a, s);
  return half % 2 == 0 ? launch_as<T, 2, false, PAGED>(a, s) : launch_as<T, 1, false, PAGED>(a, s);
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
  if (p->fresh & ~3) return set_error(KDA_ERR_INVALID_ARG, "fresh %d is not 0 .. 3", p->fresh);
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
  a.R = p->rotary_dim; a.mag = p->magnitude; a.inverse = p->inverse; a.fresh = p->fresh;
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
  a.fresh = r->fresh;
  const cudaError_t st = launch<__nv_bfloat16, true>(a, r->interleaved, (cudaStream_t)stream);
  return st == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "append launch failed: %s", cudaGetErrorString(st));
}

}  // extern "C"
