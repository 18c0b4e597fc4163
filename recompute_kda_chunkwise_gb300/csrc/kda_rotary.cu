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
// tokens, bf16: 151 MB each way.
//
// Split. A CTA takes a tile of tokens with all their heads. A token's sines
// and cosines are formed once, in shared memory, for all of its heads (each
// costs some 40 instructions: formed anew for every head they would take as
// long as the memory). Its threads take 16-byte vectors, both ends of eight
// (fp32: four) pairs each; the first loads are under way while the angles are
// formed, which is what a call for one token waits for.
#include <math.h>

#include "kda_blocks.h"
#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 32;          // tokens of a CTA, at most
constexpr int kTableBytes = 32768;    // sines and cosines of a tile
constexpr int kBatch = 2;             // items of a thread whose loads are in flight together

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

template <typename T>
struct alignas(16) Vec {
  T x[16 / sizeof(T)];
};

// How a head's channels are cut into items of work.
enum Layout {
  kHalf,    // pairs (i, i + R/2), both halves whole vectors: an item is a vector of either, or one that passes
  kPairs,   // pairs (2i, 2i + 1): an item is a vector
  kSingle,  // pairs (i, i + R/2) that no vector divides: an item is a pair, or an element that passes
};

template <typename T, int LAYOUT, bool PAGED>
__global__ void __launch_bounds__(kThreads) kda_rotary_kernel(const RotaryArgs a) {
  constexpr int V = 16 / sizeof(T);
  extern __shared__ float2 turn[];  // [tile][R / 2]: magnitude * (cos, sin)
  __shared__ int32_t s_pos[kMaxTile];
  __shared__ int64_t s_row[kMaxTile];  // row of k_out (paged: of the pages); negative: the token is skipped
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  const int nt = static_cast<int>(a.S - t0 < a.tile ? a.S - t0 : a.tile);
  const int half = a.R / 2;
  const int per_head = LAYOUT == kHalf ? half / V + (a.D - a.R) / V : LAYOUT == kPairs ? a.D / V : half + a.D - a.R;
  const int turned = (a.Hq + a.Hk) * per_head;
  const int per_token = turned + (PAGED ? a.Hk * (a.D / V) : 0);
  const int total = nt * per_token;

  struct Item {
    const T* src;
    T* dst;
    int t, c;      // token of the tile; first pair of the item, -1: passes
    int other;     // elements from an item's a to its b
  };
  // `row`: whether destinations are wanted (they need s_row)
  auto item_of = [&](int e, bool row) {
    Item it;
    it.t = e / per_token;
    int r = e - it.t * per_token;
    const int64_t tok = t0 + it.t;
    it.other = half;
    it.dst = nullptr;
    if (PAGED && r >= turned) {  // a vector of values
      r = (r - turned) * V;
      it.src = static_cast<const T*>(a.v) + tok * a.vs + r;
      if (row) it.dst = static_cast<T*>(a.vo) + s_row[it.t] * (static_cast<int64_t>(a.Hk) * a.D) + r;
      it.c = -1;
      return it;
    }
    int head = r / per_head, c = r - head * per_head, off;
    if (LAYOUT == kHalf) {
      const bool pass = c >= half / V;
      off = pass ? a.R + (c - half / V) * V : c * V;
      it.c = pass ? -1 : off;
    } else if (LAYOUT == kPairs) {
      off = c * V;
      it.c = off < a.R ? off / 2 : -1;
    } else {
      off = c < half ? c : half + c;
      it.c = c < half ? c : -1;
    }
    if (head < a.Hq) {
      it.src = static_cast<const T*>(a.q) + tok * a.qs + head * a.D + off;
      it.dst = static_cast<T*>(a.qo) + (tok * a.Hq + head) * a.D + off;
    } else {
      head -= a.Hq;
      it.src = static_cast<const T*>(a.k) + tok * a.ks + head * a.D + off;
      if (row) it.dst = static_cast<T*>(a.ko) + (s_row[it.t] * a.Hk + head) * a.D + off;
    }
    return it;
  };
  Vec<T> va[kBatch], vb[kBatch];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = base + u * kThreads;
      if (e < total) {
        const Item it = item_of(e, false);
        if (LAYOUT == kSingle && !(PAGED && e % per_token >= turned)) {
          va[u].x[0] = *it.src;
          if (it.c >= 0) vb[u].x[0] = it.src[it.other];
        } else {
          va[u] = *reinterpret_cast<const Vec<T>*>(it.src);
          if (LAYOUT == kHalf && it.c >= 0) vb[u] = *reinterpret_cast<const Vec<T>*>(it.src + it.other);
        }
      }
    }
  };
  load(tid);

  for (int t = warp; t < nt; t += kThreads / 32) {
    const int64_t tok = t0 + t;
    int64_t row = tok;
    int pos = 0;
    if (!PAGED && a.positions) {
      pos = a.positions[tok];
    } else {
      const int n = sequence_of(a.cu, a.N, tok, lane);
      // where cu_seqlens decreases, sequence n need not hold the token
      bool ok = n < a.N && tok >= a.cu[n] && tok < a.cu[n + 1];
      if (ok) {
        if (PAGED) {
          const int64_t p = static_cast<int64_t>(a.lens[n]) - (a.cu[n + 1] - tok);
          ok = p >= 0 && p / a.page < a.width;
          if (ok) {
            const int64_t page = a.table[static_cast<int64_t>(n) * a.width + p / a.page];
            ok = page >= 0 && page < a.pages;
            row = page * a.page + p % a.page;
            pos = static_cast<int>(p);
          }
        } else {
          pos = static_cast<int>(tok - a.cu[n]);
        }
      }
      if (!ok) {
        row = -1;
        if (lane == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
      }
    }
    if (lane == 0) {
      s_pos[t] = pos;
      s_row[t] = row;
    }
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
    float c = swap ? sn : cs, s = swap ? cs : sn;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
    if (a.inverse) s = -s;
    turn[i] = make_float2(a.mag * c, a.mag * s);
  }
  __syncthreads();

  for (int base = tid; base < total; base += kBatch * kThreads) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = base + u * kThreads;
      if (e >= total) continue;
      const Item it = item_of(e, true);
      if (s_row[it.t] < 0) continue;
      const float2* const w = turn + it.t * half + it.c;
      if (LAYOUT == kSingle) {
        if (PAGED && e % per_token >= turned) {
          *reinterpret_cast<Vec<T>*>(it.dst) = va[u];
        } else if (it.c >= 0) {
          const float x = ldf(&va[u].x[0]), y = ldf(&vb[u].x[0]);
          const float2 r = *w;
          stf(it.dst, fmaf(x, r.x, -y * r.y));
          stf(it.dst + it.other, fmaf(x, r.y, y * r.x));
        } else {
          *it.dst = va[u].x[0];
        }
        continue;
      }
      if (it.c >= 0) {
        if (LAYOUT == kHalf) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float x = ldf(&va[u].x[j]), y = ldf(&vb[u].x[j]);
            const float2 r = w[j];
            stf(&va[u].x[j], fmaf(x, r.x, -y * r.y));
            stf(&vb[u].x[j], fmaf(x, r.y, y * r.x));
          }
          *reinterpret_cast<Vec<T>*>(it.dst + it.other) = vb[u];
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            if (it.c + j / 2 < half) {  // a vector may reach past the channels that turn
              const float x = ldf(&va[u].x[j]), y = ldf(&va[u].x[j + 1]);
              const float2 r = w[j / 2];
              stf(&va[u].x[j], fmaf(x, r.x, -y * r.y));
              stf(&va[u].x[j + 1], fmaf(x, r.y, y * r.x));
            }
          }
        }
      }
      *reinterpret_cast<Vec<T>*>(it.dst) = va[u];
    }
    load(base + kBatch * kThreads);
  }
}

template <typename T, bool PAGED>
cudaError_t launch(RotaryArgs a, bool pairs, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int layout = pairs ? kPairs : a.R / 2 % V == 0 ? kHalf : kSingle;
  // Tokens of a CTA: enough for two rounds of its threads, but no fewer CTAs
  // than two an SM; the table of a tile within its bytes.
  const int64_t vectors = static_cast<int64_t>(a.Hq + a.Hk) * a.D / V;
  int64_t tile = (2 * kBatch * kThreads + vectors - 1) / vectors;
  if (tile > a.S / 304) tile = a.S / 304;
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
  if (n < wide || n * elt % 16 != 0 || n > ((int64_t)1 << 40))
    return set_error(KDA_ERR_INVALID_ARG, "%s %lld must be at least %lld and a multiple of 16 bytes", name, (long long)n,
                     (long long)wide);
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
