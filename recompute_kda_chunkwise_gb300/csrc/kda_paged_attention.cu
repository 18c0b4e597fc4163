// kda_paged_attention.cu -- attention of new tokens over a paged cache, on
// the tcgen05 tensor cores.
//
//   o = softmax(scale q K^T, causal from the cache's end) V
//
// Tiles. The query heads of one key/value head share its keys, so their rows
// (token, head of the group) fill one 128-row tile: a decode step of a
// grouped head reads K and V once for the whole group, and a chunk of tokens
// fills the tensor cores' 128 rows. Keys come in tiles of 128: S = Q K^T and
// O += P V are 128 x 128 x D and 128 x D x 128 products with fp32 sums in
// TMEM; P goes back to TMEM as bf16, over those of its own scores that have
// been read, and is the A operand of the second product from there. bf16
// because the product takes both operands in one type and V is held in bf16:
// against float64 the output's error goes from 0.0017 of its size (bf16
// outputs of fp32 arithmetic) to 0.0023. P as a sum of two bf16 parts would
// keep 0.0017 and double the second product. The row's sum adds the
// probabilities before they are rounded, in fp32.
//
// Two streams. Even and odd key tiles of a segment go to two warpgroups, each
// with its own S, running maximum, sum and O: while one forms its
// probabilities (a thread owns a row) the tensor cores run the other's
// products. The two are joined once, at the end. A row's O is rescaled
// only when its maximum has grown by more than 2^8 (probabilities then stay
// below 2^8, far inside bf16's and fp32's range; the division by the sum
// takes the factor out).
//
// Split. A call's work is counted in key tiles over all (sequence, key/value
// head, row tile) items, and each CTA takes an equal run of them, cutting
// items where the runs end: ragged lengths, one long sequence and many short
// ones all load every SM alike. An item cut over several CTAs leaves its
// parts (maximum, sum, O in fp32) in the workspace; the CTA that finishes
// last adds them in the order of the keys, so the result does not depend on
// which one it was.
//
// Loads. One warp fetches K and one V, by TMA into a ring of 128-row slots
// each, ahead of the products and across item ends. A copy stays inside a
// page: boxes of gcd(page_size, 128) rows, whose pages a warp looks up 32 at a
// time, a batch ahead. Rows past what an item sees are masked out of S by
// selection and set to zero in V, so stale cache rows (NaN among them) have no
// part in the result. A key that only some of the tile's rows see is masked out
// of S for the others, and where its V holds an infinity or a NaN (zero times
// which is not zero) that V row is zeroed too and added afterwards, to the rows
// that see it.
//
// Bound: decode steps by HBM (K and V once): 32 sequences of 16384 keys, 64
// query heads on 8 of 128 channels, take 235 us with their append, 87% of the
// measured copy rate; about 13 us of it is the start, the cuts and the joins.
// Chunks by the tensor cores, in principle: a 128 x 128 tile is 1024 cycles of
// theirs and 512 of exponentials. Chunks of up to 2048 tokens over 8192 keys
// take 722 us with their append, 57% of the measured bf16 rate, a tile every
// 1655 cycles: each stream's scores, probabilities (1725 cycles of latency for
// a thread's 128) and products (1585) wait for one another, and two streams
// hide half of that. Without the loads that stays as it is; without the
// exponentials it is 1555. The look at V rows that not every row of a tile
// sees is 0.5% of it.
#include <math.h>

#include "kda_attention.cuh"
#include "kda_device.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace tc {

// TMA: a 5-D tile (channel of 64, row of 8, 64-channel block, group of 8 rows, page).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int block, int group, int page,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(block), "r"(group), "r"(page), "r"(bar)
      : "memory");
}

}  // namespace tc

namespace {

using namespace tc;

constexpr int kRows = 128;               // query rows of an item, keys of a tile
constexpr int kSoftmaxWarps = 8;         // two warpgroups
constexpr int kMmaWarp = 0, kLoadWarp = 1;  // kLoadWarp: K, the one after it: V
constexpr int kSoftmaxWarp = 4;             // the first; the warp before it is idle
constexpr int kThreads = 32 * (kSoftmaxWarp + kSoftmaxWarps);
constexpr int kMaxCtas = 152;            // one per SM
constexpr int kRingBytes = 6 * 32768;    // K slots, then V slots
constexpr float kRescale = 8.f;          // log2 growth of a maximum that rescales O

// One item's part that a CTA works on.
struct Segment {
  int n, hk, mt;      // sequence, key/value head, row tile
  int j0, j1;         // key tiles [j0, j1); j0 == j1: no key is seen
  int tiles;          // of the whole item (0: none)
  int rows;           // rows of the tile in use
  int lo, L;          // first token and number of tokens of the sequence
  int seen;           // keys that the tile's last row sees
  int first;          // keys that token 0 of the sequence sees (may be <= 0)
};

// Walks a CTA's segments; every role keeps its own copy.
struct Walk {
  const PagedArgs* a;
  int64_t left;       // tiles of the run that remain (an empty item counts as one)
  int n, hk, mt, j;   // next item and its first tile
  int lo, L, len;     // of sequence n
  int group;

  __device__ __forceinline__ int row_tiles() const { return (L * group + kRows - 1) / kRows; }
  __device__ __forceinline__ int seen_of(int m) const {
    const int last = min((m + 1) * kRows, L * group) - 1;
    return max(len - L + last / group + 1, 0);
  }
  __device__ __forceinline__ int tiles_of(int m) const { return (seen_of(m) + kRows - 1) / kRows; }
  __device__ __forceinline__ void sequence(int i) {
    n = i;
    lo = a->cu[i];
    L = a->cu[i + 1] - lo;
    len = a->lens[i];
    if (len < 0 || static_cast<int64_t>(len) > static_cast<int64_t>(a->width) * a->page) len = 0;
  }
  __device__ __forceinline__ int64_t head_tiles() const {  // one key/value head of the sequence
    int64_t t = 0;
    for (int m = 0, e = row_tiles(); m < e; ++m) t += max(tiles_of(m), 1);
    return t;
  }
  __device__ bool next(Segment& s) {
    if (left <= 0) return false;
    while (mt >= row_tiles()) {  // past the sequence's last row tile
      mt = 0;
      if (++hk >= a->Hkv || L == 0) {
        hk = 0;
        if (n + 1 >= a->N) return false;
        sequence(n + 1);
      }
    }
    s.n = n; s.hk = hk; s.mt = mt; s.lo = lo; s.L = L;
    s.tiles = tiles_of(mt);
    s.seen = seen_of(mt);
    s.first = len - L + 1;
    s.rows = min(kRows, L * group - mt * kRows);
    const int weight = max(s.tiles, 1);
    const int take = static_cast<int>(min(static_cast<int64_t>(weight - j), left));
    s.j0 = min(j, s.tiles);
    s.j1 = min(j + take, s.tiles);
    left -= take;
    j += take;
    if (j >= weight) {
      j = 0;
      ++mt;
    }
    return true;
  }
};

struct Shared {
  uint64_t full[2][6], empty[2][6];   // ring slots of K, of V
  uint64_t s_full[2], p_ready[2];     // per stream
  uint64_t q_ready, done, drain;
  uint32_t tmem;
  int abort_, last;
  int bad_page[16];                   // of the last 16 segments
  int64_t sum[kThreads / 32];
  int64_t run, total, start_base;
  int start_n;
  int bad;
  uint32_t held[8];                   // a segment's held keys (see add_held): 256 of them, from a tile's start
  float m[2][kRows], l[2][kRows];
};

struct Parts {        // the workspace behind the status header
  uint32_t* count;    // [kMaxCtas] parts of a cut item that are done, by the CTA of its first part
  float* ml;          // [2 * kMaxCtas][2][kRows]
  float* o;           // [2 * kMaxCtas][kRows][D]
  int* bad;           // [2 * kMaxCtas]
};
constexpr size_t kCountBytes = 1024, kBadBytes = 2048;
static_assert(kMaxCtas * 4 <= kCountBytes && 2 * kMaxCtas * 4 <= kBadBytes, "");
__host__ __device__ inline Parts parts_of(void* scratch) {
  Parts p;
  p.count = static_cast<uint32_t*>(scratch);
  p.bad = reinterpret_cast<int*>(static_cast<char*>(scratch) + kCountBytes);
  p.ml = reinterpret_cast<float*>(static_cast<char*>(scratch) + kCountBytes + kBadBytes);
  p.o = p.ml + 2 * kMaxCtas * 2 * kRows;
  return p;
}

// Bounded wait; false when it ran out (the CTA's abort flag is then set) or
// another role gave up. After an abort every role still walks through its
// segments and barriers, but issues no copy and no product any more.
__device__ __forceinline__ bool wait(Shared* sh, uint64_t* bar, uint32_t parity, int* status) {
  const uint32_t at = smem_addr(bar);
  for (int it = 0; it < (1 << 22); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 15) == 15 && *const_cast<volatile int*>(&sh->abort_)) return false;
  }
  *const_cast<volatile int*>(&sh->abort_) = 1;
  set_status(status, KDA_ERR_TIMEOUT);
  return false;
}

// Waits, at most so long, without giving up.
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_addr(bar);
  for (int it = 0; it < (1 << 20); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(at), "r"(parity)
        : "memory");
    if (ok) return;
  }
}

// wait() of a whole warp, with one answer. Lanes may wait for barriers of
// their own: the warp goes on when all of them are through.
__device__ __forceinline__ bool wait_warp(Shared* sh, uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(~0u, wait(sh, bar, parity, status));
}

// a / b of non-negative numbers, in 32 bits where both fit (nearly always: a
// 64-bit division is a long chain of instructions at the start of every call).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Every CTA adds up the call's tiles and finds the start of its run.
__device__ void plan(const PagedArgs& a, Shared* sh, Walk& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.N + kThreads - 1) / kThreads;
  const int n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
  int bad = 0;
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) {
    const int lo = a.cu[n], hi = a.cu[n + 1], len = a.lens[n];
    if (lo < 0 || hi < lo || hi > a.S || (n == 0 && lo != 0) || (n == a.N - 1 && hi != a.S)) {
      bad = 1;
      break;
    }
    if ((len < 0 || static_cast<int64_t>(len) > static_cast<int64_t>(a.width) * a.page) && blockIdx.x == 0)
      set_status(a.status, KDA_ERR_DEVICE_CHECK);
    w.sequence(n);
    mine += w.head_tiles() * a.Hkv;
  }
  bad = __syncthreads_or(bad);
  int64_t upto = mine;  // inclusive sum over the threads of the warp, then over the warps
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t t = __shfl_up_sync(~0u, upto, m);
    if (lane >= m) upto += t;
  }
  if (lane == 31) sh->sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) upto += sh->sum[i];
    total += sh->sum[i];
  }
  if (bad) total = 0;
  const int64_t run = quotient(total + gridDim.x - 1, gridDim.x);  // one tile may be a CTA's run
  const int64_t start = static_cast<int64_t>(blockIdx.x) * run;
  if (start < total && start >= upto - mine && start < upto) {
    int64_t base = upto - mine;
    for (int n = n0; n < n1; ++n) {
      w.sequence(n);
      const int64_t t = w.head_tiles() * a.Hkv;
      if (start < base + t) {
        sh->start_n = n;
        sh->start_base = base;
        break;
      }
      base += t;
    }
  }
  if (tid == 0) {
    sh->run = run;
    sh->total = total;
    if (bad && blockIdx.x == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
  }
  __syncthreads();
  w.left = total - start < run ? total - start : run;
  if (w.left <= 0) return;
  w.sequence(sh->start_n);
  int64_t rest = start - sh->start_base;
  const int64_t head = w.head_tiles();
  w.hk = static_cast<int>(quotient(rest, head));
  rest -= w.hk * head;
  w.mt = 0;
  for (int t; rest >= (t = max(w.tiles_of(w.mt), 1)); ++w.mt) rest -= t;
  w.j = static_cast<int>(rest);
}

// Whether one of eight bf16 values is an infinity or a NaN: adding 1 to an
// exponent of all ones carries into the sign's place.
__device__ __forceinline__ bool not_finite(uint4 x) {
  uint32_t top = 0;
  for (uint32_t u : {x.x, x.y, x.z, x.w}) top |= (u & 0x7f807f80u) + 0x00800080u;
  return (top & 0x80008000u) != 0;
}

// Adds a stream's held keys to its O in TMEM: keys that some rows of the tile see
// and others do not, whose V row is not finite and was zero in the product. They
// lie in key tile `tile` + `odd`, the one of the two that is this stream's. Each
// row that sees one forms its probability again, in fp32 (its sum has it
// already), and takes the V row from the cache; the other rows' O stays as it
// was. Rare, and kept out of the loops' code and registers.
template <int D>
__device__ __noinline__ void add_held(const PagedArgs& a, const uint32_t* held, int n, int hk, int tile, int odd, int limit,
                                      const uint4* q, float m, float sc, uint32_t keep, uint32_t sign, uint32_t my_o) {
  const float ref = m == -INFINITY ? 0.f : m;
  for (int w = 4 * odd; w < 4 * odd + 4; ++w) {
    for (uint32_t left = held[w]; left; left &= left - 1) {
      const int key = tile * kRows + 32 * w + __ffs(left) - 1;
      const int64_t page = a.table[static_cast<int64_t>(n) * a.width + key / a.page];
      if (page < 0 || page >= a.pages) continue;
      const int64_t at = ((page * a.page + key % a.page) * a.Hkv + hk) * D;
      const uint4* const k = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + at);
      const uint32_t* const v = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.v) + at);
      const bool sees = key < limit;
      float p = 0.f;
      if (sees) {
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = q[c], y = k[c];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u = (xs[i] & keep) ^ sign;
            p = fmaf(__uint_as_float(u << 16), __uint_as_float(ys[i] << 16), p);
            p = fmaf(__uint_as_float(u & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), p);
          }
        }
        p = ex2(fmaf(p, sc, -ref));
      }
      __syncwarp();
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t x[16];
        tmem_ask(my_o + c, x);
        tmem_got(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = v[c / 2 + i];
          const float lo = fmaf(p, __uint_as_float(u << 16), __uint_as_float(x[2 * i]));
          const float hi = fmaf(p, __uint_as_float(u & 0xffff0000u), __uint_as_float(x[2 * i + 1]));
          x[2 * i] = sees ? __float_as_uint(lo) : x[2 * i];
          x[2 * i + 1] = sees ? __float_as_uint(hi) : x[2 * i + 1];
        }
        tmem_st(my_o + c, x);
        tmem_st_wait();
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kda_paged_attention_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap kmap,
                               const __grid_constant__ CUtensorMap vmap, const int box, const float sc,
                               const uint32_t keep, const uint32_t sign) {
  constexpr int kSlot = kRows * D * 2;       // bytes of a ring slot
  constexpr int kSlots = kRingBytes / kSlot / 2;  // of K, and of V: 3 at D = 128, 6 at D = 64
  // A slot holds its rows in groups of eight, each 64-channel block of a group
  // as 8 x 128 swizzled bytes: one copy then brings every channel of a box.
  // (The query tile is the usual one, a block of all 128 rows after another.)
  constexpr int kGroup = 8 * D * 2;  // bytes of eight rows
  constexpr int kHalf = kRows * 128;  // bytes of a 64-channel block of the query tile
  score_regs();
  extern __shared__ __align__(1024) uint8_t ring[];
  uint8_t* const qtile = ring + kRingBytes;
  Shared* const sh = reinterpret_cast<Shared*>(qtile + kSlot);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.Hq / a.Hkv;

  if (smem_addr(ring) & 1023) {  // the swizzle needs it; no static shared memory comes before the ring
    if (tid == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2 * kSlots; ++i) {
      mbar_init(&sh->full[i / kSlots][i % kSlots], 1);
      mbar_init(&sh->empty[i / kSlots][i % kSlots], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_ready[i], 4);
    }
    mbar_init(&sh->q_ready, kSoftmaxWarps);
    mbar_init(&sh->done, 1);
    mbar_init(&sh->drain, 1);
    sh->abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&sh->tmem, 512);
  Walk w{};
  w.a = &a;
  w.group = group;
  plan(a, sh, w);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh->tmem;
  const uint32_t tmem_s = tmem, tmem_o = tmem + 256;  // S (P over it) of stream i at + 128 i, O at + 128 i
  Segment s;

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ---- loads ----
    const int which = warp - kLoadWarp;  // 0: K, 1: V
    const CUtensorMap* const map = which ? &vmap : &kmap;
    const uint32_t dst0 = smem_addr(ring) + which * (kRingBytes / 2);
    const int boxes = kRows / box;         // of a tile
    const int batch = 32 / boxes;          // tiles whose pages the lanes hold
    const uint32_t per_page = a.page / box;  // boxes of a page
    int slot = 0;
    uint32_t turn = 0;  // times the ring has been gone round
    int64_t copies = 0;
    bool ok = true;
    int page = 0, nonempty = 0;
    // lane i: page of box i of the batch that starts at tile j
    auto look_up = [&](const Segment& g, int j) {
      const uint32_t at = static_cast<uint32_t>(j * boxes + lane);
      const bool in = lane < batch * boxes && j + lane / boxes < g.j1 && at * box < static_cast<uint32_t>(g.seen);
      page = in ? a.table[static_cast<int64_t>(g.n) * a.width + at / per_page] : 0;
    };
    // a page outside the cache is recorded, and the item's rows become zero (the copy itself writes zeros)
    auto check = [&](int* flag) {
      if (which == 0 && (page < 0 || page >= a.pages)) {
        *const_cast<volatile int*>(flag) = 1;
        set_status(a.status, KDA_ERR_DEVICE_CHECK);
      }
    };
    auto next_segment = [&]() {  // the next one with keys, its first pages on their way
      while (w.next(s))
        if (s.j0 != s.j1) {
          look_up(s, s.j0);
          return true;
        }
      return false;
    };
    for (bool more = next_segment(); more;) {
      const Segment g = s;
      int* const flag = &sh->bad_page[nonempty++ & 15];
      if (which == 0 && lane == 0) *const_cast<volatile int*>(flag) = 0;
      __syncwarp();
      for (int j = g.j0; j < g.j1; j += batch) {
        check(flag);
        const int pages = page;
        if (j + batch < g.j1)
          look_up(g, j + batch);
        else
          more = next_segment();
        for (int t = j; t < min(j + batch, g.j1); ++t) {
          if (turn > 0) ok = ok && wait_warp(sh, &sh->empty[which][slot], (turn - 1) & 1, a.status);
          if (!ok) continue;
          const int here = min(boxes, (g.seen - t * kRows + box - 1) / box);  // boxes with a key that is seen
          if (lane == 0) mbar_expect_tx(&sh->full[which][slot], static_cast<uint32_t>(here * box * D * 2));
          __syncwarp();
          const uint32_t bar = smem_addr(&sh->full[which][slot]);
          uint32_t dst = dst0 + slot * kSlot;
          uint32_t part = static_cast<uint32_t>(t * boxes) % per_page;  // box within its page
          for (int i = 0; i < here; ++i) {
            const int pg = __shfl_sync(~0u, pages, (t - j) * boxes + i);
            if (elect()) tma_load_5d(dst, map, g.hk * (D / 64), static_cast<int>(part) * (box / 8), pg, bar);
            dst += box * D * 2;
            if (++part == per_page) part = 0;
          }
          ++copies;
          if (++slot == kSlots) {
            slot = 0;
            ++turn;
          }
        }
      }
    }
    // after an abort: the copies in flight land before the CTA ends
    if (!ok)
      for (int64_t p = copies > kSlots ? copies - kSlots : 0; p < copies; ++p)
        settle(&sh->full[which][p % kSlots], static_cast<uint32_t>((p / kSlots) & 1));
  } else if (warp == kMmaWarp) {
    // ---- products: QK(0), QK(1), then PV(i) and QK(i + 2) for each tile i ----
    // One warp issues for both streams, and that takes it longer than the
    // tensor cores need unless it is kept short: PV(i) and QK(i + 2) go out
    // after one wait, in which a lane each looks at P(i), V(i) and K(i + 2).
    constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);  // bf16 A and B
    constexpr uint32_t id_qk = idesc(kRows, kRows) | kBf16, id_pv = idesc(kRows, D, false, true) | kBf16;
    // matrix descriptors: the low words are sums that never carry
    const uint64_t q0 = sdesc(smem_addr(qtile), 16), k0 = sdesc(smem_addr(ring), 16),
                   v0 = sdesc(smem_addr(ring) + kRingBytes / 2, 1024);
    // high words: the bytes from one group of eight rows to the next, with the layout's constant bits
    const uint32_t hi = static_cast<uint32_t>(q0 >> 32), hi_kv = hi - (1024 >> 4) + (kGroup >> 4);
    const uint32_t qlo = static_cast<uint32_t>(q0), klo = static_cast<uint32_t>(k0), vlo = static_cast<uint32_t>(v0);
    int kslot = 0, vslot = 0;
    uint32_t kturn = 0, vturn = 0, turn = 0, turn_p[2] = {0, 0};
    bool ok = true;
    auto qk = [&](int st) {
      const uint32_t kd = klo + kslot * (kSlot >> 4), ts = tmem_s + 128 * st;
      if (elect()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma(ts, pack2(qlo + (k >> 2) * (kHalf >> 4) + (k & 3) * 2, hi),
              pack2(kd + (k >> 2) * (1024 >> 4) + (k & 3) * 2, hi_kv), id_qk, k > 0);
        mma_commit(&sh->s_full[st]);
        mma_commit(&sh->empty[0][kslot]);
      }
      if (++kslot == kSlots) {
        kslot = 0;
        ++kturn;
      }
    };
    while (ok && w.next(s)) {
      const int nt = s.j1 - s.j0;
      if (nt == 0) continue;
      ok = wait_warp(sh, lane == 0 ? &sh->q_ready : &sh->full[0][kslot], (lane == 0 ? turn : kturn) & 1, a.status);
      ++turn;
      if (!ok) break;
      fence_after_sync();
      qk(0);
      if (nt > 1) {
        ok = wait_warp(sh, &sh->full[0][kslot], kturn & 1, a.status);
        if (!ok) break;
        fence_after_sync();
        qk(1);
      }
      for (int i = 0; i < nt; ++i) {
        const int st = i & 1;
        const bool more = i + 2 < nt;
        uint64_t* const bar = lane == 1 ? &sh->full[1][vslot] : lane == 2 && more ? &sh->full[0][kslot] : &sh->p_ready[st];
        const uint32_t par = lane == 1 ? vturn : lane == 2 && more ? kturn : turn_p[st];
        ok = wait_warp(sh, bar, par & 1, a.status);
        ++turn_p[st];
        if (!ok) break;
        fence_after_sync();
        const uint32_t vd = vlo + vslot * (kSlot >> 4), ts = tmem_s + 128 * st, to = tmem_o + 128 * st;
        if (elect()) {
#pragma unroll
          for (int k = 0; k < kRows / 16; ++k)
            mma_ta(to, ts + 8 * k, pack2(vd + k * (2 * kGroup >> 4), hi_kv), id_pv, (i > 1 || k > 0) ? 1u : 0u);
          mma_commit(&sh->empty[1][vslot]);
        }
        if (++vslot == kSlots) {
          vslot = 0;
          ++vturn;
        }
        if (more) qk(st);
      }
      if (ok && elect()) mma_commit(&sh->done);
    }
    // nothing of this warp may be in flight when TMEM is freed
    if (elect()) mma_commit(&sh->drain);
    settle(&sh->drain, 0);
    __syncwarp();
  } else if (warp >= kSoftmaxWarp) {
    // ---- softmax: thread = row, warpgroup = stream ----
    const int st = (warp - kSoftmaxWarp) >> 2, row = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t my_s = tmem_s + 128 * st + lane_base;
    const uint32_t my_o = tmem_o + 128 * st + lane_base;
    uint32_t turn_s = 0, turn_d = 0;
    int64_t tiles0 = 0;  // tiles before the segment
    const Parts parts = parts_of(a.scratch);
    uint32_t seg = 0;
    while (w.next(s)) {
      const int nt = s.j1 - s.j0;
      const int at = s.mt * kRows + row;  // row of the sequence: token * group + head
      const bool used = row < s.rows;
      const int token = at / group, head = s.hk * group + at % group;
      __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.o) +
                                 (static_cast<int64_t>(s.lo + token) * a.Hq + head) * D;
      if (nt == 0) {  // nothing to see for any row of the tile
        if (used)
          for (int c = st * (D / 2); c < (st + 1) * (D / 2); c += 8)
            *reinterpret_cast<uint4*>(out + c) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      const int limit = used ? s.first + token : 0;  // keys this row sees
      // Keys from `some` on are not seen by the tile's first row, those before
      // by every row in use: at most 127, in this tile of keys and the next.
      const int some = max(s.first + s.mt * kRows / group, 0);
      if (lane == 0) sh->held[4 * ((s.j0 + st + some / kRows) & 1) + (warp & 3)] = 0;  // of the one that is this stream's
      {
        // Q rows into the tile, 16-byte chunks in the 128-byte swizzle; this
        // warpgroup's half of the channels
        if (used) {
          const uint4* const src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(s.lo + token) * a.Hq + head) * D);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint4 x = src[st * (D / 16) + c];
            x.x = (x.x & keep) ^ sign; x.y = (x.y & keep) ^ sign; x.z = (x.z & keep) ^ sign; x.w = (x.w & keep) ^ sign;
            *reinterpret_cast<uint4*>(qtile + sw128_chunk(row, st * (D / 16) + c, kRows)) = x;
          }
        }
        fence_async_smem();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_ready);
      }
      float m = -INFINITY, l = 0.f;
      const bool warp_used = (row & ~31) < s.rows;
      for (int i = st; i < nt; i += 2) {
        wait_warp(sh, &sh->s_full[st], turn_s++ & 1, a.status);
        fence_after_sync();
        const int k0 = (s.j0 + i) * kRows;
        if (warp_used) {
          const int open = limit - k0;  // keys of the tile that the row sees
          if (__any_sync(~0u, open < kRows)) {  // an item's last tiles: -inf into S first, off the common path
#pragma unroll 1
            for (int c0 = 0; c0 < kRows; c0 += 32) {
              uint32_t y[32];
              tmem_ask(my_s + c0, y);
              tmem_got(y);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c0 + c >= open) y[c] = 0xff800000u;
              tmem_st(my_s + c0, y);
            }
            tmem_st_wait();
          }
          // One pass over the row, 32 scores at a time with the next 32 on
          // their way: probabilities against the maximum so far, written over
          // scores that have been read. Where the maximum has grown by more
          // than 2^8 (in a stream's first scores, and rarely after) the row
          // goes over to it first, and what there is of the row is scaled.
          // The loop stays rolled: its code and that of the warp that issues
          // the products then both stay in the instruction cache.
          const uint64_t sc2 = pack2(__float_as_uint(sc), __float_as_uint(sc));
          uint64_t sum[4] = {0, 0, 0, 0};
          uint32_t x[32];
          auto highest = [&]() {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              top[c / 2 & 3] = fmaxf(fmaxf(top[c / 2 & 3], __uint_as_float(x[c])), __uint_as_float(x[c + 1]));
            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sc;
          };
          score_ask(my_s);
          score_got(x);
          float mn = highest();
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            const bool grow = mn > m + kRescale;  // m = -inf: any finite maximum
            if (__any_sync(~0u, grow)) {
              // by a whole number of octaves: the factor is exact, for P too
              const float k = ceilf(mn - m);
              const float f = !grow ? 1.f : k < 126.f ? __uint_as_float((127u - static_cast<uint32_t>(k)) << 23) : 0.f;
              if (grow) m = m == -INFINITY ? mn : m + k;
              l *= f;
              const uint64_t f2 = pack2(__float_as_uint(f), __float_as_uint(f));
#pragma unroll
              for (int c = 0; c < 4; ++c) sum[c] = fma2(sum[c], f2, 0);
              tmem_st_wait();
              uint32_t y[16];
#pragma unroll 1
              for (int c = 0; c < 16 * h; c += 16) {
                tmem_ask(my_s + c, y);
                tmem_got(y);
#pragma unroll
                for (int q = 0; q < 16; ++q)
                  y[q] = pack_bf16(__uint_as_float(y[q] << 16) * f, __uint_as_float(y[q] & 0xffff0000u) * f);
                tmem_st(my_s + c, y);
              }
              if (i >= 2) {  // the stream's O exists, and is complete: S of this tile was issued after it
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  tmem_ask(my_o + c, y);
                  tmem_got(y);
#pragma unroll
                  for (int q = 0; q < 16; ++q) y[q] = __float_as_uint(__uint_as_float(y[q]) * f);
                  tmem_st(my_o + c, y);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const uint64_t ref2 = pack2(__float_as_uint(-ref), __float_as_uint(-ref));
            uint64_t t[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) t[c] = fma2(pack2(x[2 * c], x[2 * c + 1]), sc2, ref2);
            score_ask(my_s + (32 * (h + 1) & 96));  // after the last: not used
            uint32_t p[16];
            auto exps = [&](int c) {
              const float2 e = unpack2(t[c]);
              const float e0 = ex2(e.x), e1 = ex2(e.y);
              sum[c & 3] = add2(sum[c & 3], pack2(__float_as_uint(e0), __float_as_uint(e1)));
              p[c] = pack_bf16(e0, e1);
            };
#pragma unroll
            for (int c = 0; c < 8; ++c) exps(c);
            score_got(x);
            mn = highest();
#pragma unroll
            for (int c = 8; c < 16; ++c) exps(c);
            tmem_st(my_s + 16 * h, p);
          }
          const float2 all = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += all.x + all.y;
          tmem_st_wait();
        }
        if (k0 + kRows > some) {
          // keys that not every row of the tile sees: V rows past what any row
          // sees to zero, and those that are not finite (the probabilities of
          // rows that do not see them are zero, but zero times a NaN is not).
          // Behind the probabilities, when V has long arrived.
          const int64_t vpos = tiles0 + i;
          const int slot = static_cast<int>(vpos % kSlots), key = k0 + row;
          const bool here = wait_warp(sh, &sh->full[1][slot], static_cast<uint32_t>((vpos / kSlots) & 1), a.status);
          uint8_t* const v = ring + kRingBytes / 2 + slot * kSlot + (row >> 3) * kGroup + (row & 7) * 128;
          auto chunk = [&](int c) {  // each lane from another one on: eight rows are a multiple of 128 bytes apart
            const int x = (c + lane) % (D / 8);
            return reinterpret_cast<uint4*>(v + x / 8 * 1024 + x % 8 * 16);
          };
          bool hold = false;
          if (here && key >= some && key < s.seen) {
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) hold |= not_finite(*chunk(c));
          }
          if (here && (hold || key >= s.seen)) {
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) *chunk(c) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
          if (hold) atomicOr(&sh->held[((key - some / kRows * kRows) >> 5) & 7], 1u << lane);
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_ready[st]);
      }
      wait_warp(sh, &sh->done, turn_d++ & 1, a.status);
      fence_after_sync();
      // join the two streams: this warpgroup writes its half of the channels
      sh->m[st][row] = m;
      sh->l[st][row] = l;
      named_bar_sync(1, 256);
      {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= sh->held[i];
        if (any) {  // the same for all 256 threads
          if (warp_used)
            add_held<D>(a, sh->held, s.n, s.hk, some / kRows, (s.j0 + st + some / kRows) & 1, limit,
                        reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                       (static_cast<int64_t>(s.lo + token) * a.Hq + head) * D),
                        m, sc, keep, sign, my_o);
          fence_before_sync();
          named_bar_sync(1, 256);
          fence_after_sync();
        }
      }
      const float m0 = sh->m[0][row], m1 = sh->m[1][row];
      const float mm = fmaxf(m0, m1);
      const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - mm), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
      const float ll = sh->l[0][row] * f0 + sh->l[1][row] * f1;
      const bool whole = nt == s.tiles;
      const int bad = *const_cast<volatile int*>(&sh->bad_page[seg++ & 15]);
      const int part = 2 * static_cast<int>(blockIdx.x) + (s.j0 == 0 ? 1 : 0);
      // A sum of zero: no key is seen (zeros), or every score that is was -inf (0 / 0, as the definition has it).
      const float none = limit > 0 ? __uint_as_float(0x7fc00000u) : 0.f;
      const float inv = !whole ? 1.f : bad ? 0.f : ll == 0.f ? none : 1.f / ll;
      if (warp_used) {
#pragma unroll 1
        for (int c = st * (D / 2); c < (st + 1) * (D / 2); c += 32) {
          uint32_t x[32], y[32];
          tmem_ask(tmem_o + lane_base + c, x);
          tmem_got(x);
          if (nt > 1) {
            tmem_ask(tmem_o + 128 + lane_base + c, y);
            tmem_got(y);
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            // a stream without a key of this row: its O holds nothing to add
            float v = m0 == -INFINITY ? 0.f : __uint_as_float(x[k]) * f0;
            if (nt > 1 && m1 != -INFINITY) v = fmaf(__uint_as_float(y[k]), f1, v);
            x[k] = __float_as_uint(inv == 0.f ? 0.f : v * inv);
          }
          if (used && whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint4 o;
              o.x = pack_bf16(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
              o.y = pack_bf16(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
              o.z = pack_bf16(__uint_as_float(x[k + 4]), __uint_as_float(x[k + 5]));
              o.w = pack_bf16(__uint_as_float(x[k + 6]), __uint_as_float(x[k + 7]));
              *reinterpret_cast<uint4*>(out + c + k) = o;
            }
          } else if (used) {
            float* const po = parts.o + (static_cast<int64_t>(part) * kRows + row) * D + c;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<uint4*>(po + k) = make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          }
        }
      }
      tiles0 += nt;
      if (!whole) {
        if (st == 0 && used) {
          parts.ml[part * 2 * kRows + row] = mm;
          parts.ml[part * 2 * kRows + kRows + row] = ll;
        }
        if (warp == kSoftmaxWarp && lane == 0) parts.bad[part] = bad;
        // The CTAs of this item: the run that holds its first tile, and those after it.
        const int64_t run_end = min((static_cast<int64_t>(blockIdx.x) + 1) * sh->run, sh->total);
        const int64_t item0 = run_end - w.left - s.j1, item1 = item0 + s.tiles;
        const int c0 = static_cast<int>(quotient(item0, sh->run)), c1 = static_cast<int>(quotient(item1 - 1, sh->run));
        named_bar_sync(1, 256);
        if (warp == kSoftmaxWarp && lane == 0) {
          __threadfence();  // this CTA's part, written before the barrier, ...
          sh->last = atomicAdd(&parts.count[c0], 1u) == static_cast<uint32_t>(c1 - c0);
          __threadfence();  // ... and the others' before what follows it
        }
        named_bar_sync(1, 256);
        if (sh->last) {
          // parts c0 (its slot 1) .. c1 (their slot 0), in the order of the keys
          int any = 0;
          for (int c = c0; c <= c1; ++c) any |= __ldcg(&parts.bad[2 * c + (c == c0)]);
          if (st == 0 && used) {
            float top = -INFINITY, sum = 0.f;
            for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(&parts.ml[(2 * c + (c == c0)) * 2 * kRows + row]));
            for (int c = c0; c <= c1; ++c) {
              const float* const q = &parts.ml[(2 * c + (c == c0)) * 2 * kRows + row];
              const float pm = __ldcg(q);
              sum += __ldcg(q + kRows) * (pm == -INFINITY ? 0.f : ex2(pm - top));
            }
            sh->m[0][row] = top;
            sh->l[0][row] = any ? 0.f : sum == 0.f ? none : 1.f / sum;
          }
          named_bar_sync(1, 256);
          for (int e = tid - 32 * kSoftmaxWarp; e < s.rows * (D / 8); e += 256) {
            const int r = e / (D / 8), c8 = e % (D / 8) * 8;
            const float top = sh->m[0][r], scale = sh->l[0][r];
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int c = c0; c <= c1; ++c) {
              const int p = 2 * c + (c == c0);
              const float pm = __ldcg(&parts.ml[p * 2 * kRows + r]);
              if (pm == -INFINITY) continue;
              const float f = ex2(pm - top);
              const float4* const q = reinterpret_cast<const float4*>(parts.o + (static_cast<int64_t>(p) * kRows + r) * D + c8);
              const float4 x = __ldcg(q), y = __ldcg(q + 1);
              v[0] = fmaf(x.x, f, v[0]); v[1] = fmaf(x.y, f, v[1]); v[2] = fmaf(x.z, f, v[2]); v[3] = fmaf(x.w, f, v[3]);
              v[4] = fmaf(y.x, f, v[4]); v[5] = fmaf(y.y, f, v[5]); v[6] = fmaf(y.z, f, v[6]); v[7] = fmaf(y.w, f, v[7]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = scale == 0.f ? 0.f : v[k] * scale;
            const int ar = s.mt * kRows + r;
            __nv_bfloat16* const po = static_cast<__nv_bfloat16*>(a.o) +
                                      (static_cast<int64_t>(s.lo + ar / group) * a.Hq + s.hk * group + ar % group) * D + c8;
            *reinterpret_cast<uint4*>(po) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
          }
        }
      }
      // O, m and l are read: the next segment may start
      named_bar_sync(1, 256);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Pages [pages][page][Hkv][D] as (64 channels, row of 8, 64-channel block of
// any head, group of 8 rows, page); box: every channel of one head, `box` rows
// of one page.
bool page_map(CUtensorMap* m, const void* base, const PagedArgs& a, int box) {
  const EncodeFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint32_t blocks = (cuuint32_t)a.D / 64;
  const cuuint64_t row = (cuuint64_t)a.D * 2 * a.Hkv;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)blocks * a.Hkv, (cuuint64_t)a.page / 8, (cuuint64_t)a.pages};
  const cuuint64_t strides[4] = {row, 128, row * 8, row * a.page};
  const cuuint32_t boxes[5] = {64, 8, blocks, (cuuint32_t)box / 8, 1}, ones[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const PagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, int box, cudaStream_t s) {
  const size_t smem = kRingBytes + kRows * D * 2 + sizeof(Shared);
  auto* const kernel = kda_paged_attention_kernel<D>;
  static PerDevice kept;
  int64_t sms = 0;
  cudaError_t e = kept.get(&sms, [&](int dev, int64_t* n) {
    const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    int count = 0;
    const cudaError_t got = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
    *n = count;
    return set != cudaSuccess ? set : got;
  });
  // the status word and the counters that follow it
  if (e == cudaSuccess) e = cudaMemsetAsync(a.status, 0, kHeaderBytes + kCountBytes, s);
  if (e != cudaSuccess) return e;
  const int ctas = static_cast<int>(sms < kMaxCtas ? sms : kMaxCtas);
  // Exponentials are taken in base 2. sc > 0, so that masked scores stay -inf:
  // a negative scale moves to the queries' sign, a scale of 0 to zero queries.
  float sc = fabsf(a.scale) * 1.4426950408889634f;
  const uint32_t keep = sc > 0.f ? ~0u : 0u, sign = a.scale < 0.f ? 0x80008000u : 0u;
  if (!(sc > 0.f)) sc = 1.f;
  kernel<<<ctas, kThreads, smem, s>>>(a, k, v, box, sc, keep, sign);
  return cudaGetLastError();
}

}  // namespace

size_t paged_attention_scratch_bytes(const PagedArgs& a) {
  return kCountBytes + kBadBytes + sizeof(float) * 2 * kMaxCtas * kRows * (2 + a.D);
}

kda_status launch_paged_attention(const PagedArgs& a, cudaStream_t s) {
  int box = kRows;
  while (a.page % box) box /= 2;  // the largest power of two up to 128 that divides the page: at least 8
  CUtensorMap k, v;
  if (!in_context(reinterpret_cast<const void*>(&kda_paged_attention_kernel<64>),
                  [&]() { return page_map(&k, a.k, a, box) && page_map(&v, a.v, a, box); }))
    return set_error(KDA_ERR_CUDA, "the tensor maps of the cache could not be made");
  const cudaError_t e = a.D == 128 ? launch<128>(a, k, v, box, s) : launch<64>(a, k, v, box, s);
  return e == cudaSuccess ? KDA_OK : set_error(KDA_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

}  // namespace kda
