// kda_packed_fwd.cu -- forward of causal attention over packed sequences
// (kda_attention_fwd of kda_blocks.h) on the tcgen05 tensor cores.
//
//   o = softmax(scale q K^T) V,   lse = log sum exp(scale q K^T)
//
// Tiles. An item is 256 tokens of one query head: two streams of 128 rows that
// share every tile of 128 keys, K and V loaded once for both. S = Q K^T and
// O += P V are 128 x 128 x D and 128 x D x 128 products with fp32 sums in
// TMEM; P goes back to TMEM as bf16 over scores that have been read, and is the
// A operand of the second product from there. While one stream's warpgroup
// forms its probabilities (a thread owns a row) the tensor cores run the other's
// products. A row's O is rescaled only when its maximum has grown by more than
// 2^8, by a whole power of two: the factor is exact and the sum takes it out.
// bf16 probabilities because both operands have one type; the row's sum adds
// them in fp32 before they are rounded.
//
// A thread takes its whole row into registers: the maximum first, then 128
// exponentials without a branch between them (690 us for the case below where pieces
// of 32 with a running maximum took 744). The registers come from the other warps
// (687 -> 667). Heads of 64 leave TMEM room for a third tile of scores: the products
// go stream by stream, and each tile's scores are issued three tiles ahead, into the
// place of the tile whose P has just been used, so that they are there when their
// warpgroup comes to them (595 -> 522); a tile of K and its V are one slot, so that a
// product has one wait (506 -> 493; 472 with a barrier for each place of a stream).
//
// Items are handed out heaviest first to one CTA per SM. The next item's queries,
// keys and values are fetched, and its first scores formed, while the last item's
// outputs are written.
//
// Bound: the tensor cores (1024 cycles for a tile of 128 x 128 at D = 128), and the
// chain scores -> probabilities -> products of each stream, of which two hide most.
// 8192 tokens, 64 query heads on 8 of 128: 662 us, 1660 TFLOP/s, 86% of the measured
// bf16 rate; 32768 tokens, 16 heads on 2: 1825. (Clocks of different days differ by some
// 2%: each pair of figures here is of one.) Heads of 64, with the same exponentials
// for half the products: 472 us, 1165 TFLOP/s. One thread issues all products and its
// instructions between them count: descriptors of one addition (771 -> 744 us), one
// joint wait for all that a batch needs (662; 708 with two), the stream a constant (690;
// 754 where it was computed). P handed over in two parts is no faster (686 and 695).
#include <math.h>

#include "kda_packed.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 0, kLoadWarp = 1, kSoftmaxWarp = 4;  // warps 2 and 3 have work where lengths are refused
constexpr int kThreads = 32 * (kSoftmaxWarp + kSoftmaxWarps);
constexpr float kRescale = 8.f;

template <int D>
struct Cfg {
  static constexpr int kTile = kRows * D * 2;              // bytes of 128 rows
  static constexpr int kEach = D == 128 ? 1 : 2;           // tiles of a slot: K and V in turn, or one of each
  static constexpr int kSlots = D == 128 ? 5 : 6;
  static constexpr int kBytes = (2 + kSlots * kEach) * kTile;
  static constexpr int kScores = D == 128 ? 2 : 3;         // tiles of S in TMEM, besides the streams' O
};

struct Shared {
  Handout items;
  uint64_t full[6], empty[6];
  uint64_t q_full, q_empty;
  // of a stream's scores, by the place in TMEM where they lie (see below)
  uint64_t s_full[2][3], p_ready[2][3];
  uint64_t o_done[2], o_free[2];
  uint64_t drain;
  uint32_t tmem;
  int abort_;
};

// Registers a thread: what the block is launched with, and its split.
constexpr int kLaunchRegs = 168, kFewRegs = 120, kManyRegs = 184;
static_assert(128 * kFewRegs + 32 * kSoftmaxWarps * kManyRegs <= kThreads * kLaunchRegs, "a split above the launch's would wait for ever");

// What every role knows of an item.
struct Item {
  int lo, L, head, hk, row0;  // row0: first row of stream 0 in the sequence
  int n[2];                   // key tiles of each stream
};
__device__ __forceinline__ bool item_at(const PackedArgs& a, int tiles, int64_t x, Item& it) {
  if (x >= static_cast<int64_t>(tiles) * a.Hq) return false;
  const Tile t = tile_of(a, tiles, static_cast<int>(x / a.Hq));
  it.lo = t.lo;
  it.L = t.L;
  it.head = static_cast<int>(x % a.Hq);
  it.hk = it.head / (a.Hq / a.Hkv);
  it.row0 = (t.w - 1) * 2 * kRows;
  it.n[0] = 2 * t.w - 1;
  it.n[1] = it.row0 + kRows < t.L ? 2 * t.w : 0;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kda_packed_fwd_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const float sc) {
  constexpr int kTile = Cfg<D>::kTile, kSlots = Cfg<D>::kSlots, kEach = Cfg<D>::kEach, kScores = Cfg<D>::kScores;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const ring = smem + 2 * kTile;  // behind the two query tiles
  Shared* const sh = reinterpret_cast<Shared*>(smem + Cfg<D>::kBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* const ab = &sh->abort_;

  if (smem_addr(smem) & 1023) {  // the swizzle needs it; no static shared memory comes before
    if (tid == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    handout_init(&sh->items, 1 + kSoftmaxWarps);
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      for (int place = 0; place < 3; ++place) {
        mbar_init(&sh->s_full[i][place], 1);
        mbar_init(&sh->p_ready[i][place], 4);
      }
      mbar_init(&sh->o_done[i], 1);
      mbar_init(&sh->o_free[i], 4);
    }
    mbar_init(&sh->drain, 1);
    sh->abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&sh->tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  after_kernel();
  if (a.clears && blockIdx.x == 0 && tid < kClearBytes / 4) a.head[tid] = 0;
  if (a.clears) __syncthreads();
  const int tiles = tiles_of(a, 2 * kRows);  // 0: lengths that do not fit, no warp has work
  const uint32_t tmem = sh->tmem;
  const uint32_t tmem_s = tmem, tmem_o = tmem + 128 * kScores;  // tile i of S (P over it) at + 128 i, O of stream i at + D i
  Item it;

  if (warp == kLoadWarp) {
    registers_down<kFewRegs>();
    // ---- loads: Q, then K and V in turn ----
    Ring r;
    bool ok = true;
    uint32_t items = 0;
    int64_t copies = 0;
    for (int64_t x = blockIdx.x; item_at(a, tiles, x, it);) {
      if (items > 0) ok = ok && wait_all(ab, &sh->q_empty, (items - 1) & 1, a.status);
      if (!ok) {
        handout_give(&sh->items, items + 1, kNoItem);
        break;
      }
      const int streams = it.n[1] ? 2 : 1, nk = it.n[1] ? it.n[1] : it.n[0];
      if (elect()) {
        mbar_expect_tx(&sh->q_full, streams * kTile);
        for (int s = 0; s < streams; ++s)
          load_rows<D>(smem + s * kTile, &qmap, it.head, it.lo + it.row0 + s * kRows, &sh->q_full);
      }
      ++items;
      for (int j = 0; j < nk; ++j) {
        for (int v = 0; v < 2; v += kEach) {
          if (r.turn > 0) ok = ok && wait_all(ab, &sh->empty[r.slot], (r.turn - 1) & 1, a.status);
          if (!ok) break;
          if (elect()) {
            mbar_expect_tx(&sh->full[r.slot], kEach * kTile);
            uint8_t* const to = ring + r.slot * kEach * kTile;
            load_rows<D>(to, v ? &vmap : &kmap, it.hk, it.lo + j * kRows, &sh->full[r.slot]);
            if (kEach == 2) load_rows<D>(to + kTile, &vmap, it.hk, it.lo + j * kRows, &sh->full[r.slot]);
          }
          ++copies;
          r.next(kSlots);
        }
      }
      x = handout_next(&sh->items, items, &a.tickets[0], ok, static_cast<int64_t>(tiles) * a.Hq);
    }
    // after an abort: the copies in flight land before the CTA ends
    if (!ok) {
      for (int64_t p = copies > kSlots ? copies - kSlots : 0; p < copies; ++p)
        settle_for(&sh->full[p % kSlots], static_cast<uint32_t>((p / kSlots) & 1));
      if (items > 0) settle_for(&sh->q_full, (items - 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    registers_down<kFewRegs>();
    // ---- products, issued by one thread ----
    if (elect()) {
      const uint32_t q_at = desc_k(smem), k_at = desc_k(ring), v_at = desc_mn(ring + (kEach - 1) * kTile);
      constexpr uint32_t kStep = kTile >> 4;  // from a slot's descriptor to the next
      const uint32_t full = smem_addr(sh->full), p_ready = smem_addr(sh->p_ready);
      Ring rk;  // the ring's position of K(j); V(j) is the next one
      uint32_t items = 0, turn_p[2] = {0, 0}, used_o[2] = {0, 0};  // turn_p, three places: a bit for each
      bool ok = true;
      if constexpr (kScores == 3) {
        // Scores are issued three tiles ahead, in the place of the tile whose P has just been used. The order is
        // stream 0, stream 1 of the first keys, of the second, ...; stream 0 has no part in the last.
        // A stream has a barrier for each place: scores come to one again only behind the wait for the P that was
        // formed there, so neither barrier can complete twice before it is seen. (One for even and one for odd tiles
        // could: an item of one stream has tiles 0 and 2 on their way at once. One for both streams would let
        // a stream through that had no part in the item before.)
        while (item_at(a, tiles, handout_take_alone(&sh->items, items), it)) {
          const bool two = it.n[1] > 0;
          const int n0 = it.n[0], nk = two ? it.n[1] : n0;
          ++items;
          if (!ok) continue;
          auto scores = [&](int s, int j, int place) {
            mma_scores<D>(tmem_s + 128 * place, q_at + s * kStep, k_at + rk.slot * 2 * kStep);
            mma_commit(&sh->s_full[s][place]);
            if (s == two) {
              if (j + 1 == nk) mma_commit(&sh->q_empty);
              rk.next(kSlots);
            }
          };
          auto wait1 = [&](uint32_t bar, uint32_t turn) {
            return wait_for(ab, a.status, [&]() { return poll(bar, turn); });
          };
          auto first = [&](int s, int j, int place) {
            ok = ok && wait1(smem_addr(&sh->q_full), items - 1) && wait1(full + 8 * rk.slot, rk.turn);
            if (!ok) return;
            fence_after_sync();
            scores(s, j, place);
          };
          Ring rv = rk;
          int place = 0;
          // O (+)= P V of stream s, tile j; then scores of (ns, nj) if `more`, the first with those keys if `fresh`
          auto outputs = [&](int s, int j, bool more, bool fresh, int ns, int nj) {
            if (!ok) return;
            const uint32_t turn = turn_p[s] >> place, p = p_ready + 24 * s + 8 * place;
            turn_p[s] ^= 1u << place;
            const bool wait_k = more && fresh;
            const uint32_t k_full = wait_k ? full + 8 * rk.slot : p, k_turn = wait_k ? rk.turn : turn;
            ok = wait_for(ab, a.status, [&]() { return fresh ? poll2(p, turn, k_full, k_turn) : poll(p, turn); });
            if (j == 0 && used_o[s]++ > 0) ok = ok && wait1(smem_addr(&sh->o_free[s]), used_o[s] - 2);
            if (!ok) return;
            fence_after_sync();
            mma_rows<D, 128>(tmem_o + D * s, tmem_s + 128 * place, v_at + rv.slot * 2 * kStep, j > 0);
            if (more) scores(ns, nj, place);
            if (s == two) {
              mma_commit(&sh->empty[rv.slot]);
              rv.next(kSlots);
            }
            if (j + 1 == (s ? nk : n0)) mma_commit(&sh->o_done[s]);
            place = place == 2 ? 0 : place + 1;
          };
          first(0, 0, 0);
          if (two) {
            first(1, 0, 1);
            if (n0 > 1) first(0, 1, 2);
            else first(1, 1, 2);
            for (int j = 0; j < n0; ++j) {
              outputs(0, j, j + 1 < n0, false, 1, j + 1);
              if (j + 2 == n0) outputs(1, j, true, true, 1, n0);
              else outputs(1, j, j + 2 < n0, true, 0, j + 2);
            }
            outputs(1, n0, false, false, 0, 0);
          } else {
            if (n0 > 1) first(0, 1, 1);
            if (n0 > 2) first(0, 2, 2);
            for (int j = 0; j < n0; ++j) outputs(0, j, j + 3 < n0, true, 0, j + 3);
          }
        }
      }
      auto qk = [&](int s, int slot) {
        mma_scores<D>(tmem_s + 128 * s, q_at + s * kStep, k_at + slot * kStep);
        mma_commit(&sh->s_full[s][0]);
      };
      while (kScores == 2 && item_at(a, tiles, handout_take_alone(&sh->items, items), it)) {
        const int nk = it.n[1] ? it.n[1] : it.n[0];
        ++items;
        if (!ok) continue;
        const uint32_t first = full + 8 * rk.slot;
        ok = wait3(ab, a.status, smem_addr(&sh->q_full), items - 1, first, rk.turn, first, rk.turn);
        if (!ok) continue;
        fence_after_sync();
        qk(0, rk.slot);
        if (it.n[1]) qk(1, rk.slot);
        mma_commit(&sh->empty[rk.slot]);
        if (nk == 1) mma_commit(&sh->q_empty);
        for (int j = 0; ok && j < nk; ++j) {
          Ring rv = rk;
          rv.next(kSlots);
          rk = rv;
          rk.next(kSlots);  // K(j + 1)
          const bool more = j + 1 < nk;
          const uint32_t v_full = full + 8 * rv.slot, k_full = more ? full + 8 * rk.slot : v_full;
          const uint32_t k_turn = more ? rk.turn : rv.turn;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || j >= it.n[s]) continue;
            // P, V, the next K, and at an item's start O
            ok = wait3(ab, a.status, p_ready + 24 * s, turn_p[s]++, v_full, rv.turn, k_full, k_turn);
            if (j == 0 && used_o[s]++ > 0) {
              const uint32_t o_free = smem_addr(&sh->o_free[s]), turn = used_o[s] - 2;
              ok = ok && wait3(ab, a.status, o_free, turn, o_free, turn, o_free, turn);
            }
            if (!ok) continue;
            fence_after_sync();
            mma_rows<D, 128>(tmem_o + 128 * s, tmem_s + 128 * s, v_at + rv.slot * kStep, j > 0);
            if (j + 1 == it.n[s]) mma_commit(&sh->o_done[s]);
            if (j + 1 < it.n[s]) qk(s, rk.slot);
          }
          if (ok) {
            mma_commit(&sh->empty[rv.slot]);
            if (more) mma_commit(&sh->empty[rk.slot]);
            if (j + 2 == nk) mma_commit(&sh->q_empty);
          }
        }
      }
      // nothing of this thread may be in flight when TMEM is freed
      mma_commit(&sh->drain);
      settle_for(&sh->drain, 0);
    }
    __syncwarp();
  } else if (warp < kSoftmaxWarp) {
    registers_down<kFewRegs>();
    if (tiles == 0) {
      if (a.fresh & 1) fill_nan(a.o, a.S * a.Hq * (D / 2), tid - 64, 64);
      if (a.fresh & 2) fill_nan(a.lse, a.S * a.Hq, tid - 64, 64);
    }
  } else {
    registers_up<kManyRegs>();
    // ---- softmax: thread = row, warpgroup = stream ----
    const int st = (warp - kSoftmaxWarp) >> 2, row = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t my_o = tmem_o + D * st + lane_base;
    uint32_t turn_s = 0, turn_d = 0, items = 0;  // turn_s: a bit for each place
    int64_t pos = 0;  // ring position of the item's K(0)
    while (item_at(a, tiles, handout_take(&sh->items, items++), it)) {
      const int nt = it.n[st], nk = it.n[1] ? it.n[1] : it.n[0];
      const int at = it.row0 + st * kRows + row;  // row of the sequence
      const bool used = at < it.L;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nt; ++j) {
        const int number = it.n[1] == 0 ? j : 2 * j + (j < it.n[0] ? st : 0);  // of the tile in the products' order
        const int place = kScores == 2 ? 0 : number % 3;
        const uint32_t my_s = tmem_s + 128 * (kScores == 2 ? st : place) + lane_base;
        wait_all(ab, &sh->s_full[st][place], turn_s >> place & 1, a.status);
        turn_s ^= 1u << place;
        fence_after_sync();
        if (j + 1 == nt) {  // the tile on the diagonal: -inf into S first, off the common path
          const int open = used ? row + 1 : 0;
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
          const int past = it.L - j * kRows;  // rows of the tile from here on are another sequence's
          if (past < kRows) {
            const int64_t vpos = kEach == 2 ? pos + j : pos + 2 * j + 1;
            const int slot = static_cast<int>(vpos % kSlots);
            if (wait_all(ab, &sh->full[slot], static_cast<uint32_t>((vpos / kSlots) & 1), a.status) && row >= past)
              zero_row<D>(ring + (slot * kEach + kEach - 1) * kTile, row);
            fence_async_smem();
          }
        }
        // The whole row in registers: its maximum first, then probabilities without a branch.
        uint32_t x[4][32];
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto highest = [&](const uint32_t(&y)[32]) {
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            top[c / 2 & 3] = fmaxf(fmaxf(top[c / 2 & 3], __uint_as_float(y[c])), __uint_as_float(y[c + 1]));
        };
#pragma unroll
        for (int h = 0; h < 4; ++h) tmem_ask(my_s + 32 * h, x[h]);
#pragma unroll
        for (int h = 0; h < 4; ++h) tmem_got(x[h]);
#pragma unroll
        for (int h = 0; h < 4; ++h) highest(x[h]);
        const float mn = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sc;
        const bool grow = mn > m + kRescale;  // m = -inf: any finite maximum
        if (__any_sync(~0u, grow)) {
          // by a whole number of octaves: the factor is exact
          const float k = ceilf(mn - m);
          const float f = !grow ? 1.f : k < 126.f ? __uint_as_float((127u - static_cast<uint32_t>(k)) << 23) : 0.f;
          if (grow) m = m == -INFINITY ? mn : m + k;
          l *= f;
          if (j > 0) {
            // The stream's O exists, and is complete where S of this tile was issued after it; else V of
            // the tile before is given up when it is.
            if (kScores == 3) {
              const int64_t vpos = pos + j - 1;
              wait_all(ab, &sh->empty[vpos % kSlots], static_cast<uint32_t>((vpos / kSlots) & 1), a.status);
              fence_after_sync();
            }
            uint32_t y[16];
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
        const uint64_t sc2 = pack2(__float_as_uint(sc), __float_as_uint(sc));
        const uint64_t ref2 = pack2(__float_as_uint(-ref), __float_as_uint(-ref));
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t p[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 e = unpack2(fma2(pack2(x[h][2 * c], x[h][2 * c + 1]), sc2, ref2));
            const float e0 = ex2(e.x), e1 = ex2(e.y);
            sum[c & 3] = add2(sum[c & 3], pack2(__float_as_uint(e0), __float_as_uint(e1)));
            p[c] = pack_bf16(e0, e1);
          }
          tmem_st(my_s + 16 * h, p);
        }
        const float2 all = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        l += all.x + all.y;
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_ready[st][place]);
      }
      pos += kEach == 2 ? nk : 2 * nk;
      if (nt == 0) continue;
      const bool fine = wait_all(ab, &sh->o_done[st], turn_d++ & 1, a.status);
      fence_after_sync();
      // every row sees its own key: l is 0 or NaN only where the scores are not finite
      const float inv = 1.f / l;
      const int64_t tok = static_cast<int64_t>(it.lo) + at;
      __nv_bfloat16* const out = a.o + (tok * a.Hq + it.head) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t x[32];
        tmem_ask(my_o + c, x);
        tmem_got(x);
        if (used && fine) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            auto two = [&](int e) {
              return pack_bf16(__uint_as_float(x[k + e]) * inv, __uint_as_float(x[k + e + 1]) * inv);
            };
            *reinterpret_cast<uint4*>(out + c + k) = make_uint4(two(0), two(2), two(4), two(6));
          }
        }
      }
      if (used && fine)
        a.lse[static_cast<int64_t>(it.head) * a.S + tok] = (m + log2f(l)) * 0.6931471805599453f;
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->o_free[st]);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const PackedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  const size_t smem = Cfg<D>::kBytes + sizeof(Shared);
  static PerDevice kept;
  int64_t sms = 0;
  const cudaError_t e = packed_sms(kept, kda_packed_fwd_kernel<D>, smem, &sms, kLaunchRegs);
  if (e != cudaSuccess) return e;
  const int64_t most = (a.S / (2 * kRows) + a.N) * a.Hq;  // items
  int64_t ctas = sms < kPackedMaxCtas ? sms : kPackedMaxCtas;
  if (ctas > most) ctas = most;
  return launch_after(kda_packed_fwd_kernel<D>, ctas, kThreads, smem, s, a, q, k, v, a.scale * 1.4426950408889634f);
}

}  // namespace

cudaError_t launch_packed_fwd(const PackedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              cudaStream_t s) {
  return a.D == 128 ? launch<128>(a, q, k, v, s) : launch<64>(a, q, k, v, s);
}

}  // namespace kda
