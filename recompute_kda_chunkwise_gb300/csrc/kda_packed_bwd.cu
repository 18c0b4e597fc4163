// kda_packed_bwd.cu -- backward of causal attention over packed sequences
// (kda_attention_bwd of kda_blocks.h) on the tcgen05 tensor cores.
//
//   P = exp(scale q k - lse)      delta = sum(d_o o)
//   dv = P^T d_o      dS = P (d_o v^T - delta)      dk = scale dS^T q      dq = scale dS k
//
// Two passes, one over queries for each tile of keys (dk, dv: 4 products) and
// one over keys for each tile of queries (dq: 3 products), 7 products where 5
// would do. A single pass would add every tile's part of dq to memory in fp32:
// in the order in which CTAs come (other bits every time), or in turns, with
// CTAs waiting for one another. Here each sum is one CTA's, in TMEM.
//
// dk, dv. Keys are the rows (TMEM lanes) of S^T = K Q^T and dP^T = V d_o^T, so
// that P^T and dS^T, written back over the scores as bf16, are A operands of
// dv += P^T d_o and dk += dS^T Q straight from TMEM: neither goes through
// shared memory, whose bandwidth bounds products of two operands there. While
// the warps form P^T the tensor cores run dS^T's product and the next dP^T, and
// the other way round: the order is dv(t), S(t+1), dk(t), dP(t+1).
// A key/value head's keys go over all query heads of its group in one item, or
// over a part of them where there are few items: the parts are then added up,
// in order, by another kernel.
//
// dq. Queries are the rows; dS is dq's A operand in TMEM. dP has two buffers,
// so that the next tile's scores and dP are formed while dS is. delta comes from
// the forward's o, which was rounded to bf16; but a row's dS sums to zero, so what
// this pass finds it to sum to is delta's error, and the other pass gets delta
// without it. Rows whose keys all lie in one tile sum their delta up themselves.
// (Gradients of 77 tokens: 0.0026 of their size off float64 before, 0.0023 with
// it, 0.0017 if nothing but the outputs were rounded.) dS and P are rounded to
// bf16 because the products' operands have one type; as sums of two parts each
// they would cost 40% more products.
//
// Bound: the tensor cores in principle, 512 cycles a product of 128 x 128 x 128: 3584
// a tile for both passes; counters show them active 77% (dk, dv) and 70% (dq) of
// the time. What is left is latency: from a warpgroup's arrival to the product that
// waited for it (300 to 400 cycles) and from there to the scores. 8192 tokens, 64
// query heads on 8 of 128: 2282 us (40 for delta, 1020 dq, 1205 dk and dv), 1204
// TFLOP/s counted as five products; 32768 tokens, 16 heads on 2: 1210. Heads of 64:
// 1689 us, 814 TFLOP/s, bound by the arithmetic between the products. Without
// loads, or without exponentials, neither pass is more than 3% faster. What brought
// it there, in us: a ring each for K and V 2995 -> 2505; descriptors of one addition
// 2452; lse and delta in the ring with d_o instead of a barrier a step 2414; one
// issuing thread with joint waits, dq's scores read a tile ahead 2296; registers for
// dq's arithmetic (2319 before it by the same clock: days differ by 1 to 2%) 2282, with
// 48 bytes a thread spilled in dq's kernel for heads of 128 (-Xptxas -v).
#include <math.h>

#include "kda_packed.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kRows = 128;
// Warpgroups of arithmetic, each a part of a tile's columns: four threads a row.
// With two, heads of 64 take 1909 us instead of 1832 (8192 tokens, 64 heads); heads of
// 128 are alike (2362 and 2339).
constexpr int kGroups = 4, kMathWarps = 4 * kGroups;
constexpr int kCols = kRows / kGroups, kParts = kCols / 32;
constexpr int kMmaWarp = 0, kLoadWarp = 1, kMathWarp = 4;
constexpr int kThreads = 32 * (kMathWarp + kMathWarps);
// Registers a thread of the dq kernel: what the block is launched with, and its split (2319 -> 2282 us
// for the whole backward; that of dk and dv needs no more, and its other warps no fewer).
constexpr int kLaunchRegs = 96, kFewRegs = 64, kManyRegs = 104;
static_assert(128 * kFewRegs + 32 * kMathWarps * kManyRegs <= kThreads * kLaunchRegs, "a split above the launch's would wait for ever");

// P x 32 columns of a tile, a thread's.
template <int P>
__device__ __forceinline__ void load_scores(uint32_t at, uint32_t (&x)[P][32]) {
#pragma unroll
  for (int c = 0; c < P; ++c) tmem_ask(at + 32 * c, x[c]);
#pragma unroll
  for (int c = 0; c < P; ++c) tmem_got(x[c]);
}
// Exponentials (base 2) of a pair, in place.
__device__ __forceinline__ void ex2_pair(uint64_t t, uint32_t& lo, uint32_t& hi) {
  const float2 e = unpack2(t);
  lo = __float_as_uint(ex2(e.x));
  hi = __float_as_uint(ex2(e.y));
}
// Zero where a column is not seen.
template <int P>
__device__ __forceinline__ void hide(uint32_t (&x)[P][32], const uint32_t (&see)[P]) {
#pragma unroll
  for (int c = 0; c < P; ++c)
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(see[c] >> e & 1)) x[c][e] = 0u;
}
// Rounded to bf16, two to a column, over the first half of the columns.
template <int P>
__device__ __forceinline__ void store_bf16(uint32_t at, const uint32_t (&x)[P][32]) {
#pragma unroll
  for (int c = 0; c < P; ++c) {
    uint32_t y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = pack_bf16(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1]));
    tmem_st(at + 16 * c, y);
  }
}
// `f` times a row's sums (n fp32 columns of TMEM) to fp32 or bf16 memory.
template <int N, typename T>
__device__ __forceinline__ void write_row(uint32_t at, float f, T* dst, bool used) {
  constexpr int step = N < 32 ? N : 32;
#pragma unroll 1
  for (int c = 0; c < N; c += step) {
    uint32_t x[step];
    tmem_ask(at + c, x);
    tmem_got(x);
    if (!used) continue;
#pragma unroll
    for (int e = 0; e < step; e += 16 / sizeof(T)) {
      auto v = [&](int k) { return __uint_as_float(x[e + k]) * f; };
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(dst + c + e) = make_float4(v(0), v(1), v(2), v(3));
      else
        *reinterpret_cast<uint4*>(dst + c + e) =
            make_uint4(pack_bf16(v(0), v(1)), pack_bf16(v(2), v(3)), pack_bf16(v(4), v(5)), pack_bf16(v(6), v(7)));
    }
  }
}

// ---- delta[h][s] = sum over channels of d_o o: eight lanes a row ----
template <int D>
__global__ void __launch_bounds__(256) kda_packed_delta_kernel(const __grid_constant__ PackedArgs a) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;
  const int sub = threadIdx.x & 7;
  before_kernel();
  if (!a.list && i < kClearBytes / 4 && sub == 0) a.head[i] = 0;
  float sum = 0.f;
  if (i < a.S * a.Hq) {
    const uint4* const x = reinterpret_cast<const uint4*>(a.o_in + i * D);
    const uint4* const y = reinterpret_cast<const uint4*>(a.d_o + i * D);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint4 u = x[sub + 8 * c], v = y[sub + 8 * c];
      const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = unpack_bf16(us[e]), q = unpack_bf16(vs[e]);
        sum = fmaf(p.x, q.x, sum);
        sum = fmaf(p.y, q.y, sum);
      }
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (sub == 0 && i < a.S * a.Hq) a.delta[(i % a.Hq) * a.S + i / a.Hq] = sum;
}

// ---- dk and dv ----
template <int D>
struct KvCfg {
  static constexpr int kTile = kRows * D * 2;
  static constexpr int kQ = D == 128 ? 3 : 5, kDo = D == 128 ? 2 : 4;  // slots of queries, of d_o
  static constexpr int kBytes = (2 + kQ + kDo) * kTile;
};
template <int D>
struct KvShared {
  alignas(16) float row[KvCfg<D>::kDo][2][kRows];  // -lse (base 2) and -delta of a step's queries, with its d_o
  Handout items;
  uint64_t kv_full, kv_empty;
  uint64_t q_full[5], q_empty[5], do_full[4], do_empty[4];
  uint64_t s_full, dp_full, p_ready, ds_ready, done, acc_free, drain;
  uint32_t tmem;
  int abort_;
};
struct KvItem {
  int64_t slot0;  // of the sequence's first tile in the statistics
  int lo, L, j, nt, hk, head0, heads, part;  // key tile j of nt; query heads head0 .. + heads
  __device__ __forceinline__ int steps() const { return heads * (nt - j); }
};
__device__ __forceinline__ bool item_at(const PackedArgs& a, int tiles, int64_t x, KvItem& it) {
  const int per = a.Hkv * a.split;
  if (x >= static_cast<int64_t>(tiles) * per) return false;
  const Tile t = tile_of(a, tiles, static_cast<int>(x / per));
  const int r = static_cast<int>(x % per);
  it.lo = t.lo;
  it.L = t.L;
  it.slot0 = t.slot(0);
  it.nt = (t.L + kRows - 1) / kRows;
  it.j = it.nt - t.w;
  it.hk = r / a.split;
  it.part = r % a.split;
  it.heads = a.Hq / a.Hkv / a.split;
  it.head0 = it.hk * (a.Hq / a.Hkv) + it.part * it.heads;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kda_packed_dkv_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap domap, const float sc) {
  using C = KvCfg<D>;
  constexpr int kTile = C::kTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const kt = smem;
  uint8_t* const vt = smem + kTile;
  uint8_t* const qt = smem + 2 * kTile;
  uint8_t* const dot = qt + C::kQ * kTile;
  KvShared<D>* const sh = reinterpret_cast<KvShared<D>*>(smem + C::kBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* const ab = &sh->abort_;

  if (smem_addr(smem) & 1023) {
    if (tid == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  if (tid == 0) {
    handout_init(&sh->items, 2 + kMathWarps);
    mbar_init(&sh->kv_full, 1);
    mbar_init(&sh->kv_empty, 1);
    for (int i = 0; i < C::kQ; ++i) {
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->q_empty[i], 1);
    }
    for (int i = 0; i < C::kDo; ++i) {
      mbar_init(&sh->do_full[i], 1);
      mbar_init(&sh->do_empty[i], 1 + kMathWarps);  // the products with d_o, and the rows' lse and delta
    }
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->dp_full, 1);
    mbar_init(&sh->p_ready, kMathWarps);
    mbar_init(&sh->ds_ready, kMathWarps);
    mbar_init(&sh->done, 1);
    mbar_init(&sh->acc_free, kMathWarps);
    mbar_init(&sh->drain, 1);
    sh->abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&sh->tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  before_kernel();
  after_kernel();
  const int tiles = tiles_of(a, kRows);  // 0: lengths that do not fit, no warp has work
  const uint32_t tmem = sh->tmem;
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
  KvItem it;

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ---- loads: a warp for K, V and q, another for d_o ----
    const bool second = warp != kLoadWarp;
    uint64_t* const full = second ? sh->do_full : sh->q_full;
    uint64_t* const empty = second ? sh->do_empty : sh->q_empty;
    uint8_t* const at = second ? dot : qt;
    const int slots = second ? C::kDo : C::kQ;
    Ring r;
    bool ok = true;
    uint32_t items = 0;
    int64_t copies = 0, x = blockIdx.x;
    bool kv = false;  // copies of K and V are in flight, or have been
    for (; item_at(a, tiles, x, it); ++items) {
      if (!second) {
        if (items > 0) ok = ok && wait_all(ab, &sh->kv_empty, (items - 1) & 1, a.status);
        kv = ok;
        if (ok && elect()) {
          mbar_expect_tx(&sh->kv_full, 2 * kTile);
          load_rows<D>(kt, &kmap, it.hk, it.lo + it.j * kRows, &sh->kv_full);
          load_rows<D>(vt, &vmap, it.hk, it.lo + it.j * kRows, &sh->kv_full);
        }
      }
      for (int h = 0; ok && h < it.heads; ++h) {
        for (int m = it.j; m < it.nt; ++m) {
          if (r.turn > 0) ok = wait_all(ab, &empty[r.slot], (r.turn - 1) & 1, a.status);
          if (!ok) break;
          if (elect()) {
            mbar_expect_tx(&full[r.slot], kTile + (second ? sizeof(sh->row[0]) : 0));
            load_rows<D>(at + r.slot * kTile, second ? &domap : &qmap, it.head0 + h, it.lo + m * kRows, &full[r.slot]);
            if (second)
              bulk_load(smem_addr(sh->row[r.slot]), a.stats + ((it.head0 + h) * a.stat_tiles + it.slot0 + m) * 256,
                        sizeof(sh->row[0]), &full[r.slot]);
          }
          ++copies;
          r.next(slots);
        }
      }
      x = second ? handout_take(&sh->items, items + 1)
                 : handout_next(&sh->items, items + 1, &a.tickets[1], ok, static_cast<int64_t>(tiles) * a.Hkv * a.split);
    }
    // after an abort: the copies in flight land before the CTA ends
    if (!ok) {
      for (int64_t p = copies > slots ? copies - slots : 0; p < copies; ++p)
        settle_for(&full[p % slots], static_cast<uint32_t>((p / slots) & 1));
      if (kv) settle_for(&sh->kv_full, (items - 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ---- products, issued by one thread ----
    if (elect()) {
      const uint32_t k_at = desc_k(kt), v_at = desc_k(vt), q_at = desc_k(qt), do_at = desc_k(dot);
      const uint32_t q_mn = desc_mn(qt), do_mn = desc_mn(dot);
      constexpr uint32_t kStep = kTile >> 4;  // from a slot's descriptor to the next
      const uint32_t q_full = smem_addr(sh->q_full), do_full = smem_addr(sh->do_full), p_ready = smem_addr(&sh->p_ready),
                     ds_ready = smem_addr(&sh->ds_ready), acc_free = smem_addr(&sh->acc_free);
      Ring rq, rd;  // of step t
      uint32_t items = 0, turn = 0;
      bool ok = true;
      for (; item_at(a, tiles, handout_take_alone(&sh->items, items), it); ++items) {
        const int steps = it.steps();
        // K and V, the first Q and d_o
        ok = ok && wait3(ab, a.status, smem_addr(&sh->kv_full), items, q_full + 8 * rq.slot, rq.turn, do_full + 8 * rd.slot,
                         rd.turn);
        if (!ok) continue;
        fence_after_sync();
        mma_scores<D>(t_s, k_at, q_at + rq.slot * kStep);
        mma_commit(&sh->s_full);
        mma_scores<D>(t_dp, v_at, do_at + rd.slot * kStep);
        mma_commit(&sh->dp_full);
        if (steps == 1) mma_commit(&sh->kv_empty);
        for (int t = 0; t < steps; ++t, ++turn) {
          const bool more = t + 1 < steps;
          Ring nq = rq, nd = rd;
          nq.next(C::kQ);
          nd.next(C::kDo);
          // P(t), the next Q, and at an item's start the accumulators
          const uint32_t nq_full = more ? q_full + 8 * nq.slot : p_ready, nq_turn = more ? nq.turn : turn;
          const bool first = t == 0 && items > 0;
          ok = wait3(ab, a.status, p_ready, turn, nq_full, nq_turn, first ? acc_free : p_ready, first ? items - 1 : turn);
          if (!ok) break;
          fence_after_sync();
          mma_rows<D, kCols>(t_dv, t_s, do_mn + rd.slot * kStep, t > 0);
          mma_commit(&sh->do_empty[rd.slot]);
          if (more) {
            mma_scores<D>(t_s, k_at, q_at + nq.slot * kStep);
            mma_commit(&sh->s_full);
          }
          // dS(t), the next d_o
          const uint32_t nd_full = more ? do_full + 8 * nd.slot : ds_ready, nd_turn = more ? nd.turn : turn;
          ok = wait3(ab, a.status, ds_ready, turn, nd_full, nd_turn, ds_ready, turn);
          if (!ok) break;
          fence_after_sync();
          mma_rows<D, kCols>(t_dk, t_dp, q_mn + rq.slot * kStep, t > 0);
          mma_commit(&sh->q_empty[rq.slot]);
          if (more) {
            mma_scores<D>(t_dp, v_at, do_at + nd.slot * kStep);
            mma_commit(&sh->dp_full);
            if (t + 2 == steps) mma_commit(&sh->kv_empty);
          } else {
            mma_commit(&sh->done);
          }
          rq = nq;
          rd = nd;
        }
      }
      mma_commit(&sh->drain);
      settle_for(&sh->drain, 0);
    }
    __syncwarp();
  } else if (warp >= kMathWarp) {
    const int wg = (warp - kMathWarp) >> 2, row = tid & 127, mt = tid - 32 * kMathWarp;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t my_s = t_s + lane_base + kCols * wg, my_dp = t_dp + lane_base + kCols * wg;
    const uint64_t sc2 = twice2(sc);
    uint32_t turn = 0, items = 0;
    Ring rq, rd;
    for (; item_at(a, tiles, handout_take(&sh->items, items), it); ++items) {
      const int steps = it.steps();
      int m = it.j;
      for (int t = 0; t < steps; ++t, ++turn) {
        const int past = it.L - m * kRows;       // query rows of the tile from here on are another sequence's
        const bool diagonal = m == it.j, tail = past < kRows;
        if (++m == it.nt) m = it.j;
        const ulonglong2* const lse2 = reinterpret_cast<const ulonglong2*>(sh->row[rd.slot][0] + kCols * wg);
        const ulonglong2* const del2 = reinterpret_cast<const ulonglong2*>(sh->row[rd.slot][1] + kCols * wg);
        // columns (queries) that see this thread's key
        uint32_t see[kParts];
#pragma unroll
        for (int c = 0; c < kParts; ++c) see[c] = ~0u;
        if (diagonal || tail) {
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            const int c0 = kCols * wg + 32 * c, lo = diagonal ? row - c0 : 0, hi = past - c0;
            see[c] = lo >= 32 ? 0u : lo > 0 ? ~0u << lo : ~0u;
            see[c] &= hi >= 32 ? ~0u : hi > 0 ? ~(~0u << hi) : 0u;
          }
        }
        const bool all = !(diagonal || tail);
        wait_both(ab, &sh->do_full[rd.slot], rd.turn & 1, &sh->s_full, turn & 1, a.status);  // lse and delta; S
        if (tail) {  // those rows' Q and d_o to zero, once the scores' products have read them
          wait_all(ab, &sh->dp_full, turn & 1, a.status);
          if (mt < 2 * kRows && row >= past) zero_row<D>(mt < kRows ? qt + rq.slot * kTile : dot + rd.slot * kTile, row);
          fence_async_smem();
        }
        fence_after_sync();
        uint32_t p[kParts][32], x[kParts][32];
        load_scores(my_s, p);
#pragma unroll
        for (int c = 0; c < kParts; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 l = lse2[(32 * c + e) / 4];
            ex2_pair(fma2(pack2(p[c][e], p[c][e + 1]), sc2, l.x), p[c][e], p[c][e + 1]);
            ex2_pair(fma2(pack2(p[c][e + 2], p[c][e + 3]), sc2, l.y), p[c][e + 2], p[c][e + 3]);
          }
        if (!all) hide(p, see);
        store_bf16(my_s, p);
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_ready);
        wait_all(ab, &sh->dp_full, turn & 1, a.status);
        fence_after_sync();
        load_scores(my_dp, x);
#pragma unroll
        for (int c = 0; c < kParts; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 d = del2[(32 * c + e) / 4];
            const float2 g = unpack2(mul2(pack2(p[c][e], p[c][e + 1]), add2(pack2(x[c][e], x[c][e + 1]), d.x)));
            const float2 h = unpack2(mul2(pack2(p[c][e + 2], p[c][e + 3]), add2(pack2(x[c][e + 2], x[c][e + 3]), d.y)));
            x[c][e] = __float_as_uint(g.x);
            x[c][e + 1] = __float_as_uint(g.y);
            x[c][e + 2] = __float_as_uint(h.x);
            x[c][e + 3] = __float_as_uint(h.y);
          }
        if (!all) hide(x, see);
        store_bf16(my_dp, x);
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->ds_ready);
          mbar_arrive(&sh->do_empty[rd.slot]);
        }
        rq.next(C::kQ);
        rd.next(C::kDo);
      }
      const bool fine = wait_all(ab, &sh->done, items & 1, a.status);
      fence_after_sync();
      // this warpgroup's part of the channels of dv and of dk
      constexpr int kCh = D / kGroups;
      const int at = it.j * kRows + row;
      const bool used = fine && at < it.L;
      const int64_t dst = (static_cast<int64_t>(it.lo + at) * a.Hkv + it.hk) * D + wg * kCh;
      const uint32_t acc = lane_base + wg * kCh;
      if (a.split > 1) {
        const int64_t all_rows = a.S * a.Hkv * D;
        write_row<kCh>(t_dv + acc, 1.f, a.part + it.part * all_rows + dst, used);
        write_row<kCh>(t_dk + acc, a.scale, a.part + (a.split + it.part) * all_rows + dst, used);
      } else {
        write_row<kCh>(t_dv + acc, 1.f, a.dv + dst, used);
        write_row<kCh>(t_dk + acc, a.scale, a.dk + dst, used);
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_free);
    }
  } else if (tiles == 0 && a.fresh) {  // the one warp that has no other work
    fill_nan(a.dk, a.S * a.Hkv * (D / 2), lane, 32);
    fill_nan(a.dv, a.S * a.Hkv * (D / 2), lane, 32);
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Sums of the parts of dk and dv, in order.
__global__ void __launch_bounds__(256) kda_packed_parts_kernel(const __grid_constant__ PackedArgs a) {
  const int64_t all = a.S * a.Hkv * a.D;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= 2 * all || tiles_of(a, kRows) == 0) return;
  const int g = i >= all;
  const int64_t at = i - g * all;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < a.split; ++p) {
    const float4 x = *reinterpret_cast<const float4*>(a.part + (g * a.split + p) * all + at);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  *reinterpret_cast<uint2*>((g ? a.dk : a.dv) + at) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// ---- dq, and a better delta for the other pass ----
template <int D>
struct QCfg {
  static constexpr int kTile = kRows * D * 2;
  static constexpr int kK = D == 128 ? 3 : 5, kV = D == 128 ? 2 : 4;  // slots: a tile of K is held for longer
  static constexpr int kBytes = (2 + kK + kV) * kTile;
  static constexpr bool kAhead = D == 128;  // scores are read a tile ahead
};
struct QShared {
  Handout items;
  float sum[kGroups][kRows];  // per row, of each warpgroup's columns
  uint64_t k_full[5], k_empty[5], v_full[4], v_empty[4];
  uint64_t q_full, q_empty;
  // dP and dS by buffer: an item's last dS can be there before the one before it is seen
  uint64_t s_full, s_read, dp_full[2], ds_ready[2], done, acc_free, drain;
  uint32_t tmem;
  int abort_;
};
struct QItem {
  int64_t slot;  // in the statistics
  int lo, L, m, head, hk;  // query tile m: key tiles 0 .. m
};
__device__ __forceinline__ bool item_at(const PackedArgs& a, int tiles, int64_t x, QItem& it) {
  if (x >= static_cast<int64_t>(tiles) * a.Hq) return false;
  const Tile t = tile_of(a, tiles, static_cast<int>(x / a.Hq));
  it.lo = t.lo;
  it.L = t.L;
  it.m = t.w - 1;
  it.slot = t.slot(it.m);
  it.head = static_cast<int>(x % a.Hq);
  it.hk = it.head / (a.Hq / a.Hkv);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kda_packed_dq_kernel(const __grid_constant__ PackedArgs a, const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ CUtensorMap domap, const float sc) {
  using C = QCfg<D>;
  constexpr int kTile = C::kTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const kt = smem + 2 * kTile;  // behind the tiles of q and d_o
  uint8_t* const vt = kt + C::kK * kTile;
  QShared* const sh = reinterpret_cast<QShared*>(smem + C::kBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* const ab = &sh->abort_;

  if (smem_addr(smem) & 1023) {
    if (tid == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  if (tid == 0) {
    handout_init(&sh->items, 2 + kMathWarps);
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(&sh->v_full[i], 1);
      mbar_init(&sh->v_empty[i], 1);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->s_read, kMathWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->dp_full[i], 1);
      mbar_init(&sh->ds_ready[i], kMathWarps);
    }
    mbar_init(&sh->done, 1);
    mbar_init(&sh->acc_free, kMathWarps);
    mbar_init(&sh->drain, 1);
    sh->abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&sh->tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  before_kernel();
  after_kernel();
  const int tiles = tiles_of(a, kRows);  // 0: lengths that do not fit, no warp has work
  const uint32_t tmem = sh->tmem;
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dq = tmem + 384;  // dP at t_dp and t_dp + 128 in turn
  QItem it;

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    registers_down<kFewRegs>();
    // ---- loads: a warp for q, d_o and K, another for V: neither waits for the other's slots ----
    const bool v = warp != kLoadWarp;
    uint64_t* const full = v ? sh->v_full : sh->k_full;
    uint64_t* const empty = v ? sh->v_empty : sh->k_empty;
    uint8_t* const at = v ? vt : kt;
    const int slots = v ? C::kV : C::kK;
    Ring r;
    bool ok = true;
    uint32_t items = 0;
    int64_t copies = 0, x = blockIdx.x;
    bool rows = false;  // copies of q and d_o are in flight, or have been
    for (; item_at(a, tiles, x, it); ++items) {
      if (!v) {
        if (items > 0) ok = ok && wait_all(ab, &sh->q_empty, (items - 1) & 1, a.status);
        rows = ok;
        if (ok && elect()) {
          mbar_expect_tx(&sh->q_full, 2 * kTile);
          load_rows<D>(smem, &qmap, it.head, it.lo + it.m * kRows, &sh->q_full);
          load_rows<D>(smem + kTile, &domap, it.head, it.lo + it.m * kRows, &sh->q_full);
        }
      }
      for (int j = 0; j <= it.m; ++j) {
        if (r.turn > 0) ok = ok && wait_all(ab, &empty[r.slot], (r.turn - 1) & 1, a.status);
        if (!ok) break;
        if (elect()) {
          mbar_expect_tx(&full[r.slot], kTile);
          load_rows<D>(at + r.slot * kTile, v ? &vmap : &kmap, it.hk, it.lo + j * kRows, &full[r.slot]);
        }
        ++copies;
        r.next(slots);
      }
      x = v ? handout_take(&sh->items, items + 1)
            : handout_next(&sh->items, items + 1, &a.tickets[0], ok, static_cast<int64_t>(tiles) * a.Hq);
    }
    if (!ok) {
      for (int64_t p = copies > slots ? copies - slots : 0; p < copies; ++p)
        settle_for(&full[p % slots], static_cast<uint32_t>((p / slots) & 1));
      if (rows) settle_for(&sh->q_full, (items - 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    registers_down<kFewRegs>();
    // ---- products, issued by one thread ----
    if (elect()) {
      const uint32_t q_at = desc_k(smem), do_at = desc_k(smem + kTile), k_at = desc_k(kt), v_at = desc_k(vt),
                     k_mn = desc_mn(kt);
      constexpr uint32_t kStep = kTile >> 4;  // from a slot's descriptor to the next
      const uint32_t k_full = smem_addr(sh->k_full), v_full = smem_addr(sh->v_full), ds_full = smem_addr(sh->ds_ready),
                     s_read = smem_addr(&sh->s_read), acc_free = smem_addr(&sh->acc_free);
      Ring rk, ks, vs;  // K(j); K and V of the next scores
      uint32_t items = 0, turn = 0;
      bool ok = true;
      auto scores = [&](uint32_t n, bool last) {  // S and dP of the CTA's n-th tile
        mma_scores<D>(t_s, q_at, k_at + ks.slot * kStep);
        mma_commit(&sh->s_full);
        mma_scores<D>(t_dp + 128 * (n & 1), do_at, v_at + vs.slot * kStep);
        mma_commit(&sh->dp_full[n & 1]);
        mma_commit(&sh->v_empty[vs.slot]);
        if (last) mma_commit(&sh->q_empty);
        ks.next(C::kK);
        vs.next(C::kV);
      };
      for (; item_at(a, tiles, handout_take_alone(&sh->items, items), it); ++items) {
        ok = ok && wait3(ab, a.status, smem_addr(&sh->q_full), items, k_full + 8 * ks.slot, ks.turn, v_full + 8 * vs.slot,
                         vs.turn);
        if (!ok) continue;
        fence_after_sync();
        scores(turn, it.m == 0);
        // S has one buffer: the next scores can be formed once every warp has read the
        // last. Where they are read a tile ahead, dq(j), S(j + 2) and dP(j + 2) are one
        // batch behind one wait; else S(j + 1) and dP(j + 1) come before dq(j).
        auto next = [&](uint32_t bar, uint32_t par, uint32_t n, bool last) {
          ok = wait3(ab, a.status, bar, par, k_full + 8 * ks.slot, ks.turn, v_full + 8 * vs.slot, vs.turn);
          if (!ok) return;
          fence_after_sync();
          scores(n, last);
        };
        if (C::kAhead && it.m > 0) next(s_read, items, turn + 1, it.m == 1);
        for (int j = 0; ok && j <= it.m; ++j, ++turn) {
          if (!C::kAhead && j < it.m) next(s_read, turn, turn + 1, j + 1 == it.m);
          const bool more = C::kAhead && j + 2 <= it.m;
          const uint32_t ds = ds_full + 8 * (turn & 1), par = turn >> 1;
          ok = ok && wait3(ab, a.status, ds, par, more ? k_full + 8 * ks.slot : ds, more ? ks.turn : par,
                           more ? v_full + 8 * vs.slot : ds, more ? vs.turn : par);
          if (j == 0 && items > 0)
            ok = ok && wait3(ab, a.status, acc_free, items - 1, acc_free, items - 1, acc_free, items - 1);
          if (!ok) break;
          fence_after_sync();
          mma_rows<D, kCols>(t_dq, t_dp + 128 * (turn & 1), k_mn + rk.slot * kStep, j > 0);
          mma_commit(&sh->k_empty[rk.slot]);
          if (j == it.m) mma_commit(&sh->done);
          rk.next(C::kK);
          if (more) scores(turn + 2, j + 2 == it.m);
        }
      }
      mma_commit(&sh->drain);
      settle_for(&sh->drain, 0);
    }
    __syncwarp();
  } else if (warp < kMathWarp) {
    registers_down<kFewRegs>();
    if (tiles == 0 && a.fresh) fill_nan(a.dq, a.S * a.Hq * (D / 2), lane, 32);
  } else {
    registers_up<kManyRegs>();
    const int wg = (warp - kMathWarp) >> 2, row = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t my_s = t_s + lane_base + kCols * wg;
    const uint64_t sc2 = twice2(sc);
    uint32_t turn = 0, items = 0;
    Ring rk;
    // a row's sum over all warpgroups' columns
    auto together = [&](float x) {
      sh->sum[wg][row] = x;
      named_bar_sync(1, 32 * kMathWarps);
      x = sh->sum[0][row];
#pragma unroll
      for (int i = 1; i < kGroups; ++i) x += sh->sum[i][row];
      named_bar_sync(1, 32 * kMathWarps);
      return x;
    };
    for (; item_at(a, tiles, handout_take(&sh->items, items), it); ++items) {
      const int at = it.m * kRows + row;
      const bool used = at < it.L;
      const int64_t stat = static_cast<int64_t>(it.head) * a.S + it.lo + at;
      const uint64_t lse2 = twice2(used ? a.lse[stat] * -1.4426950408889634f : 0.f);
      float delta = used ? a.delta[stat] : 0.f;
      // What a row's dS sums to, over all keys: zero but for the rounding of the o
      // that delta was formed from.
      uint64_t rest2[2] = {0, 0};
      uint32_t p[kParts][32], x[kParts][32];  // scores, then probabilities; dP, then dS
      auto read_scores = [&](uint32_t n) {
        wait_voting(ab, &sh->s_full, n & 1, a.status);
        fence_after_sync();
        load_scores(my_s, p);
      };
      auto scores_read = [&]() {
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->s_read);
      };
      if (C::kAhead) {
        read_scores(turn);
        scores_read();
      }
      for (int j = 0; j <= it.m; ++j, ++turn) {
        const uint32_t my_dp = t_dp + 128 * (turn & 1) + lane_base + kCols * wg;
        const bool diagonal = j == it.m;
        uint32_t see[kParts];  // keys that this thread's query sees
#pragma unroll
        for (int c = 0; c < kParts; ++c) see[c] = ~0u;
        if (diagonal) {
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            const int hi = (used ? row + 1 : 0) - (kCols * wg + 32 * c);
            see[c] = hi >= 32 ? ~0u : hi > 0 ? ~(~0u << hi) : 0u;
          }
        }
        if (!C::kAhead) {
          read_scores(turn);
          scores_read();
        }
#pragma unroll
        for (int c = 0; c < kParts; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) ex2_pair(fma2(pack2(p[c][e], p[c][e + 1]), sc2, lse2), p[c][e], p[c][e + 1]);
        if (diagonal) hide(p, see);
        if (diagonal && it.L - j * kRows < kRows) {  // rows of K past the sequence to zero: S has read them
          if (wg == 0 && at >= it.L) zero_row<D>(kt + rk.slot * kTile, row);
          fence_async_smem();
        }
        wait_voting(ab, &sh->dp_full[turn & 1], turn >> 1 & 1, a.status);
        fence_after_sync();
        load_scores(my_dp, x);
        if (it.m == 0) {
          // All keys in one tile: delta as the sum that it is, free of o's rounding. A
          // sequence's first query sees one key, with probability 1 but for the rounding of
          // lse: made exact, its dS is zero.
          hide(x, see);
          if (at == 0 && wg == 0 && p[0][0] < 0x7f800000u) p[0][0] = __float_as_uint(1.f);
          uint64_t sum = 0;
#pragma unroll
          for (int c = 0; c < kParts; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) sum = fma2(pack2(p[c][e], p[c][e + 1]), pack2(x[c][e], x[c][e + 1]), sum);
          const float2 s = unpack2(sum);
          delta = together(s.x + s.y);
        }
        const uint64_t delta2 = twice2(-delta);
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 g = unpack2(mul2(pack2(p[c][e], p[c][e + 1]), add2(pack2(x[c][e], x[c][e + 1]), delta2)));
            x[c][e] = __float_as_uint(g.x);
            x[c][e + 1] = __float_as_uint(g.y);
          }
        }
        if (diagonal) hide(x, see);
        store_bf16(my_dp, x);
#pragma unroll
        for (int c = 0; c < kParts; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) rest2[e / 2 & 1] = add2(rest2[e / 2 & 1], pack2(x[c][e], x[c][e + 1]));
        // One arrival then stands for dS and for the next scores, and the issuing thread
        // has one wait a tile. (Heads of 64, whose products are half as long, lose by it.)
        if (C::kAhead && !diagonal) read_scores(turn + 1);
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->ds_ready[turn & 1]);
        rk.next(C::kK);
      }
      {
        const float2 s = unpack2(add2(rest2[0], rest2[1]));
        const float rest = together(s.x + s.y);
        if (wg == 0) {
          float* const to = a.stats + (it.head * a.stat_tiles + it.slot) * 256 + row;
          to[0] = unpack2(lse2).x;
          to[kRows] = used ? -(delta + rest) : 0.f;
        }
      }
      const bool fine = wait_voting(ab, &sh->done, items & 1, a.status);
      fence_after_sync();
      constexpr int kCh = D / kGroups;
      write_row<kCh>(t_dq + lane_base + wg * kCh, a.scale,
                     a.dq + (static_cast<int64_t>(it.lo + at) * a.Hq + it.head) * D + wg * kCh, used && fine);
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_free);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const PackedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   const CUtensorMap& d_o, cudaStream_t s) {
  const size_t smem_kv = KvCfg<D>::kBytes + sizeof(KvShared<D>), smem_q = QCfg<D>::kBytes + sizeof(QShared);
  static PerDevice kept_kv, kept_q;
  int64_t sms = 0;
  cudaError_t e = packed_sms(kept_kv, kda_packed_dkv_kernel<D>, smem_kv, &sms);
  if (e == cudaSuccess) e = packed_sms(kept_q, kda_packed_dq_kernel<D>, smem_q, &sms, kLaunchRegs);
  if (e != cudaSuccess) return e;
  if (sms > kPackedMaxCtas) sms = kPackedMaxCtas;
  const float sc = a.scale * 1.4426950408889634f;
  const int64_t tiles = a.S / kRows + a.N, kv = tiles * a.Hkv * a.split, nq = tiles * a.Hq;
  kda_packed_delta_kernel<D><<<static_cast<unsigned>((a.S * a.Hq * 8 + 255) / 256), 256, 0, s>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_after(kda_packed_dq_kernel<D>, nq < sms ? nq : sms, kThreads, smem_q, s, a, q, k, v, d_o, sc);
  if (e == cudaSuccess)
    e = launch_after(kda_packed_dkv_kernel<D>, kv < sms ? kv : sms, kThreads, smem_kv, s, a, q, k, v, d_o, sc);
  if (e == cudaSuccess && a.split > 1) {
    kda_packed_parts_kernel<<<static_cast<unsigned>((2 * a.S * a.Hkv * a.D / 4 + 255) / 256), 256, 0, s>>>(a);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

cudaError_t launch_packed_bwd(const PackedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              const CUtensorMap& d_o, cudaStream_t s) {
  return a.D == 128 ? launch<128>(a, q, k, v, d_o, s) : launch<64>(a, q, k, v, d_o, s);
}

}  // namespace kda
