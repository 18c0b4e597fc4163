// kda_packed.cuh -- what the kernels of causal attention over packed sequences
// share: their arguments, the list of row tiles, waits, and tensor maps.
#pragma once

#include "kda_attention.cuh"
#include "kda_blocks.h"
#include "kda_device.cuh"

namespace kda {

constexpr int kPackedMaxSeqs = 65536;
constexpr int kPackedMaxCtas = 152;  // one per SM

struct PackedArgs {
  const int32_t* cu;
  int* head;           // of the workspace: a status word, and the tickets
  int* status;         // the call's status word: the head's, or the caller's
  int* tickets;        // items handed out, by kernel (zeroed before the call's first)
  const int* list;     // count, then from list + 4 on {first token, length, weight, sequence} of each tile; null: one sequence
  int64_t S;
  int N, Hq, Hkv, D;
  float scale;
  __nv_bfloat16 *o, *dq, *dk, *dv;   // contiguous
  const __nv_bfloat16 *o_in, *d_o;
  float* lse;          // [Hq][S]
  float* delta;        // [Hq][S]
  float* stats;        // [Hq][stat_tiles][2][128]: -lse in base 2 and -delta of each tile's rows, zero past its sequence
  int64_t stat_tiles;
  float* part;         // gradients of k and v by parts of the head group: [2][split][S][Hkv][D]
  int split;
  int clears;          // forward of one short sequence: the kernel itself clears the header
  int fresh;           // outputs to fill where cu_seqlens is refused: 1 o, 2 lse; of the backward 1 all
};
constexpr int kClearBytes = 32;  // of the workspace's header: the status word, and the tickets

// A tile of `rows` rows of a sequence. Weight w counts the tiles up to it: it
// is tile w - 1 from the sequence's start (or, for work that goes to the
// sequence's end, w tiles from there).
struct Tile {
  int lo, L, w, n;
  // place of tile m of the sequence among all sequences' tiles of 128 rows
  __device__ __forceinline__ int64_t slot(int m) const { return static_cast<int64_t>(lo) / 128 + n + m; }
};

// Tiles of the call, heaviest first, so that the last ones to be handed out are
// short. 0: lengths that do not fit (recorded).
__device__ __forceinline__ int tiles_of(const PackedArgs& a, int rows) {
  if (a.list) return a.list[0];
  if (a.cu[0] != 0 || a.cu[1] != a.S) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(a.status, KDA_ERR_DEVICE_CHECK);
    return 0;
  }
  return static_cast<int>((a.S + rows - 1) / rows);
}
__device__ __forceinline__ Tile tile_of(const PackedArgs& a, int tiles, int e) {
  if (!a.list) return {0, static_cast<int>(a.S), tiles - e, 0};
  const int4 t = reinterpret_cast<const int4*>(a.list + 4)[e];
  return {t.x, t.y, t.z, t.w};
}
// NaN (of either type) all over an output, by all CTAs: thread i of n in each. Work for
// warps that have none: in front of the roles it would cost them registers.
__device__ __forceinline__ void fill_nan(void* p, int64_t words, int i, int n) {
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * n + i; w < words; w += static_cast<int64_t>(gridDim.x) * n)
    static_cast<uint32_t*>(p)[w] = 0x7fc07fc0u;
}
namespace tc {

// Whether a phase, or up to three of them, are over.
__device__ __forceinline__ bool poll(uint32_t a, uint32_t p) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(a), "r"(p & 1)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool poll2(uint32_t a0, uint32_t p0, uint32_t a1, uint32_t p1) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      "and.pred p, p, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(a0), "r"(p0 & 1), "r"(a1), "r"(p1 & 1)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool poll3(uint32_t a0, uint32_t p0, uint32_t a1, uint32_t p1, uint32_t a2, uint32_t p2) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p, q, r;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n"
      "and.pred p, p, q;\nand.pred p, p, r;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(a0), "r"(p0 & 1), "r"(a1), "r"(p1 & 1), "r"(a2), "r"(p2 & 1)
      : "memory");
  return ok != 0;
}

// Bounded wait: false when it ran out (the CTA's abort flag is then set) or another
// role gave up. After an abort every role still walks through its items, but issues
// no copy and no product any more. `over`: whether what is waited for has happened.
template <typename F>
__device__ __forceinline__ bool wait_for(int* abort_, int* status, const F& over) {
  for (int it = 0; it < (1 << 22); ++it) {
    if (over()) return true;
    if ((it & 15) == 15 && *const_cast<volatile int*>(abort_)) return false;
  }
  *const_cast<volatile int*>(abort_) = 1;
  set_status(status, KDA_ERR_TIMEOUT);
  return false;
}
// By a whole warp, with one answer, for one phase or for two.
__device__ __forceinline__ bool wait_all(int* abort_, uint64_t* bar, uint32_t parity, int* status) {
  const uint32_t at = smem_addr(bar);
  return __all_sync(~0u, wait_for(abort_, status, [&]() { return poll(at, parity); }));
}
// The same with a vote at every look. Measured either way: dq's arithmetic is faster
// with it (heads of 64: 182 us against 187), that of dk and dv without (heads of 128:
// 1214 against 1237).
__device__ __forceinline__ bool wait_voting(int* abort_, uint64_t* bar, uint32_t parity, int* status) {
  const uint32_t at = smem_addr(bar);
  for (int it = 0; it < (1 << 22); ++it) {
    if (__all_sync(~0u, poll(at, parity))) return true;
    if ((it & 15) == 15 && __any_sync(~0u, *const_cast<volatile int*>(abort_))) return false;
  }
  *const_cast<volatile int*>(abort_) = 1;
  set_status(status, KDA_ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool wait_both(int* abort_, uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, int* status) {
  const uint32_t a0 = smem_addr(b0), a1 = smem_addr(b1);
  return __all_sync(~0u, wait_for(abort_, status, [&]() { return poll2(a0, p0, a1, p1); }));
}
// By the one thread that issues the products, for up to three phases at once (given
// twice where there are fewer): its instructions between two products are time in
// which the tensor cores run dry, since it is held up by the products themselves
// until few of them are left.
__device__ __forceinline__ bool wait3(int* abort_, int* status, uint32_t a0, uint32_t p0, uint32_t a1, uint32_t p1,
                                      uint32_t a2, uint32_t p2) {
  return wait_for(abort_, status, [&]() { return poll3(a0, p0, a1, p1, a2, p2); });
}

// Waits, at most so long, without giving up; whether the phase is over.
__device__ __forceinline__ bool settle_for(uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_addr(bar);
  for (int it = 0; it < (1 << 20); ++it)
    if (poll(at, parity)) return true;
  return false;
}

// A warpgroup's registers a thread, of those that the block was launched with. Called by all its warps,
// in the branch that they take.
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Hands items to the CTA's warps. The first is the CTA's own number, every
// further one the next that no CTA has taken, heaviest first: the order decides
// when an item is worked on, not what comes out. One warp fetches a number when
// it has issued the copies of the item before (earlier, and an item would be
// taken long before its turn), and passes it on through two slots. These waits look at no
// abort flag, so that every warp sees the same items whatever happens; after an
// abort the fetching warp passes on the end.
struct Handout {
  uint64_t full[2], empty[2];
  int64_t item[2];
};
constexpr int64_t kNoItem = INT64_MAX;
__device__ __forceinline__ void handout_init(Handout* h, int warps) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&h->full[i], 1);
    mbar_init(&h->empty[i], warps);
  }
}
__device__ __forceinline__ void settle_long(uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < 64; ++i)
    if (settle_for(bar, parity)) return;
}
// The CTA's n-th item, by one of the warps that are passed it.
__device__ __forceinline__ int64_t handout_take(Handout* h, uint32_t n) {
  if (n == 0) return blockIdx.x;
  const int slot = (n - 1) & 1;
  settle_long(&h->full[slot], (n - 1) >> 1 & 1);
  const int64_t x = *const_cast<volatile int64_t*>(&h->item[slot]);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&h->empty[slot]);
  return x;
}
// The same by a single thread that stands for its warp.
__device__ __forceinline__ int64_t handout_take_alone(Handout* h, uint32_t n) {
  if (n == 0) return blockIdx.x;
  const int slot = (n - 1) & 1;
  settle_long(&h->full[slot], (n - 1) >> 1 & 1);
  const int64_t x = *const_cast<volatile int64_t*>(&h->item[slot]);
  mbar_arrive(&h->empty[slot]);
  return x;
}
// Passes on item n > 0, by the fetching warp.
__device__ __forceinline__ void handout_give(Handout* h, uint32_t n, int64_t x) {
  const int slot = (n - 1) & 1;
  if (n > 2) settle_long(&h->empty[slot], (((n - 1) >> 1) - 1) & 1);
  if ((threadIdx.x & 31) == 0) {
    *const_cast<volatile int64_t*>(&h->item[slot]) = x;
    mbar_arrive(&h->full[slot]);
  }
  __syncwarp();
}

// The next of the call's items, fetched and passed on as number n.
__device__ __forceinline__ int64_t handout_next(Handout* h, uint32_t n, int* ticket, bool ok, int64_t items) {
  int64_t x = kNoItem;
  if (ok && items > gridDim.x) {
    int i = 0;
    if ((threadIdx.x & 31) == 0) i = atomicAdd(ticket, 1);
    x = static_cast<int64_t>(gridDim.x) + __shfl_sync(~0u, i, 0);
  }
  handout_give(h, n, x);
  return x;
}

// A ring's position: slot, and the parity of its turn.
struct Ring {
  int slot = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      ++turn;
    }
  }
};

// 128 rows of one head, from token `tok` on (rows past the tensor are zeros):
// a block of 128 x 128 swizzled bytes for each 64 channels.
template <int D>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, int head, int tok, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * 16384, map, c * 64, head, tok, bar);
}

// Matrix descriptors of such tiles, in two words: the lower is an address plus
// constants that never carry, so that a step costs the issuing thread one
// addition. (It shares its scheduler with two warps of arithmetic: descriptors
// formed anew for each product took it longer than the product.)
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(const void* tile) { return (smem_addr(tile) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(const void* tile) { return (smem_addr(tile) >> 4) | ((128u * 128u >> 4) << 16); }
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t bytes) { return pack2(lo + (bytes >> 4), kDescHi); }
__host__ __device__ constexpr uint32_t k_step(int k) { return (k >> 2) * 128 * 128 + (k & 3) * 32; }
constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);  // of an instruction: bf16 A and B

// D = A B^T: A and B 128 rows of D in shared memory (desc_k).
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int k = 0; k < D / 16; ++k) mma(d, desc_at(a, k_step(k)), desc_at(b, k_step(k)), idesc(128, 128) | kBf16, k > 0);
}
// D (+)= A B: A 128 columns of bf16 in TMEM, packed over the first half of each
// run of `run` fp32 columns (128: all in one place), B 128 rows of D in shared
// memory (desc_mn).
template <int D, int run>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  constexpr int each = run / 16;  // steps of a run
#pragma unroll
  for (int k = 0; k < 8; ++k)
    mma_ta(d, a + run * (k / each) + 8 * (k % each), desc_at(b, k * 2048), idesc(128, D, false, true) | kBf16, k > 0 ? 1u : acc);
}

// Zeros in the rows of such a tile from `from` on, by threads 0 .. 127 of `row`.
template <int D>
__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll
  for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(tile + sw128_chunk(row, c, 128)) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace tc

// [S][heads][D] bf16 as (channel, head, token), boxes of 64 channels of 128 tokens of one head.
inline bool rows_map(CUtensorMap* m, const void* base, int64_t S, int heads, int D, int64_t stride) {
  const EncodeFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)S};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t boxes[3] = {64, 1, 128}, ones[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device for a kernel's grid, with its shared memory allowed. A kernel
// that splits its registers between its warpgroups has to be launched with `regs`: with
// fewer, a warpgroup would wait for its share for ever.
template <typename K>
cudaError_t packed_sms(PerDevice& kept, K kernel, size_t smem, int64_t* sms, int regs = 0) {
  return kept.get(sms, [&](int dev, int64_t* n) {
    cudaFuncAttributes built;
    const cudaError_t read = regs > 0 ? cudaFuncGetAttributes(&built, kernel) : cudaSuccess;
    if (read != cudaSuccess) return read;
    if (regs > 0 && built.numRegs < regs) return cudaErrorInvalidConfiguration;
    const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    int count = 0;
    const cudaError_t got = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
    *n = count;
    return set != cudaSuccess ? set : got;
  });
}

cudaError_t launch_packed_fwd(const PackedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              cudaStream_t s);
cudaError_t launch_packed_bwd(const PackedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              const CUtensorMap& d_o, cudaStream_t s);

}  // namespace kda
