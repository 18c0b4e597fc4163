// kda_paged.cuh -- what the paged cache's host side and its attention kernels share.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// Sequences of one call: every CTA adds up their lengths when it plans its work.
constexpr int kPagedMaxSeqs = 65536;

struct PagedArgs {
  const void *q, *k, *v;
  void* o;
  int* status;
  void* scratch;
  const int32_t *cu, *table, *lens;
  int64_t S, pages;
  int N, Hq, Hkv, D, page, width;
  float scale;
};

size_t paged_attention_scratch_bytes(const PagedArgs& a);
kda_status launch_paged_attention(const PagedArgs& a, cudaStream_t s);

}  // namespace kda
