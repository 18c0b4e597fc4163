// kda_span.h -- which memory a call touches, and whether two parts of it meet.
// Host code without CUDA or torch.
#pragma once

#include <stdint.h>

namespace kda {

// `rows` runs of `bytes` each, `step` bytes from one to the next (step >= bytes).
struct Span {
  const char* name;
  uintptr_t at;
  int64_t rows, bytes, step;
};
inline Span whole(const char* name, const void* p, int64_t bytes) {
  return {name, reinterpret_cast<uintptr_t>(p), 1, bytes, bytes};
}

// Whether a span of one run shares a byte with another span. Exact: what lies
// between the runs of a strided one is not part of it.
inline bool meet(const Span& one, const Span& x) {
  if (one.rows == 0 || one.bytes == 0 || x.rows == 0 || x.bytes == 0) return false;
  const uintptr_t end = one.at + static_cast<uintptr_t>(one.bytes);
  if (end <= x.at) return false;
  // the first run that ends behind the start of `one`
  int64_t i = 0;
  if (one.at >= x.at + static_cast<uintptr_t>(x.bytes))
    i = static_cast<int64_t>((one.at - x.at - static_cast<uintptr_t>(x.bytes)) / static_cast<uintptr_t>(x.step)) + 1;
  return i < x.rows && x.at + static_cast<uintptr_t>(i) * static_cast<uintptr_t>(x.step) < end;
}

}  // namespace kda
