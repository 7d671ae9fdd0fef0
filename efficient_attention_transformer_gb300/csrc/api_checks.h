// Argument checks that the C entry points of the operators around the layer
// share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "flash_gau_internal.h"

namespace flashgau {

inline bool io_type(int dtype) { return dtype == FLASH_GAU_FP32 || dtype == FLASH_GAU_BF16; }

inline bool aligned(const void *p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

struct Span {
  const void *p;
  size_t n;
};
inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// Outputs apart from one another, and from inputs unless the same array
// (`same`: both of it) where that is allowed.
template <int NO, int NI>
bool separate(const Span (&out)[NO], const Span (&in)[NI], bool same) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return false;
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j]) && !(same && out[i].p == in[j].p && out[i].n == in[j].n))
        return false;
  }
  return true;
}

inline int status_of(cudaError_t err) {
  return err == cudaSuccess ? FLASH_GAU_OK : record_cuda(err);
}

}  // namespace flashgau
