// Argument checks that the C entry points share.
#pragma once

#include <stdint.h>

#include "../../include/prism.h"

namespace prism {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int N>
int check_pointers(const void* const (&required)[N], const void* const* optional, int n) {
  for (const void* p : required)
    if (!p) return PRISM_ERR_INVALID_ARG;
  for (const void* p : required)
    if (!aligned(p, 16)) return PRISM_ERR_MISALIGNED;
  for (int i = 0; i < n; ++i)
    if (optional[i] && !aligned(optional[i], 16)) return PRISM_ERR_MISALIGNED;
  return PRISM_OK;
}

// Arrays that are read by the word: log_decay, positions, seq_lens, slots.
inline int check_words(const void* a, const void* b) {
  return aligned(a, 4) && aligned(b, 4) ? PRISM_OK : PRISM_ERR_MISALIGNED;
}

inline int elem_bytes(prism_dtype t) { return t == PRISM_F32 ? 4 : 2; }

// Strides of an input whose tokens are `row` contiguous elements, as sequence and token steps;
// contiguous where given as 0.  A step that is never taken (one sequence, one token) is replaced by
// the contiguous one.
inline int resolve(const long long given[2], int B, int T, long long row, prism_dtype t, long long (&out)[2]) {
  const long long unit = 16 / elem_bytes(t);
  out[1] = given[1] == 0 || T == 1 ? row : given[1];
  out[0] = given[1] == 0 || B == 1 ? T * out[1] : given[0];
  if (out[1] < row || out[0] <= 0 || out[1] % unit || out[0] % unit) return PRISM_ERR_INVALID_ARG;
  return PRISM_OK;
}

}  // namespace prism
