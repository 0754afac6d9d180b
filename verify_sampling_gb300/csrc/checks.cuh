// Argument checks shared by the entry points.
#pragma once

#include <cstddef>
#include <cstdint>

#include "spec.h"

namespace spec {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool valid_dtype(int d) { return d == SPEC_F32 || d == SPEC_BF16; }
inline size_t dtype_size(int d) { return d == SPEC_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return SPEC_OK;
  if (!ws || have < need) return SPEC_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SPEC_ERR_ALIGNMENT;
  return SPEC_OK;
}

}  // namespace spec
