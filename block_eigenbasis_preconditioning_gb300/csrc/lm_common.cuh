// Helpers of the language-model operators (lm_*.cu).
#pragma once

#include <climits>
#include <cmath>

#include "common.cuh"

namespace dobb {
namespace lm {

// Token index i of an int32 or int64 array.
__device__ __forceinline__ int64_t load_token(const void* tokens, int token_bytes, int64_t i) {
  return token_bytes == 8 ? static_cast<const int64_t*>(tokens)[i]
                          : static_cast<const int32_t*>(tokens)[i];
}

inline bool bad_dtype(int d) { return d != DOBB_F32 && d != DOBB_BF16; }
inline bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
inline size_t dtype_bytes(int d) { return d == DOBB_F32 ? 4 : 2; }

}  // namespace lm
}  // namespace dobb
