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

// ---- pairs of fp32 values in one 64-bit register (sm_100 packed arithmetic)
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 2^x (a few units of 2^-23 of the result; results below 2^-126 are 0)
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// max that gives NaN if either operand is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 bytes of fp32 or bf16 values
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint4 fill_neg_inf() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  // largest of all values of n vectors, NaN if there is one
  template <int U>
  static __device__ __forceinline__ float max_of(const uint4 (&v)[U]) {
    float m = __uint_as_float(v[0].x);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m = max_nan(max_nan(max_nan(m, __uint_as_float(v[u].x)), __uint_as_float(v[u].y)),
                  max_nan(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
    }
    return m;
  }
  // entries 2 i and 2 i + 1 of a vector
  static __device__ __forceinline__ void put(uint4& v, int i, float lo, float hi) {
    (i == 0 ? v.x : v.z) = __float_as_uint(lo);
    (i == 0 ? v.y : v.w) = __float_as_uint(hi);
  }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ uint64_t pair(const uint4& v, int i) {
    return i == 0 ? pack2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : pack2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint4 fill_neg_inf() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  template <int U>
  static __device__ __forceinline__ float max_of(const uint4 (&v)[U]) {
    uint32_t m = v[0].x;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m = max_nan_bf16x2(m, max_nan_bf16x2(max_nan_bf16x2(v[u].x, v[u].y), max_nan_bf16x2(v[u].z, v[u].w)));
    }
    return max_nan(bf16_lo(m), bf16_hi(m));
  }
  static __device__ __forceinline__ void put(uint4& v, int i, float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = *reinterpret_cast<const uint32_t*>(&b);
  }
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
    return (i & 1) ? bf16_hi(w) : bf16_lo(w);
  }
  static __device__ __forceinline__ uint64_t pair(const uint4& v, int i) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return pack2(bf16_lo(w), bf16_hi(w));
  }
};

// Elements of [p, p + n) before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
  const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int64_t)sizeof(T);
  return h < n ? h : n;
}

// (Plain loads: the callers may write the same tensor, each thread its own part.)
// The 16 bytes at p, of which [floor16(p), floor16(p) + 32) may be read: two
// aligned loads, shifted by the (warp-uniform) misalignment s = p mod 16 > 0.
__device__ __forceinline__ uint4 load_shifted16(const void* p, uint32_t s) {
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - s);
  const uint4 a = q[0], b = q[1];
  uint32_t w[6] = {a.x, a.y, a.z, a.w, b.x, b.y};
  if (s & 8) {
    w[0] = a.z;
    w[1] = a.w;
    w[2] = b.x;
    w[3] = b.y;
    w[4] = b.z;
    w[5] = b.w;
  }
  if (s & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (s & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 bytes of T at p + i, nothing outside [p, p + n) read; s: the
// misalignment of p + i, the same for the whole warp.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* p, int64_t i, int64_t n, uint32_t s) {
  constexpr int N = 16 / (int)sizeof(T);
  if (s == 0) return *reinterpret_cast<const uint4*>(p + i);
  const int64_t before = s / (uint32_t)sizeof(T);
  if (i >= before && i - before + 2 * N <= n) return load_shifted16(p + i, s);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (sizeof(T) == 4) {
      w[k] = reinterpret_cast<const uint32_t*>(p + i)[k];
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p + i) + 2 * k;
      w[k] = h[0] | ((uint32_t)h[1] << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

inline bool bad_dtype(int d) { return d != DOBB_F32 && d != DOBB_BF16; }
inline bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
inline size_t dtype_bytes(int d) { return d == DOBB_F32 ? 4 : 2; }

// A matrix in memory: `rows` rows of `width` bytes, `stride` bytes apart (width <= stride if rows > 1).
struct RowExtent {
  RowExtent(const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype)
      : at(reinterpret_cast<uintptr_t>(p)), rows(rows), width((uint64_t)cols * dtype_bytes(dtype)),
        stride(rows > 1 ? (uint64_t)stride * dtype_bytes(dtype) : width) {}
  uintptr_t at;
  int64_t rows;
  uint64_t width, stride;
  uintptr_t end() const { return at + (uint64_t)(rows - 1) * stride + width; }
};

// Whether two matrices (rows, width > 0) share a byte: columns of one buffer
// may lie side by side.
inline bool rows_overlap(const RowExtent& x, const RowExtent& y) {
  if (x.end() <= y.at || y.end() <= x.at) return false;
  const RowExtent &a = x.rows <= y.rows ? x : y, &b = x.rows <= y.rows ? y : x;
  // row i of a against the first row of b that ends behind its begin; with equal
  // strides every row that meets b at all meets it as the first or the last does
  const int64_t step = a.stride == b.stride && a.rows > 2 ? a.rows - 1 : 1;
  for (int64_t i = 0; i < a.rows; i += step) {
    const uintptr_t lo = a.at + (uint64_t)i * a.stride, hi = lo + a.width;
    const uint64_t j = lo < b.at + b.width ? 0 : (lo - b.at - b.width) / b.stride + 1;
    if (j < (uint64_t)b.rows && b.at + j * b.stride < hi) return true;
  }
  return false;
}

}  // namespace lm
}  // namespace dobb
