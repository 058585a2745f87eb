// Log probabilities of given tokens, entropies, the most likely alternatives,
// and their gradient with respect to the logits.
//
// With y = scale * x over a row of V logits, M = max x, u_j = scale (x_j - M):
//   S = sum e^{u_j},  E = sum e^{u_j} u_j
//   log_sum = log S,  logp = u_t - log S,  entropy = log S - E / S.
// (M, S, E) of two parts join exactly: with M' the larger maximum and
// d = scale (M - M'), a part's S becomes S e^d and its E becomes
// (E + S d) e^d.  An entry -inf adds nothing to either sum.
#include "lm_common.cuh"

namespace dobb {
namespace {

constexpr int kThreads = 256;

struct LpArgs {
  const void* logits;
  int64_t rows, row_stride;
  int32_t vocab;
  const void* tokens;
  int32_t token_bytes;
  float scale;
  int32_t top_k;
  float *logp, *lse, *row_max, *log_sum, *entropy;
  int32_t* top_ids;
  float* top_logp;
  uint32_t* flags;
};

struct LpGradArgs {
  const void* logits;
  int64_t rows, row_stride;
  int32_t vocab;
  const void* tokens;
  int32_t token_bytes;
  float scale;
  const float *row_max, *log_sum, *entropy;
  const float *g, *h, *l;
  void* out;
  int64_t out_stride;
};

struct Sums {
  float m, s, e;
};

// A part's contribution at the joint maximum m.  A part that saw only -inf
// and NaN (m = -inf) holds 0 or NaN in its sums, which pass through.
__device__ __forceinline__ void add_part(Sums& r, const Sums& a, float scale) {
  if (a.m == -INFINITY) {
    r.s += a.s;
    r.e += a.e;
  } else {
    const float d = scale * (a.m - r.m), f = expf(d);
    r.s += a.s * f;
    r.e += (f > 0.f) ? (a.e + a.s * d) * f : 0.f;
  }
}

__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float scale) {
  Sums r{fmaxf(a.m, b.m), 0.f, 0.f};
  add_part(r, a, scale);
  add_part(r, b, scale);
  return r;
}

// Unsigned integers in the order of the floats; -0 equals 0, every NaN is
// the largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x == x)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) lp_forward(const LpArgs a) {
  __shared__ Sums part[kThreads / 32];
  __shared__ unsigned long long best[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    Sums t{-INFINITY, 0.f, 0.f};
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
      const float v = load_f32(x + j);
      if (v == -INFINITY) continue;
      if (v > t.m) t = join(t, Sums{v, 0.f, 0.f}, a.scale);
      const float u = a.scale * (v - t.m), f = expf(u);
      t.s += f;
      t.e += (f > 0.f) ? f * u : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Sums b;
      b.m = __shfl_down_sync(0xffffffffu, t.m, o);
      b.s = __shfl_down_sync(0xffffffffu, t.s, o);
      b.e = __shfl_down_sync(0xffffffffu, t.e, o);
      t = join(t, b, a.scale);
    }
    __syncthreads();
    if (lane == 0) part[warp] = t;
    __syncthreads();
    Sums r = part[0];
    for (int w = 1; w < kThreads / 32; ++w) r = join(r, part[w], a.scale);
    const bool empty = r.m == -INFINITY && r.s == 0.f;
    const float log_sum = logf(r.s);
    if (threadIdx.x == 0) {
      const int64_t tok = lm::load_token(a.tokens, a.token_bytes, row);
      float lp = 0.f;
      if (tok >= a.vocab) {
        lp = NAN;
        if (a.flags) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
      } else if (tok >= 0) {
        const float v = load_f32(x + tok);
        lp = empty ? -INFINITY : a.scale * (v - r.m) - log_sum;
      }
      a.logp[row] = lp;
      a.row_max[row] = r.m;
      a.log_sum[row] = log_sum;
      if (a.lse) a.lse[row] = empty ? -INFINITY : a.scale * r.m + log_sum;
      if (a.entropy) a.entropy[row] = empty ? 0.f : log_sum - r.e / r.s;
    }
    // alternatives: the largest key below the last one, top_k times
    unsigned long long last = ~0ull;
    for (int i = 0; i < a.top_k; ++i) {
      unsigned long long b = 0;
      for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
        const unsigned long long key =
            ((unsigned long long)order_key(load_f32(x + j)) << 32) | (uint32_t)(0x7fffffff - j);
        if (key < last && key > b) b = key;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long c = __shfl_xor_sync(0xffffffffu, b, o);
        b = c > b ? c : b;
      }
      __syncthreads();
      if (lane == 0) best[warp] = b;
      __syncthreads();
      b = best[0];
      for (int w = 1; w < kThreads / 32; ++w) b = best[w] > b ? best[w] : b;
      last = b;
      if (threadIdx.x == 0) {
        const int j = 0x7fffffff - (int)(uint32_t)b;
        a.top_ids[row * a.top_k + i] = j;
        a.top_logp[row * a.top_k + i] =
            empty ? -INFINITY : a.scale * (load_f32(x + j) - r.m) - log_sum;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) lp_backward(const LpGradArgs a) {
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    T* d = static_cast<T*>(a.out) + row * a.out_stride;
    const float m = a.row_max[row], log_sum = a.log_sum[row];
    const int64_t tok = lm::load_token(a.tokens, a.token_bytes, row);
    const bool empty = m == -INFINITY && log_sum == -INFINITY;
    const float g = (tok >= 0 && tok < a.vocab) ? a.g[row] : 0.f;
    const float h = a.h ? a.h[row] : 0.f;
    const float l = a.l ? a.l[row] : 0.f;
    const float ent = a.h ? a.entropy[row] : 0.f;
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
      float r = 0.f;
      if (!empty) {
        const float lp = a.scale * (load_f32(x + j) - m) - log_sum;
        const float p = expf(lp);
        if (p != 0.f) r = p * (l - g - h * (lp + ent));
        if (j == tok) r += g;
      }
      store_f32(d + j, a.scale * r);
    }
  }
}

}  // namespace
}  // namespace dobb

using namespace dobb;

namespace {

dobb_status check_logits(const void* logits, int dtype, int64_t rows, int64_t vocab,
                         int64_t row_stride, const void* tokens, int token_bytes, float scale) {
  if (lm::bad_dtype(dtype)) return fail(DOBB_ERR_INVALID_ARG, "logits dtype must be DOBB_F32 or DOBB_BF16");
  if (rows < 0) return fail(DOBB_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
  if (vocab < 1 || vocab > INT32_MAX)
    return fail(DOBB_ERR_INVALID_ARG, "vocab must lie in [1, 2^31) (got %lld)", (long long)vocab);
  if (row_stride < vocab && rows > 1)
    return fail(DOBB_ERR_INVALID_ARG, "row_stride %lld is below vocab %lld", (long long)row_stride,
                (long long)vocab);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(DOBB_ERR_INVALID_ARG, "token_bytes must be 4 or 8 (got %d)", token_bytes);
  if (!(scale > 0.f) || std::isinf(scale))
    return fail(DOBB_ERR_INVALID_ARG, "scale must be positive and finite (got %g)", scale);
  if (rows == 0) return DOBB_OK;
  if (!logits || !tokens) return fail(DOBB_ERR_INVALID_ARG, "logits and tokens must be non-NULL");
  if (lm::misaligned(logits, lm::dtype_bytes(dtype)) || lm::misaligned(tokens, token_bytes))
    return fail(DOBB_ERR_INVALID_ARG, "logits or tokens not aligned to their element size");
  return DOBB_OK;
}

}  // namespace

extern "C" dobb_status dobb_log_probs(const void* logits, dobb_dtype logits_dtype, int64_t rows,
                                      int64_t vocab, int64_t row_stride, const void* tokens,
                                      int token_bytes, float scale, int top_k, float* logp,
                                      float* lse, float* row_max, float* log_sum, float* entropy,
                                      int32_t* top_ids, float* top_logp, uint32_t* flags,
                                      void* stream) {
  dobb_status st =
      check_logits(logits, logits_dtype, rows, vocab, row_stride, tokens, token_bytes, scale);
  if (st != DOBB_OK) return st;
  if (top_k < 0 || top_k > DOBB_MAX_TOP_K || top_k > vocab)
    return fail(DOBB_ERR_INVALID_ARG, "top_k must lie in [0, min(%d, vocab)] (got %d)",
                DOBB_MAX_TOP_K, top_k);
  if (rows == 0) return DOBB_OK;
  if (!logp || !row_max || !log_sum)
    return fail(DOBB_ERR_INVALID_ARG, "logp, row_max and log_sum must be non-NULL");
  if (top_k > 0 && (!top_ids || !top_logp))
    return fail(DOBB_ERR_INVALID_ARG, "top_ids and top_logp must be non-NULL when top_k > 0");
  const LpArgs a{logits, rows,    row_stride, (int32_t)vocab, tokens,  token_bytes, scale, top_k,
                 logp,   lse,     row_max,    log_sum,        entropy, top_ids,     top_logp, flags};
  const unsigned grid = (unsigned)(rows < (1 << 30) ? rows : (1 << 30));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (logits_dtype == DOBB_F32)
    lp_forward<float><<<grid, kThreads, 0, s>>>(a);
  else
    lp_forward<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "log-probability launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

extern "C" dobb_status dobb_log_probs_backward(const void* logits, dobb_dtype logits_dtype,
                                               int64_t rows, int64_t vocab, int64_t row_stride,
                                               const void* tokens, int token_bytes, float scale,
                                               const float* row_max, const float* log_sum,
                                               const float* entropy, const float* grad_logp,
                                               const float* grad_entropy, const float* grad_lse,
                                               void* dlogits, int64_t out_stride, void* stream) {
  dobb_status st =
      check_logits(logits, logits_dtype, rows, vocab, row_stride, tokens, token_bytes, scale);
  if (st != DOBB_OK) return st;
  if (out_stride < vocab && rows > 1)
    return fail(DOBB_ERR_INVALID_ARG, "out_stride %lld is below vocab %lld", (long long)out_stride,
                (long long)vocab);
  if (rows == 0) return DOBB_OK;
  if (!row_max || !log_sum || !grad_logp || !dlogits)
    return fail(DOBB_ERR_INVALID_ARG, "row_max, log_sum, grad_logp and dlogits must be non-NULL");
  if (grad_entropy && !entropy)
    return fail(DOBB_ERR_INVALID_ARG, "grad_entropy needs the forward's entropy");
  if (lm::misaligned(dlogits, lm::dtype_bytes(logits_dtype)))
    return fail(DOBB_ERR_INVALID_ARG, "dlogits not aligned to its element size");
  if (dlogits == logits && out_stride != row_stride && rows > 1)
    return fail(DOBB_ERR_INVALID_ARG, "in place the strides must be equal");
  const LpGradArgs a{logits,  rows,    row_stride, (int32_t)vocab, tokens,       token_bytes, scale,
                     row_max, log_sum, entropy,    grad_logp,      grad_entropy, grad_lse,    dlogits,
                     out_stride};
  const unsigned grid = (unsigned)(rows < (1 << 30) ? rows : (1 << 30));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (logits_dtype == DOBB_F32)
    lp_backward<float><<<grid, kThreads, 0, s>>>(a);
  else
    lp_backward<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(DOBB_ERR_CUDA, "log-probability gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
