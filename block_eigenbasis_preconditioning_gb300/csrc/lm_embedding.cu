// Embedding lookup with scaling, and its gradient by sorted tokens.
#include "lm_common.cuh"

namespace dobb {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ lookup

struct EmbedArgs {
  const void* weight;
  int64_t vocab, dim, weight_stride;
  const void* tokens;
  int32_t token_bytes;
  int64_t count;
  float scale;
  void* out;
  int64_t out_stride;
  uint32_t* flags;
};

template <typename W, typename O>
__global__ void __launch_bounds__(kThreads) embed_forward(const EmbedArgs a) {
  for (int64_t t = blockIdx.x; t < a.count; t += gridDim.x) {
    const int64_t v = lm::load_token(a.tokens, a.token_bytes, t);
    const bool live = v >= 0 && v < a.vocab;
    if (v >= a.vocab && a.flags && threadIdx.x == 0) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
    const W* w = static_cast<const W*>(a.weight) + (live ? v : 0) * a.weight_stride;
    O* o = static_cast<O*>(a.out) + t * a.out_stride;
    for (int64_t j = threadIdx.x; j < a.dim; j += kThreads)
      store_f32(o + j, live ? a.scale * load_f32(w + j) : 0.f);
  }
}

// -------------------------------------------------------------------- sort
// Stable least-significant-digit radix sort of (token, position).  Tokens
// that take no gradient get the key `vocab` and end up last.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 8;
constexpr int kBins = 1 << kDigitBits;

struct SortArgs {
  const void* tokens;
  int32_t token_bytes;
  int32_t count, vocab;
  int32_t passes;
  uint32_t* key[2];  // pass p reads buffer p & 1, writes the other; pass 0 reads the tokens
  uint32_t* pos[2];
  uint32_t* flags;
};

__device__ __forceinline__ uint32_t token_key(const SortArgs& a, int32_t i) {
  const int64_t v = lm::load_token(a.tokens, a.token_bytes, i);
  if (v >= a.vocab && a.flags) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
  return (v >= 0 && v < a.vocab) ? (uint32_t)v : (uint32_t)a.vocab;
}

__global__ void __launch_bounds__(kSortThreads) sort_tokens(const SortArgs a) {
  __shared__ uint32_t hist[kSortWarps][kBins];
  __shared__ uint32_t total[kBins];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // each warp takes a contiguous run of items, so that the order of equal digits is kept
  const int64_t per = (((int64_t)a.count + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t lo = min((int64_t)a.count, per * warp), hi = min((int64_t)a.count, lo + per);
  for (int p = 0; p < a.passes; ++p) {
    const uint32_t* key = a.key[p & 1];
    const uint32_t* pos = a.pos[p & 1];
    const int shift = p * kDigitBits;
    for (int b = lane; b < kBins; b += 32) hist[warp][b] = 0;
    __syncwarp();
    for (int64_t i = lo + lane; i < hi; i += 32) {
      const uint32_t k = p == 0 ? token_key(a, (int32_t)i) : key[i];
      atomicAdd(&hist[warp][(k >> shift) & (kBins - 1)], 1u);
    }
    __syncthreads();
    // first place of every (digit, warp): digits in order, within a digit the warps in order
    if (threadIdx.x < kBins) {
      uint32_t sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w][threadIdx.x];
        hist[w][threadIdx.x] = sum;
        sum += c;
      }
      total[threadIdx.x] = sum;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      uint32_t base = 0;
      for (int b = 0; b < (int)threadIdx.x; ++b) base += total[b];
      for (int w = 0; w < kSortWarps; ++w) hist[w][threadIdx.x] += base;
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool in = i < hi;
      const unsigned live = __ballot_sync(0xffffffffu, in);
      if (in) {
        const uint32_t k = p == 0 ? token_key(a, (int32_t)i) : key[i];
        const uint32_t d = (k >> shift) & (kBins - 1);
        const unsigned same = __match_any_sync(live, d);
        const uint32_t at = hist[warp][d] + __popc(same & ((1u << lane) - 1u));
        __syncwarp(live);
        if (lane == 31 - __clz(same)) hist[warp][d] = at + 1;
        a.key[(p + 1) & 1][at] = k;
        a.pos[(p + 1) & 1][at] = p == 0 ? (uint32_t)i : pos[i];
      }
      __syncwarp();
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- gradient

struct EmbedGradArgs {
  const void* grad;
  int64_t dim, grad_stride;
  int32_t count, vocab;
  const uint32_t *key, *pos;  // sorted
  float scale;
  void* out;
  int64_t out_stride;
  int32_t accumulate;
};

__device__ __forceinline__ int32_t lower_bound(const uint32_t* key, int32_t n, uint32_t v) {
  int32_t lo = 0, hi = n;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (key[mid] < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// one CTA per row of the weight: the row's gradients summed in token order
template <typename G, typename O>
__global__ void __launch_bounds__(kThreads) embed_backward(const EmbedGradArgs a) {
  for (int32_t v = blockIdx.x; v < a.vocab; v += gridDim.x) {
    const int32_t lo = lower_bound(a.key, a.count, (uint32_t)v);
    const int32_t hi = lower_bound(a.key, a.count, (uint32_t)v + 1);
    if (a.accumulate && lo == hi) continue;
    O* o = static_cast<O*>(a.out) + v * a.out_stride;
    for (int64_t j = threadIdx.x; j < a.dim; j += kThreads) {
      float sum = 0.f;
      for (int32_t i = lo; i < hi; ++i)
        sum += load_f32(static_cast<const G*>(a.grad) + a.pos[i] * a.grad_stride + j);
      sum *= a.scale;
      if (a.accumulate) sum += load_f32(o + j);
      store_f32(o + j, sum);
    }
  }
}

struct Workspace {
  size_t key[2], pos[2], total;
};

Workspace workspace(int64_t count) {
  Workspace w{};
  const size_t n = ((size_t)count * 4 + 255) / 256 * 256;
  w.key[0] = 0;
  w.key[1] = n;
  w.pos[0] = 2 * n;
  w.pos[1] = 3 * n;
  w.total = 4 * n + 256;
  return w;
}

dobb_status check_grad_sizes(int64_t count, int64_t vocab, int64_t dim) {
  if (count < 0 || count > INT32_MAX)
    return fail(DOBB_ERR_INVALID_ARG, "count must lie in [0, 2^31) (got %lld)", (long long)count);
  if (vocab < 1 || vocab > (1 << 30))
    return fail(DOBB_ERR_INVALID_ARG, "vocab must lie in [1, 2^30] (got %lld)", (long long)vocab);
  if (dim < 1) return fail(DOBB_ERR_INVALID_ARG, "dim must be >= 1 (got %lld)", (long long)dim);
  return DOBB_OK;
}

}  // namespace
}  // namespace dobb

using namespace dobb;

extern "C" dobb_status dobb_embedding(const void* weight, dobb_dtype weight_dtype, int64_t vocab,
                                      int64_t dim, int64_t weight_stride, const void* tokens,
                                      int token_bytes, int64_t count, float scale, void* out,
                                      dobb_dtype out_dtype, int64_t out_stride, uint32_t* flags,
                                      void* stream) {
  if (lm::bad_dtype(weight_dtype) || lm::bad_dtype(out_dtype))
    return fail(DOBB_ERR_INVALID_ARG, "weight and out dtypes must be DOBB_F32 or DOBB_BF16");
  if (vocab < 1 || dim < 1)
    return fail(DOBB_ERR_INVALID_ARG, "vocab and dim must be >= 1 (got %lld, %lld)",
                (long long)vocab, (long long)dim);
  if (count < 0) return fail(DOBB_ERR_INVALID_ARG, "count must be >= 0 (got %lld)", (long long)count);
  if ((weight_stride < dim && vocab > 1) || (out_stride < dim && count > 1))
    return fail(DOBB_ERR_INVALID_ARG, "row strides %lld and %lld must be at least dim %lld",
                (long long)weight_stride, (long long)out_stride, (long long)dim);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(DOBB_ERR_INVALID_ARG, "token_bytes must be 4 or 8 (got %d)", token_bytes);
  if (!std::isfinite(scale)) return fail(DOBB_ERR_INVALID_ARG, "scale must be finite");
  if (count == 0) return DOBB_OK;
  if (!weight || !tokens || !out)
    return fail(DOBB_ERR_INVALID_ARG, "weight, tokens and out must be non-NULL");
  if (lm::misaligned(weight, lm::dtype_bytes(weight_dtype)) ||
      lm::misaligned(out, lm::dtype_bytes(out_dtype)) || lm::misaligned(tokens, token_bytes))
    return fail(DOBB_ERR_INVALID_ARG, "weight, tokens or out not aligned to its element size");
  const EmbedArgs a{weight, vocab, dim,        weight_stride, tokens, token_bytes,
                    count,  scale, out,        out_stride,    flags};
  const unsigned grid = (unsigned)(count < (1 << 30) ? count : (1 << 30));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int which = 2 * (weight_dtype == DOBB_BF16) + (out_dtype == DOBB_BF16);
  if (which == 0) embed_forward<float, float><<<grid, kThreads, 0, s>>>(a);
  if (which == 1) embed_forward<float, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  if (which == 2) embed_forward<__nv_bfloat16, float><<<grid, kThreads, 0, s>>>(a);
  if (which == 3) embed_forward<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "embedding launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

extern "C" size_t dobb_embedding_backward_bytes(int64_t count, int64_t vocab, int64_t dim) {
  if (check_grad_sizes(count, vocab, dim) != DOBB_OK) return 0;
  return workspace(count).total;
}

extern "C" dobb_status dobb_embedding_backward(const void* grad, dobb_dtype grad_dtype,
                                               int64_t count, int64_t dim, int64_t grad_stride,
                                               const void* tokens, int token_bytes, int64_t vocab,
                                               float scale, void* dweight, dobb_dtype dweight_dtype,
                                               int64_t dweight_stride, int accumulate,
                                               uint32_t* flags, void* ws, size_t ws_bytes,
                                               void* stream) {
  if (lm::bad_dtype(grad_dtype) || lm::bad_dtype(dweight_dtype))
    return fail(DOBB_ERR_INVALID_ARG, "grad and dweight dtypes must be DOBB_F32 or DOBB_BF16");
  dobb_status st = check_grad_sizes(count, vocab, dim);
  if (st != DOBB_OK) return st;
  if ((grad_stride < dim && count > 1) || (dweight_stride < dim && vocab > 1))
    return fail(DOBB_ERR_INVALID_ARG, "row strides %lld and %lld must be at least dim %lld",
                (long long)grad_stride, (long long)dweight_stride, (long long)dim);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(DOBB_ERR_INVALID_ARG, "token_bytes must be 4 or 8 (got %d)", token_bytes);
  if (!std::isfinite(scale)) return fail(DOBB_ERR_INVALID_ARG, "scale must be finite");
  if (accumulate != 0 && accumulate != 1)
    return fail(DOBB_ERR_INVALID_ARG, "accumulate must be 0 or 1 (got %d)", accumulate);
  if (!dweight || (count > 0 && (!grad || !tokens)))
    return fail(DOBB_ERR_INVALID_ARG, "grad, tokens and dweight must be non-NULL");
  if (lm::misaligned(dweight, lm::dtype_bytes(dweight_dtype)) ||
      (count > 0 && (lm::misaligned(grad, lm::dtype_bytes(grad_dtype)) ||
                     lm::misaligned(tokens, token_bytes))))
    return fail(DOBB_ERR_INVALID_ARG, "grad, tokens or dweight not aligned to its element size");
  const Workspace w = workspace(count);
  if (!ws || lm::misaligned(ws, 256))
    return fail(DOBB_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (ws_bytes < w.total)
    return fail(DOBB_ERR_STATE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes,
                w.total);
  if (count == 0 && accumulate) return DOBB_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(ws);
  SortArgs sa{};
  sa.tokens = tokens;
  sa.token_bytes = token_bytes;
  sa.count = (int32_t)count;
  sa.vocab = (int32_t)vocab;
  sa.passes = 1;
  while (sa.passes * kDigitBits < 32 && ((uint32_t)vocab >> (sa.passes * kDigitBits)) != 0) ++sa.passes;
  for (int i = 0; i < 2; ++i) {
    sa.key[i] = reinterpret_cast<uint32_t*>(base + w.key[i]);
    sa.pos[i] = reinterpret_cast<uint32_t*>(base + w.pos[i]);
  }
  sa.flags = flags;
  if (count > 0) sort_tokens<<<1, kSortThreads, 0, s>>>(sa);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "token sort launch: %s", cudaGetErrorString(e));
  EmbedGradArgs a{grad,
                  dim,
                  grad_stride,
                  (int32_t)count,
                  (int32_t)vocab,
                  sa.key[sa.passes & 1],
                  sa.pos[sa.passes & 1],
                  scale,
                  dweight,
                  dweight_stride,
                  accumulate};
  const unsigned grid = (unsigned)vocab;
  const int which = 2 * (grad_dtype == DOBB_BF16) + (dweight_dtype == DOBB_BF16);
  if (which == 0) embed_backward<float, float><<<grid, kThreads, 0, s>>>(a);
  if (which == 1) embed_backward<float, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  if (which == 2) embed_backward<__nv_bfloat16, float><<<grid, kThreads, 0, s>>>(a);
  if (which == 3) embed_backward<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(DOBB_ERR_CUDA, "embedding gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
