// Global l2 norm of a set of gradients, and clipping by it.
//
// The entries are cut into chunks; a chunk's sum of squares is a double in
// the workspace.  The chunks of a tensor, and then the tensors, are summed in
// a fixed order.
#include "lm_common.cuh"

namespace dobb {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 32768;          // entries per chunk
constexpr int kTensorsPerLaunch = 512; // pointer tables travel in the kernel parameters

struct ClipArgs {
  int32_t num;             // tensors of this launch
  int64_t chunk_base;      // chunks of the launches before
  double* chunk_sums;      // one per chunk
  double* tensor_sums;     // one per tensor of this launch
  const float* stats;      // [1] = c
  const void* g[kTensorsPerLaunch];
  void* out[kTensorsPerLaunch];
  int64_t numel[kTensorsPerLaunch];
  int32_t chunk0[kTensorsPerLaunch + 1];  // first chunk of every tensor, within this launch
  uint8_t g_bf16[kTensorsPerLaunch], out_bf16[kTensorsPerLaunch];
};

int64_t chunks_of(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

// the tensor that chunk c belongs to
__device__ __forceinline__ int tensor_of(const ClipArgs& a, int32_t c) {
  int lo = 0, hi = a.num;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.chunk0[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float load_any(const void* p, bool bf16, int64_t i) {
  return bf16 ? load_f32(static_cast<const __nv_bfloat16*>(p) + i)
              : load_f32(static_cast<const float*>(p) + i);
}

__global__ void __launch_bounds__(kThreads) clip_chunk_sums(const __grid_constant__ ClipArgs a) {
  __shared__ double red[32];
  for (int32_t c = blockIdx.x; c < a.chunk0[a.num]; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const int64_t lo = (int64_t)(c - a.chunk0[t]) * kChunk, hi = min(a.numel[t], lo + kChunk);
    double s = 0.0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const double v = load_any(a.g[t], a.g_bf16[t], i);
      s += v * v;
    }
    s = block_sum_d(s, red);
    if (threadIdx.x == 0) a.chunk_sums[a.chunk_base + c] = s;
  }
}

__global__ void __launch_bounds__(kThreads) clip_tensor_sums(const __grid_constant__ ClipArgs a) {
  __shared__ double red[32];
  for (int t = blockIdx.x; t < a.num; t += gridDim.x) {
    double s = 0.0;
    for (int32_t c = a.chunk0[t] + threadIdx.x; c < a.chunk0[t + 1]; c += kThreads)
      s += a.chunk_sums[a.chunk_base + c];
    s = block_sum_d(s, red);
    if (threadIdx.x == 0) a.tensor_sums[t] = s;
  }
}

__global__ void __launch_bounds__(kThreads) clip_finish(const double* tensor_sums, int num,
                                                        float max_norm, float* stats,
                                                        uint32_t* flags) {
  __shared__ double red[32];
  double s = 0.0;
  for (int t = threadIdx.x; t < num; t += kThreads) {
    s += tensor_sums[t];
    stats[2 + t] = (float)sqrt(tensor_sums[t]);
  }
  s = block_sum_d(s, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s);
    const bool finite = isfinite(norm);
    stats[0] = (float)norm;
    stats[1] = (finite && norm > (double)max_norm) ? (float)((double)max_norm / norm) : 1.f;
    if (!finite && flags) atomicOr(flags, DOBB_FLAG_NONFINITE_G);
  }
}

__global__ void __launch_bounds__(kThreads) clip_scale(const __grid_constant__ ClipArgs a) {
  const float f = a.stats[1];
  for (int32_t c = blockIdx.x; c < a.chunk0[a.num]; c += gridDim.x) {
    const int t = tensor_of(a, c);
    if (f == 1.f && a.out[t] == a.g[t] && a.g_bf16[t] == a.out_bf16[t]) continue;
    const int64_t lo = (int64_t)(c - a.chunk0[t]) * kChunk, hi = min(a.numel[t], lo + kChunk);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const float v = f * load_any(a.g[t], a.g_bf16[t], i);
      if (a.out_bf16[t])
        store_f32(static_cast<__nv_bfloat16*>(a.out[t]) + i, v);
      else
        store_f32(static_cast<float*>(a.out[t]) + i, v);
    }
  }
}

struct Workspace {
  int64_t chunks;
  size_t tensor_off, total;
};

dobb_status measure(int num, const int64_t* numel, Workspace* w) {
  if (num < 1 || !numel)
    return fail(DOBB_ERR_INVALID_ARG, "num_tensors must be > 0 and numel non-NULL");
  int64_t chunks = 0;
  for (int i = 0; i < num; ++i) {
    if (numel[i] < 0) return fail(DOBB_ERR_INVALID_ARG, "numel[%d] < 0", i);
    chunks += chunks_of(numel[i]);
    if (chunks > INT32_MAX) return fail(DOBB_ERR_UNSUPPORTED, "the tensors have too many entries");
  }
  w->chunks = chunks;
  w->tensor_off = ((size_t)chunks * 8 + 255) / 256 * 256;
  w->total = w->tensor_off + ((size_t)num * 8 + 255) / 256 * 256;
  return DOBB_OK;
}

}  // namespace
}  // namespace dobb

using namespace dobb;

extern "C" size_t dobb_clip_grads_bytes(int num, const int64_t* numel) {
  Workspace w{};
  return measure(num, numel, &w) == DOBB_OK ? w.total : 0;
}

extern "C" dobb_status dobb_clip_grads(int num, const void* const* G, const int32_t* grad_dtype,
                                       const int64_t* numel, float max_norm, void* const* out,
                                       const int32_t* out_dtype, float* stats, uint32_t* flags,
                                       void* ws, size_t ws_bytes, void* stream) {
  Workspace w{};
  dobb_status st = measure(num, numel, &w);
  if (st != DOBB_OK) return st;
  if (!G || !grad_dtype || (out && !out_dtype))
    return fail(DOBB_ERR_INVALID_ARG, "G, grad_dtype and (with out) out_dtype must be non-NULL");
  if (out && !(max_norm >= 0.f)) return fail(DOBB_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!stats) return fail(DOBB_ERR_INVALID_ARG, "stats is NULL");
  for (int i = 0; i < num; ++i) {
    if (lm::bad_dtype(grad_dtype[i]) || (out && lm::bad_dtype(out_dtype[i])))
      return fail(DOBB_ERR_INVALID_ARG, "tensor %d: dtypes must be DOBB_F32 or DOBB_BF16", i);
    if (numel[i] == 0) continue;
    if (!G[i] || (out && !out[i])) return fail(DOBB_ERR_INVALID_ARG, "G[%d] or out[%d] is NULL", i, i);
    if (lm::misaligned(G[i], lm::dtype_bytes(grad_dtype[i])) ||
        (out && lm::misaligned(out[i], lm::dtype_bytes(out_dtype[i]))))
      return fail(DOBB_ERR_INVALID_ARG, "tensor %d is not aligned to its element size", i);
    if (out && out[i] == G[i] && grad_dtype[i] != out_dtype[i])
      return fail(DOBB_ERR_INVALID_ARG, "tensor %d: in place the dtypes must be equal", i);
  }
  if (!ws || lm::misaligned(ws, 256))
    return fail(DOBB_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (ws_bytes < w.total)
    return fail(DOBB_ERR_STATE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes,
                w.total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(ws);
  double* tensor_sums = reinterpret_cast<double*>(base + w.tensor_off);
  for (int phase = 0; phase < (out ? 2 : 1); ++phase) {
    ClipArgs a;
    a.chunk_base = 0;
    a.chunk_sums = reinterpret_cast<double*>(base);
    a.stats = stats;
    for (int t0 = 0; t0 < num; t0 += kTensorsPerLaunch) {
      a.num = num - t0 < kTensorsPerLaunch ? num - t0 : kTensorsPerLaunch;
      a.tensor_sums = tensor_sums + t0;
      a.chunk0[0] = 0;
      for (int i = 0; i < a.num; ++i) {
        a.g[i] = G[t0 + i];
        a.out[i] = out ? out[t0 + i] : nullptr;
        a.numel[i] = numel[t0 + i];
        a.g_bf16[i] = grad_dtype[t0 + i] == DOBB_BF16;
        a.out_bf16[i] = out && out_dtype[t0 + i] == DOBB_BF16;
        a.chunk0[i + 1] = a.chunk0[i] + (int32_t)chunks_of(numel[t0 + i]);
      }
      const int32_t chunks = a.chunk0[a.num];
      const int grid = chunks < 4096 ? chunks : 4096;
      if (phase == 0) {
        if (grid > 0) clip_chunk_sums<<<grid, kThreads, 0, s>>>(a);
        clip_tensor_sums<<<a.num, kThreads, 0, s>>>(a);
      } else if (grid > 0) {
        clip_scale<<<grid, kThreads, 0, s>>>(a);
      }
      a.chunk_base += chunks;
    }
    if (phase == 0)
      clip_finish<<<1, kThreads, 0, s>>>(tensor_sums, num, out ? max_norm : INFINITY, stats, flags);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "clipping launch: %s", cudaGetErrorString(e));
  }
  return DOBB_OK;
}
