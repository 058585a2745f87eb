// Global l2 norm of a set of gradients, and clipping by it, in two kernels.
//
// The tensors' entries are cut into chunks, and the chunks, tensor after
// tensor, into one stretch of equal length per CTA.  The first kernel squares
// and sums: a CTA leaves one fp64 sum per tensor of its stretch, in slot (CTA +
// tensor), which no other pair has, and zeros in the slots between its own
// and the next CTA's.  The second kernel sums the slots (every CTA all of
// them, in the same order: some KB from L2), and scales the stretches, last
// chunk first: what the first kernel read last is still in L2.
//
// Within a chunk a thread sums the squares of 32 of its entries in four fp32
// chains, and adds the result to an fp32 pair (hi, lo) whose sum is exact but for
// the rounding of lo.  Where the result lies outside [2^-116, 2^100) (large, tiny
// or non-finite entries: fp32 squares are not exact enough, or the pair could
// overflow on the way) the thread sums its entries again in fp64.
//
// Bound by HBM: the GPT-2 XL gradients, fp32 to bf16, 15.5 GB with the second
// read in 2.25 ms, the copy rate; sums alone 5.9 TB/s.  Scaling 8 entries a
// thread, strided, instead of 4 side by side took 3.29 ms.  Two CTAs an SM with
// 64 entries a thread in flight instead of four with 32, and small tensors a
// warp each instead of one after another: 12 layers of width 768 (2048 inside)
// with their vectors in a graph, bf16 in place, 62 to 37 us, fp32 to bf16 115 to
// 104; calls on GPT-2 Small fp32 179 to 172.
#include <algorithm>
#include <vector>

#include "lm_common.cuh"

namespace dobb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 2;     // per SM
constexpr int kEach = 64;    // entries of a chunk per thread, in flight together
constexpr int kSum = 32;     // of which so many are summed in plain fp32
constexpr int kChunk = kEach * kThreads;
// Neighbouring tensors of up to this many entries (biases, norms) are taken
// together, a warp each: one after another each costs its latency.
constexpr int kSmall = 4096;
constexpr int kSms = 152;
constexpr int kMaxTensors = 512;  // of a launch: the tables travel in the kernel parameters
constexpr int kFewTensors = 32;   // a table of 1 KB, launched faster

template <int K>
struct Table {
  int32_t num;        // tensors
  int32_t chunks, grid;
  int64_t slot0;      // first slot of this launch
  const void* g[K];
  void* out[K];
  int64_t numel[K];
  int32_t chunk0[K + 1];  // first chunk of every tensor
  uint8_t g_bf16[K], out_bf16[K];
};

int64_t chunks_of(int64_t numel) { return numel / kChunk + (numel % kChunk != 0); }

// Stretch of CTA b: chunks [first(b), first(b + 1)); the CTA of chunk c.
template <int K>
__device__ __forceinline__ int32_t first_chunk(const Table<K>& a, int32_t b) {
  return (int32_t)((int64_t)b * a.chunks / a.grid);
}
template <int K>
__device__ __forceinline__ int32_t cta_of(const Table<K>& a, int32_t c) {
  return (int32_t)((((int64_t)c + 1) * a.grid - 1) / a.chunks);
}

// the tensor that chunk c belongs to
template <int K>
__device__ __forceinline__ int tensor_of(const Table<K>& a, int32_t c) {
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

// A thread's sum of squares: hi + lo + wide.
struct Squares {
  float hi = 0.f, lo = 0.f;
  double wide = 0.0;
  __device__ __forceinline__ void add(float s) {  // Knuth's two-sum
    const float t = hi + s, z = t - hi;
    lo += (hi - (t - z)) + (s - z);
    hi = t;
  }
};

// Where 32 squares sum to less than this, their rounding (2^-150 each, below
// the smallest normal number) could show; zeros alone are exact.
constexpr float kSmallest = 1.2e-35f;  // 2^-116
// A launch has fewer than 2^31 chunks, over 304 CTAs where there are as many: a
// thread adds fewer than 2^24 sums to its pair, which stays below 2^124.
constexpr float kLargest = 0x1p100f;

// n entries, up to kEach per thread of THREADS (tid: 0 ... THREADS - 1).
template <int THREADS, typename T>
__device__ __forceinline__ void add_chunk(Squares& sum, const T* p, int32_t n, int tid) {
  using V = lm::Vec16<T>;
  constexpr int kVecs = kEach / V::N;
  const int32_t head = (int32_t)lm::head_of(p, n), nvec = (n - head) / V::N, tail0 = head + nvec * V::N;
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
  // an entry before or behind the vectors: fewer than 8 each
  const int32_t at = tid < head ? tid : (tid >= 8 && tid - 8 < n - tail0) ? tail0 + tid - 8 : -1;
  uint4 x[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
    x[u] = tid + u * THREADS < nvec ? __ldg(v + tid + u * THREADS) : make_uint4(0, 0, 0, 0);
  float single = at >= 0 ? load_f32(p + at) : 0.f;
#pragma unroll
  for (int part = 0; part < kVecs; part += kSum / V::N) {
    uint64_t s[2] = {0, 0};
    uint32_t bits = 0;
#pragma unroll
    for (int u = part; u < part + kSum / V::N; ++u) {
      bits |= x[u].x | x[u].y | x[u].z | x[u].w;
#pragma unroll
      for (int i = 0; i < V::N / 2; ++i) {
        const uint64_t w = V::pair(x[u], i);
        s[i & 1] = lm::fma2(w, w, s[i & 1]);
      }
    }
    float a, b, c, d;
    lm::unpack2(s[0], a, b);
    lm::unpack2(s[1], c, d);
    const float t = fmaf(single, single, (a + b) + (c + d));
    // (bits: the signs of zeros are no entries)
    const bool zero = (bits & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu)) == 0 && single == 0.f;
    if ((t >= kSmallest && t < kLargest) || zero) {
      sum.add(t);
    } else {
#pragma unroll 1
      for (int32_t j = tid + part * THREADS; j < min(nvec, (part + kSum / V::N) * THREADS); j += THREADS)
#pragma unroll 1
        for (int i = 0; i < V::N; ++i) {
          const double y = load_f32(p + head + j * V::N + i);
          sum.wide += y * y;
        }
      sum.wide += (double)single * single;
    }
    single = 0.f;
  }
}

template <int K>
__global__ void __launch_bounds__(kThreads, kCtas) clip_sums(const __grid_constant__ Table<K> a, double* slots) {
  __shared__ double red[32];
  asm volatile("griddepcontrol.launch_dependents;");
  slots += a.slot0;
  const int32_t b = blockIdx.x, end = first_chunk(a, b + 1);
  int32_t c = first_chunk(a, b);
  int t = tensor_of(a, c);
  if (b == 0)
    for (int i = threadIdx.x; i < t; i += kThreads) slots[i] = 0.0;
  while (c < end) {
    Squares sum;
    const int32_t stop = min(end, a.chunk0[t + 1]);
    int m = 0;  // small tensors side by side, empty ones among them
    while (m < kWarps && t + m < a.num && a.numel[t + m] <= kSmall && a.chunk0[t + m + 1] <= end) ++m;
    if (m > 1) {
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (warp < m) {
        const int32_t n = (int32_t)a.numel[t + warp];
        for (int32_t lo = 0; lo < n; lo += 32 * kEach) {
          if (a.g_bf16[t + warp])
            add_chunk<32>(sum, static_cast<const __nv_bfloat16*>(a.g[t + warp]) + lo, min(32 * kEach, n - lo), lane);
          else
            add_chunk<32>(sum, static_cast<const float*>(a.g[t + warp]) + lo, min(32 * kEach, n - lo), lane);
        }
        const double s = warp_sum_d((double)sum.hi + sum.lo + sum.wide);
        if (lane == 0) slots[b + t + warp] = s;
      }
      t += m - 1;
      c = a.chunk0[t + 1];
    }
    for (; c < stop; ++c) {
      const int64_t lo = (int64_t)(c - a.chunk0[t]) * kChunk;
      const int32_t n = (int32_t)min((int64_t)kChunk, a.numel[t] - lo);
      if (a.g_bf16[t])
        add_chunk<kThreads>(sum, static_cast<const __nv_bfloat16*>(a.g[t]) + lo, n, threadIdx.x);
      else
        add_chunk<kThreads>(sum, static_cast<const float*>(a.g[t]) + lo, n, threadIdx.x);
    }
    const double s = m > 1 ? 0.0 : block_sum_d((double)sum.hi + sum.lo + sum.wide, red);
    // the next slot that is written by this CTA or the next one
    int next = t;
    int32_t after = a.grid + a.num;
    if (c < a.chunks) {
      do ++next;
      while (next < a.num && a.chunk0[next + 1] <= c);
      if (c < a.chunk0[t + 1]) next = t;
      after = b + (c == end) + next;
    }
    if (m <= 1 && threadIdx.x == 0) slots[b + t] = s;
    for (int i = b + t + 1 + threadIdx.x; i < after; i += kThreads) slots[i] = 0.0;
    t = next;
  }
}

// Four entries (eight where both sides are bf16), a whole number of loads and
// stores of up to 16 bytes, neighbouring lanes side by side.
template <typename T, int E>
struct Entries {
  static constexpr int kWords = E * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);  // in place, p is written later
      w[0] = v.x, w[1] = v.y, w[kWords - 2] = v.z, w[kWords - 1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if (kWords == 4)
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[kWords - 2], w[kWords - 1]));
    else
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  }
  __device__ __forceinline__ uint64_t pair(int i) const {
    return sizeof(T) == 2 ? lm::pack2(lm::bf16_lo(w[i]), lm::bf16_hi(w[i]))
                          : lm::pack2(__uint_as_float(w[2 * i % kWords]), __uint_as_float(w[(2 * i + 1) % kWords]));
  }
  __device__ __forceinline__ void put(int i, uint64_t v) {
    float lo, hi;
    lm::unpack2(v, lo, hi);
    if (sizeof(T) == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      w[2 * i % kWords] = __float_as_uint(lo);
      w[(2 * i + 1) % kWords] = __float_as_uint(hi);
    }
  }
};

// n entries by `threads` threads: a last chunk of a tensor, a small tensor, or
// (value by value) one that is not on the vectors' boundaries.  Out of line:
// it would only push the common path out of the instruction cache.
template <typename G, typename O, int E>
__device__ __noinline__ void scale_some(const G* p, O* o, int32_t n, float f, int tid, int threads) {
  const uintptr_t off = (reinterpret_cast<uintptr_t>(p) % (E * sizeof(G))) |
                        (reinterpret_cast<uintptr_t>(o) % (E * sizeof(O)));
  const int32_t packed = off == 0 ? n / E * E : 0;
  const uint64_t f2 = lm::pack2(f, f);
#pragma unroll 4
  for (int32_t j = tid * E; j < packed; j += threads * E) {
    Entries<G, E> x;
    x.load(p + j);
    Entries<O, E> r;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) r.put(i, lm::mul2(x.pair(i), f2));
    r.store(o + j);
  }
#pragma unroll 8
  for (int32_t j = packed + tid; j < n; j += threads) store_f32(o + j, f * load_f32(p + j));
}

template <typename G, typename O>
__device__ __forceinline__ void scale_chunk(const G* p, O* o, int32_t n, float f, int tid, int threads) {
  constexpr int E = sizeof(G) + sizeof(O) == 4 ? 8 : 4;
  constexpr int kTimes = kChunk / E / kThreads;
  const uintptr_t off = (reinterpret_cast<uintptr_t>(p) % (E * sizeof(G))) |
                        (reinterpret_cast<uintptr_t>(o) % (E * sizeof(O)));
  if (off != 0 || n != kChunk || threads != kThreads) return scale_some<G, O, E>(p, o, n, f, tid, threads);
  const uint64_t f2 = lm::pack2(f, f);
  Entries<G, E> x[kTimes];
#pragma unroll
  for (int u = 0; u < kTimes; ++u) x[u].load(p + (threadIdx.x + u * kThreads) * E);
#pragma unroll
  for (int u = 0; u < kTimes; ++u) {
    Entries<O, E> r;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) r.put(i, lm::mul2(x[u].pair(i), f2));
    r.store(o + (threadIdx.x + u * kThreads) * E);
  }
}

// The same by a factor below the normal range of fp32, which fp32 would hold with
// few bits or none (a norm of 1e39 brought to 1): each product in fp64, rounded to
// fp32 and the output.
template <typename G, typename O>
__device__ __noinline__ void scale_tiny(const G* p, O* o, int32_t n, double c, int tid, int threads) {
  for (int32_t j = tid; j < n; j += threads) store_f32(o + j, (float)(c * (double)load_f32(p + j)));
}

// scale 0: the norms only
template <int K>
__global__ void __launch_bounds__(kThreads, kCtas) clip_scale(const __grid_constant__ Table<K> a, const double* slots,
                                                          int64_t num_slots, float max_norm, float* stats,
                                                          float* norms, uint32_t* flags, int scale) {
  __shared__ double red[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < num_slots; i += kThreads) sum += slots[i];
  const double norm = sqrt(block_sum_d(sum, red));
  const bool finite = isfinite(norm);
  const double c64 = finite && norm > (double)max_norm ? (double)max_norm / norm : 1.0;
  const float f = (float)c64;
  const bool tiny = c64 < 0x1p-126 && c64 > 0.0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    stats[0] = (float)norm;
    stats[1] = f;
    if (!finite && flags) atomicOr(flags, DOBB_FLAG_NONFINITE_G);
  }
  // every tensor's own norm: a warp each
  const int lane = threadIdx.x & 31;
  for (int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < a.num; t += gridDim.x * (kThreads / 32)) {
    double s = 0.0;
    if (a.chunk0[t + 1] > a.chunk0[t]) {
      const int32_t last = cta_of(a, a.chunk0[t + 1] - 1);
      for (int32_t b = cta_of(a, a.chunk0[t]) + lane; b <= last; b += 32) s += slots[a.slot0 + b + t];
    }
    s = warp_sum_d(s);
    if (lane == 0) norms[t] = (float)sqrt(s);
  }
  if (!scale) return;
  const int32_t b = blockIdx.x, first = first_chunk(a, b);
  int32_t c = first_chunk(a, b + 1) - 1;
  // the n entries of tensor t from lo on
  auto scale_part = [&](int t, int64_t lo, int32_t n, int tid, int threads) {
    auto scaled = [&](auto* p, auto* o) {
      if (tiny)
        scale_tiny(p, o, n, c64, tid, threads);
      else
        scale_chunk(p, o, n, f, tid, threads);
    };
    const float* gf = static_cast<const float*>(a.g[t]) + lo;
    const __nv_bfloat16* gb = static_cast<const __nv_bfloat16*>(a.g[t]) + lo;
    float* of = static_cast<float*>(a.out[t]) + lo;
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(a.out[t]) + lo;
    if (a.g_bf16[t]) {
      if (a.out_bf16[t])
        scaled(gb, ob);
      else
        scaled(gb, of);
    } else if (a.out_bf16[t]) {
      scaled(gf, ob);
    } else {
      scaled(gf, of);
    }
  };
  const bool skip = f == 1.f;  // in place there is nothing to change
  for (int t = c >= first ? tensor_of(a, c) : 0; c >= first; --t) {
    int m = 0;
    while (m < kWarps && m <= t && a.numel[t - m] <= kSmall && a.chunk0[t - m] >= first) ++m;
    if (m > 1) {
      const int mine = t - (threadIdx.x >> 5);
      if (mine > t - m && !(skip && a.out[mine] == a.g[mine]))
        scale_part(mine, 0, (int32_t)a.numel[mine], lane, 32);
      t -= m - 1;
      c = a.chunk0[t] - 1;
      continue;
    }
    const int32_t stop = max(first, a.chunk0[t]);
    if (skip && a.out[t] == a.g[t]) c = min(c, stop - 1);
    for (; c >= stop; --c) {
      const int64_t lo = (int64_t)(c - a.chunk0[t]) * kChunk;
      scale_part(t, lo, (int32_t)min((int64_t)kChunk, a.numel[t] - lo), threadIdx.x, kThreads);
    }
  }
}

int grid_of(int64_t chunks) { return (int)(chunks < kCtas * kSms ? chunks : kCtas * kSms); }

// Slots of all launches; a launch takes up to kMaxTensors tensors.
dobb_status measure(int num, const int64_t* numel, size_t* slots) {
  if (num < 1 || !numel)
    return fail(DOBB_ERR_INVALID_ARG, "num_tensors must be > 0 and numel non-NULL");
  size_t n = 0;
  for (int t0 = 0; t0 < num; t0 += kMaxTensors) {
    const int k = num - t0 < kMaxTensors ? num - t0 : kMaxTensors;
    int64_t chunks = 0;
    for (int i = t0; i < t0 + k; ++i) {
      if (numel[i] < 0) return fail(DOBB_ERR_INVALID_ARG, "numel[%d] < 0", i);
      chunks += chunks_of(numel[i]);
      if (chunks > INT32_MAX) return fail(DOBB_ERR_UNSUPPORTED, "the tensors have too many entries");
    }
    n += grid_of(chunks) + k;
  }
  *slots = n;
  return DOBB_OK;
}

size_t slot_bytes(size_t slots) { return (slots * 8 + 255) / 256 * 256; }

struct ClipCall {
  int num;
  const void* const* G;
  const int32_t* grad_dtype;
  const int64_t* numel;
  float max_norm;
  void* const* out;
  const int32_t* out_dtype;
  float* stats;
  uint32_t* flags;
  double* slots;
  size_t num_slots;
  cudaStream_t stream;
};

// Refuses an output that shares memory with another output or another gradient:
// blocks in any order would read and write it.  (A tied weight listed twice and
// scaled in place comes out scaled once, twice or something in between.)
dobb_status check_overlap(const ClipCall& r) noexcept try {
  struct Extent {
    uintptr_t lo, hi;
    int tensor;
    bool written;
  };
  std::vector<Extent> e;
  e.reserve(2 * (size_t)r.num);
  auto add = [&](const void* p, int dtype, int i, bool written) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    e.push_back({lo, lo + (uintptr_t)r.numel[i] * lm::dtype_bytes(dtype), i, written});
  };
  for (int i = 0; i < r.num; ++i) {
    if (r.numel[i] == 0) continue;
    add(r.out[i], r.out_dtype[i], i, true);
    if (r.out[i] != r.G[i]) add(r.G[i], r.grad_dtype[i], i, false);
  }
  std::sort(e.begin(), e.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  // the ends of all extents, and of all written ones, so far
  const Extent *any = nullptr, *written = nullptr;
  for (const Extent& x : e) {
    const Extent* before = x.written ? any : written;
    if (before && x.lo < before->hi)
      return fail(DOBB_ERR_INVALID_ARG, "tensors %d and %d overlap, and one is written", std::min(x.tensor, before->tensor),
                  std::max(x.tensor, before->tensor));
    if (!any || x.hi > any->hi) any = &x;
    if (x.written && (!written || x.hi > written->hi)) written = &x;
  }
  return DOBB_OK;
} catch (...) {
  return fail(DOBB_ERR_STATE, "no memory for the list of tensors");
}

template <int K>
cudaError_t run_clip(const ClipCall& r) {
  Table<K> a;
  for (int phase = 0; phase < 2; ++phase) {
    a.slot0 = 0;
    for (int t0 = 0; t0 < r.num; t0 += kMaxTensors) {
      a.num = r.num - t0 < kMaxTensors ? r.num - t0 : kMaxTensors;
      if (phase == 0 || r.num > kMaxTensors) {
        a.chunk0[0] = 0;
        for (int i = 0; i < a.num; ++i) {
          a.g[i] = r.G[t0 + i];
          a.out[i] = r.out ? r.out[t0 + i] : nullptr;
          a.numel[i] = r.numel[t0 + i];
          a.g_bf16[i] = r.grad_dtype[t0 + i] == DOBB_BF16;
          a.out_bf16[i] = r.out && r.out_dtype[t0 + i] == DOBB_BF16;
          a.chunk0[i + 1] = a.chunk0[i] + (int32_t)chunks_of(a.numel[i]);
        }
        a.chunks = a.chunk0[a.num];
        a.grid = grid_of(a.chunks);
      }
      cudaLaunchConfig_t cfg{};
      cfg.blockDim = dim3(kThreads);
      cfg.stream = r.stream;
      cudaError_t e = cudaSuccess;
      if (phase == 0) {
        cfg.gridDim = dim3((unsigned)a.grid);
        if (a.grid > 0)
          e = cudaLaunchKernelEx(&cfg, clip_sums<K>, a, r.slots);
        else
          e = cudaMemsetAsync(r.slots + a.slot0, 0, (size_t)a.num * 8, r.stream);
      } else {
        // beside the end of the sums, when it follows them at once
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = r.num <= kMaxTensors && a.grid > 0 ? 1 : 0;
        const int norm_grid = (a.num + kThreads / 32 - 1) / (kThreads / 32);
        cfg.gridDim = dim3((unsigned)(r.out && a.grid > 0 ? a.grid : norm_grid));
        e = cudaLaunchKernelEx(&cfg, clip_scale<K>, a, (const double*)r.slots, (int64_t)r.num_slots, r.max_norm,
                               r.stats, r.stats + 2 + t0, t0 == 0 ? r.flags : nullptr,
                               (int)(r.out && a.grid > 0));
      }
      if (e != cudaSuccess) return e;
      a.slot0 += a.grid + a.num;
    }
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace dobb

using namespace dobb;

extern "C" size_t dobb_clip_grads_bytes(int num, const int64_t* numel) {
  size_t slots = 0;
  return measure(num, numel, &slots) == DOBB_OK ? slot_bytes(slots) : 0;
}

extern "C" dobb_status dobb_clip_grads(int num, const void* const* G, const int32_t* grad_dtype,
                                       const int64_t* numel, float max_norm, void* const* out,
                                       const int32_t* out_dtype, float* stats, uint32_t* flags,
                                       void* ws, size_t ws_bytes, void* stream) {
  size_t slots = 0;
  dobb_status st = measure(num, numel, &slots);
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
  if (ws_bytes < slot_bytes(slots))
    return fail(DOBB_ERR_STATE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes,
                slot_bytes(slots));
  const ClipCall r{num,   G,     grad_dtype, numel,
                   out ? max_norm : INFINITY,
                   out,   out_dtype, stats, flags, static_cast<double*>(ws),
                   slots, static_cast<cudaStream_t>(stream)};
  if (out) {
    st = check_overlap(r);
    if (st != DOBB_OK) return st;
  }
  const cudaError_t e = num <= kFewTensors ? run_clip<kFewTensors>(r) : run_clip<kMaxTensors>(r);
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "clipping launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
