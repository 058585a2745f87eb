// Layer norm over the rows of a matrix, and its gradients.
//
// With mean and variance of a row of D entries, rstd = 1 / sqrt(var + eps),
// xh = (x - mean) rstd, u = G w for the gradient G of the output:
//   out = xh w + b
//   dx = rstd (u - mean(u) - xh mean(u xh)),  dw = sum_rows G xh,  db = sum_rows G
// Both directions read a row once and hold it in the registers of the warps
// that share it.  Measured (of the copy rate): forward 16384 x 4096 fp32 to bf16 67 us (89 %),
// 8192 x 1600 bf16 15 us (51 %: four rows a group, so start and end are half of it);
// gradients 113 us (88 %) and 28 us (41 %, 5 of them the join of the blocks' sums).
#pragma once

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "lm_common.cuh"
#include "tc_ptx.cuh"

namespace dobb {
namespace {

// A block's fifteen warps are split into groups; a group takes a row at a time, up
// to 256 P columns a warp (rows of up to 128 columns share a warp).  The forward pass
// holds a row in few warps (P = 8), as a row's joins cost a warp as much as 300 entries
// do; the backward pass keeps its columns' sums of G xh and G in registers while the
// rows pass by (P = 2; 3 in the widest rows).  The parameters lie in shared memory.  One
// more warp copies the rows in, in bulk and as far ahead as shared memory holds: 16
// warps that load a row ahead into registers have 32 KB an SM in flight, too few for
// HBM (8192 x 1600 bf16: 22 us forward, 26 us backward).
constexpr int kWarps = 15;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxDim = kWarps * 256 * 3;  // beyond, blocks go over the rows in memory
constexpr int kMaxForwardDim = 16384;     // (the parameters and a row are in shared memory)
constexpr int kSms = 152;
constexpr int kMaxSlots = 16;       // of a group in the forward pass: kForwardSlots
constexpr int kForwardSlots = 4;
constexpr int kRingBytes = 200 * 1024;

// Rows on their way to shared memory.  Whoever waits for a turn of a slot has waited for
// its turn before: a barrier that is two phases behind reads like one that is ahead.
// Backward a slot has the rows of all groups, and all of them wait for it; forward, where
// rows are longer for the slots that fit, every group has slots of its own.
struct Ring {
  int32_t slots, slot_bytes;
  int32_t rows;      // of a block at a time, those of all groups
  int32_t first;     // where the first slot begins
  int32_t second;    // of a slot: where the second tensor's rows begin
  int32_t pitch[2];  // bytes from row to row, 0: the rows are one piece in memory
};

struct Shape {
  int32_t warps, groups, lanes;  // warps per row, groups, lanes per row (of one warp)
};

__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// The columns of one thread.  ALIGNED (every row starts on a multiple of four
// entries, D a multiple of 4): pieces of four neighbours, a piece a lane, so that fp32 in
// shared memory has no bank conflicts (with eight neighbours a lane, parameters as pairs:
// 8192 x 1600 26 us forward).  Otherwise single values, neighbouring lanes on
// neighbouring columns.  Either way warp w of a group has the columns 256 P w ... 256 P
// (w + 1) - 1.
template <int P, bool ALIGNED>
struct Columns {
  static constexpr int kPieces = 2 * P;
  int32_t first, some_lanes, count;  // count: pieces or values
  __device__ __forceinline__ Columns(int w, int lane, int32_t dim, int32_t lanes)
      : first(w * 256 * P + (ALIGNED ? lane * 4 : lane)), some_lanes(lanes) {
    const int32_t step = (ALIGNED ? 4 : 1) * this->lanes();
    count = first < dim ? min((dim - first + step - 1) / step, ALIGNED ? kPieces : 8 * P) : 0;
  }
  // (fewer than 32 in the narrowest rows only)
  __device__ __forceinline__ int32_t lanes() const { return P == 1 ? some_lanes : 32; }
  __device__ __forceinline__ int32_t piece(int q) const { return first + q * 4 * lanes(); }
  __device__ __forceinline__ int32_t single(int i) const { return first + i * lanes(); }
  __device__ __forceinline__ int32_t column(int i) const { return ALIGNED ? piece(i / 4) + i % 4 : single(i); }
  __device__ __forceinline__ bool has(int i) const { return (ALIGNED ? i / 4 : i) < count; }
};

// The values 4 q ... 4 q + 3 of a row in shared memory, as two pairs.  Only called
// where has(4 q); what lies behind the row's end reads as 0.
template <typename T, int P, bool ALIGNED>
__device__ __forceinline__ void read_four(uint64_t& lo, uint64_t& hi, const T* row, int q, const Columns<P, ALIGNED>& c) {
  if (ALIGNED) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(row + c.piece(q));
      lo = lm::pack2(a.x, a.y);
      hi = lm::pack2(a.z, a.w);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(row + c.piece(q));
      lo = lm::pack2(lm::bf16_lo(a.x), lm::bf16_hi(a.x));
      hi = lm::pack2(lm::bf16_lo(a.y), lm::bf16_hi(a.y));
    }
  } else {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = c.has(4 * q + i) ? load_f32(row + c.single(4 * q + i)) : 0.f;
    lo = lm::pack2(v[0], v[1]);
    hi = lm::pack2(v[2], v[3]);
  }
}

template <typename T, int P, bool ALIGNED>
__device__ __forceinline__ void store_four(T* row, uint64_t lo, uint64_t hi, int q, const Columns<P, ALIGNED>& c) {
  float f[4];
  lm::unpack2(lo, f[0], f[1]);
  lm::unpack2(hi, f[2], f[3]);
  if (ALIGNED) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(row + c.piece(q)) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
      *reinterpret_cast<uint2*>(row + c.piece(q)) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c.has(4 * q + i)) store_f32(row + c.single(4 * q + i), f[i]);
  }
}

// pair i with what lies behind the row's end as zeros (ALIGNED: pieces end with it)
template <int P, bool ALIGNED>
__device__ __forceinline__ uint64_t only(uint64_t v, int i, const Columns<P, ALIGNED>& c) {
  if (ALIGNED) return v;
  float lo, hi;
  lm::unpack2(v, lo, hi);
  return lm::pack2(lo, c.has(2 * i + 1) ? hi : 0.f);
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  lm::unpack2(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ uint64_t both(float v) { return lm::pack2(v, v); }

// The parameters to shared memory, by the first `threads` threads.
__device__ __forceinline__ void copy_params(float* to, const void* p, int bf16, int32_t dim, float none, int threads) {
  const int32_t fours = p && !(reinterpret_cast<uintptr_t>(p) & (bf16 ? 7 : 15)) ? dim / 4 : 0;
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < fours; i += threads) {
    float4 v;
    if (bf16) {
      const uint2 a = __ldg(static_cast<const uint2*>(p) + i);
      v = make_float4(lm::bf16_lo(a.x), lm::bf16_hi(a.x), lm::bf16_lo(a.y), lm::bf16_hi(a.y));
    } else {
      v = __ldg(static_cast<const float4*>(p) + i);
    }
    to[4 * i] = v.x;
    to[4 * i + 1] = v.y;
    to[4 * i + 2] = v.z;
    to[4 * i + 3] = v.w;
  }
#pragma unroll 4
  for (int32_t i = 4 * fours + threadIdx.x; i < dim; i += threads)
    to[i] = !p ? none : bf16 ? load_f32(static_cast<const __nv_bfloat16*>(p) + i) : static_cast<const float*>(p)[i];
}

struct RingBarriers {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int32_t late;  // a wait gave up: all others do
};
struct GroupBarriers {
  uint64_t full[kWarps * kForwardSlots], empty[kWarps * kForwardSlots];
  int32_t late;
};
constexpr uint64_t kWaitNs = 2000000000ull;
// How long a wait lasts at most, and how many rows are copied in (all of them but in the
// self-test of the waits).
struct Patience {
  uint64_t limit;
  int64_t loaded;
};

template <typename B>
__device__ __forceinline__ void ring_init(B& b, int slots, int arrivals) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < slots; ++s) {
      ptx::mbar_init(&b.full[s], 1);
      ptx::mbar_init(&b.empty[s], arrivals);
    }
    b.late = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
}
template <typename B>
__device__ __forceinline__ bool ring_wait(B& b, uint64_t* bar, uint32_t parity, uint64_t limit) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*(volatile int32_t*)&b.late) return false;
    if (ptx::global_timer_ns() - t0 > limit) {
      *(volatile int32_t*)&b.late = 1;
      return false;
    }
  }
  return true;
}

// `n` entries from p to the image of their 16-byte granules; the granules at the
// tensor's ends [begin, end) only as far as it goes.  Returns the bytes in flight.
template <typename T>
__device__ __forceinline__ uint32_t copy_in(unsigned char* image, const T* p, int64_t n, const T* begin, const T* end, uint64_t* bar) {
  const uintptr_t from = reinterpret_cast<uintptr_t>(p), to = from + (uint64_t)n * sizeof(T);
  uintptr_t lo = from & ~(uintptr_t)15, hi = (to + 15) & ~(uintptr_t)15;
  const uintptr_t granule = lo;
  const auto by_value = [&](uintptr_t a, uintptr_t b) {
    for (; a < b; a += sizeof(T)) *reinterpret_cast<T*>(image + (a - granule)) = *reinterpret_cast<const T*>(a);
    ptx::fence_proxy_async_smem();  // a later turn's copy comes over it
  };
  if (lo < reinterpret_cast<uintptr_t>(begin)) {
    lo += 16;
    by_value(from, lo < to ? lo : to);
  }
  if (hi > reinterpret_cast<uintptr_t>(end) && hi > lo) {
    hi -= 16;
    by_value(hi > from ? hi : from, to);
  }
  if (hi <= lo) return 0;
  ptx::bulk_load(image + (lo - granule), reinterpret_cast<const void*>(lo), (uint32_t)(hi - lo), bar);
  return (uint32_t)(hi - lo);
}

// Row i of the rows from row0 on in a slot.
template <typename T>
__device__ __forceinline__ const T* ring_row(const unsigned char* slot, int32_t pitch, const T* row0, int64_t stride, int i, int32_t dim) {
  if (pitch == 0) return reinterpret_cast<const T*>(slot + (reinterpret_cast<uintptr_t>(row0) & 15)) + (int64_t)i * dim;
  return reinterpret_cast<const T*>(slot + (size_t)i * pitch + (reinterpret_cast<uintptr_t>(row0 + i * stride) & 15));
}

// sum over `lanes` neighbouring lanes, a power of two
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  if (lanes == 32) return warp_sum(v);
  for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float param(const void* p, int bf16, int64_t i) {
  return bf16 ? load_f32(static_cast<const __nv_bfloat16*>(p) + i) : static_cast<const float*>(p)[i];
}

// xh of an entry is (x h - mean) rstd: h = 1, or 2^-100 in rows whose sums or
// differences would leave fp32.
constexpr float kDown = 0x1p-100f;
// rstd of a row scaled down.  Beyond fp32 (rstd above 2^28 although entries of 2^100 have
// neighbours 2^77 away) only where every difference is 0: any finite factor will do.
__device__ __forceinline__ float in_range(float scaled) { return scaled == INFINITY ? FLT_MAX : scaled; }
struct RowScale {
  float h, mean, rstd;
  __device__ __forceinline__ float xhat(float x) const { return fmaf(x, h, -mean) * rstd; }
};

// mean and rstd of the row, from those of entries scaled by h
__device__ __forceinline__ RowScale row_scale(float h, float mean, float var, float eps, float& row_mean, float& row_rstd) {
  if (h == 1.f) {
    row_mean = mean;
    row_rstd = 1.f / sqrtf(var + eps);
    return {1.f, mean, row_rstd};
  }
  const double rstd = 1.0 / sqrt((double)var * 0x1p200 + (double)eps);
  row_mean = mean * 0x1p100f;
  row_rstd = (float)rstd;
  return {h, mean, in_range((float)(rstd * 0x1p100))};
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

__device__ __forceinline__ RowScale given_scale(float mean, float rstd) {
  const float h = fabsf(mean) < 0x1p100f && rstd > kDown ? 1.f : kDown;
  return {h, mean * h, h == 1.f ? rstd : in_range(rstd * 0x1p100f)};
}

// A block's sum of f(i), i < n: eight at a time of each thread in fp32, then in fp64.
template <typename F>
__device__ __forceinline__ double block_sum_of(int32_t n, double* red, F f) {
  double total = 0.0;
#pragma unroll 1
  for (int32_t i0 = threadIdx.x; i0 < n; i0 += 8 * kThreads) {
    float part = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u * kThreads < n) part += f(i0 + u * kThreads);
    total += (double)part;
  }
  return block_sum_d(total, red);
}

// ------------------------------------------------------------------- host

struct Plan {
  bool wide;  // more columns than a block's registers hold
  int p;
  Shape shape;
  unsigned blocks;   // of the main kernel
  int32_t partials;  // blocks' sums to join
};

inline int rows_at_once(const Shape& s) { return s.groups * (32 / s.lanes); }

// the rows over the blocks
void spread(Plan& p, int64_t rows) {
  const int64_t at_once = rows_at_once(p.shape);
  p.blocks = (unsigned)std::min<int64_t>((rows + at_once - 1) / at_once, kSms);
  p.partials = (int32_t)p.blocks;
}

Plan plan(int64_t rows, int64_t dim, bool backward) {
  Plan r{};
  r.wide = dim > (backward ? kMaxDim : kMaxForwardDim);
  if (r.wide) {
    const int64_t chunks = (dim + kThreads - 1) / kThreads;
    r.partials = (int32_t)std::min<int64_t>(rows, std::max<int64_t>(1, 4 * kSms / chunks));
    r.blocks = (unsigned)(backward ? chunks * r.partials : std::min<int64_t>(rows, 4 * kSms));
    return r;
  }
  if (backward) {
    // as many rows at a time as possible, in as few columns a lane (20000 x 2048 bf16: three rows
    // of P = 2 62 us, five of P = 3 55; 16000 x 2500, three rows either way, 61 and 66)
    for (int p = 1; p <= 3; ++p)
      if (dim <= 256 * p * kWarps && (r.p == 0 || kWarps / ((dim + 256 * p - 1) / (256 * p)) > kWarps / ((dim + 256 * r.p - 1) / (256 * r.p)))) r.p = p;
  } else {
    r.p = 1;
    while (r.p < (rows <= 2 * kSms && dim <= 512 * kWarps ? 2 : 8) && dim > 256 * r.p) r.p *= 2;  // (few rows: more warps for each)
  }
  r.shape.warps = (int)((dim + 256 * r.p - 1) / (256 * r.p));
  r.shape.lanes = 32;
  while (r.shape.lanes > 4 && dim <= 4 * r.shape.lanes) r.shape.lanes /= 2;
  // few rows: a block for each
  const int64_t per_sm = (rows + kSms - 1) / kSms, in_warp = 32 / r.shape.lanes;
  r.shape.groups = (int)std::min<int64_t>(kWarps / r.shape.warps, (per_sm + in_warp - 1) / in_warp);
  spread(r, rows);
  return r;
}

// one tensor's rows in a slot
int32_t image_bytes(int64_t rows, int64_t dim, int64_t stride, size_t bytes, int32_t count, int32_t& pitch) {
  const bool one_piece = stride == dim || rows == 1;
  pitch = one_piece ? 0 : (int32_t)((dim * bytes + 30) / 16 * 16);
  return one_piece ? (int32_t)((count * dim * bytes + 30) / 16 * 16) : count * pitch;
}

Ring ring_of(const Plan& p, int64_t rows, int64_t dim, int64_t x_stride, int x_dtype, int64_t g_stride, int g_dtype, bool backward) {
  Ring r{};
  r.rows = rows_at_once(p.shape);
  const int32_t slot_rows = backward ? r.rows : 32 / p.shape.lanes;
  r.second = image_bytes(rows, dim, x_stride, lm::dtype_bytes(x_dtype), slot_rows, r.pitch[0]);
  r.slot_bytes = r.second;
  if (backward) r.slot_bytes += image_bytes(rows, dim, g_stride, lm::dtype_bytes(g_dtype), slot_rows, r.pitch[1]);
  const int64_t turns = (rows + (int64_t)p.blocks * r.rows - 1) / ((int64_t)p.blocks * r.rows);
  r.first = (int32_t)(((dim + 3) / 4 * 16 * (backward ? 1 : 2) + 127) / 128 * 128);
  const int64_t room = (kRingBytes - r.first) / (backward ? r.slot_bytes : r.slot_bytes * p.shape.groups);
  r.slots = (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)(backward ? kMaxSlots : kForwardSlots), room, turns}));
  return r;
}

// the parameters and the ring, and in their place at the end the sums of the groups
size_t ring_smem(const Plan& p, const Ring& r, bool backward, bool sums) {
  return std::max((size_t)r.first + (size_t)r.slots * r.slot_bytes * (backward ? 1 : p.shape.groups), sums ? (size_t)p.shape.warps * p.shape.groups * 32 * 8 * p.p * 4 : 0);
}

// The forward pass's: one group less where a slot for each does not fit (fp32 rows of 14333 to
// 14336 columns, parameters and two rows; the backward pass's shapes all fit).
Ring forward_ring(Plan& p, int64_t rows, int64_t dim, int64_t x_stride, int x_dtype) {
  Ring r = ring_of(p, rows, dim, x_stride, x_dtype, 0, 0, false);
  while (ring_smem(p, r, false, false) > (size_t)lm::kMostSmem && p.shape.groups > 1) {
    --p.shape.groups;
    spread(p, rows);
    r = ring_of(p, rows, dim, x_stride, x_dtype, 0, 0, false);
  }
  return r;
}

dobb_status check_norm(int64_t rows, int64_t dim, int x_dtype, int64_t x_stride, int other_dtype, int64_t other_stride,
                       int param_dtype) {
  if (lm::bad_dtype(x_dtype) || lm::bad_dtype(other_dtype) || lm::bad_dtype(param_dtype))
    return fail(DOBB_ERR_INVALID_ARG, "every dtype must be DOBB_F32 or DOBB_BF16");
  if (rows < 0) return fail(DOBB_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
  if (dim < 1 || dim > INT32_MAX / 2)
    return fail(DOBB_ERR_INVALID_ARG, "dim must lie in [1, 2^30) (got %lld)", (long long)dim);
  if (rows > 1 && (x_stride < dim || other_stride < dim))
    return fail(DOBB_ERR_INVALID_ARG, "a row stride is below dim %lld", (long long)dim);
  if (rows > 1 && (x_stride > INT64_MAX / 8 / rows || other_stride > INT64_MAX / 8 / rows))
    return fail(DOBB_ERR_UNSUPPORTED, "rows times a row stride is too large");
  return DOBB_OK;
}

dobb_status check_patience(const Patience& p, int64_t rows) {
  if (p.loaded < 0 || p.loaded > rows || p.limit == 0 || p.limit > 5000000000ull)
    return fail(DOBB_ERR_INVALID_ARG, "loaded_rows must lie in [0, rows], timeout_ns in [1, 5e9]");
  return DOBB_OK;
}

bool aligned_rows(const void* p, int64_t stride, int dtype, int64_t rows) {
  return !lm::misaligned(p, 4 * lm::dtype_bytes(dtype)) && (rows <= 1 || stride % 4 == 0);
}

template <auto kernel, typename A>
cudaError_t launch(unsigned blocks, unsigned threads, size_t smem, cudaStream_t s, bool programmatic, const A& args) {
  if (smem > 0) {
    const cudaError_t e = lm::allow_smem<kernel>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = programmatic ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace
}  // namespace dobb
