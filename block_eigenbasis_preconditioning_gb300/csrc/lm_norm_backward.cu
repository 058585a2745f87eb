// The gradients of layer norm.
#include "lm_norm.cuh"

namespace dobb {
namespace {

struct NormGradArgs {
  const void *grad, *x;
  int64_t rows, grad_stride, x_stride;
  int32_t dim;
  const void* weight;
  int32_t param_bf16;
  const float *mean, *rstd;
  void* dx;
  int64_t dx_stride;
  float* partial;    // blocks x 2 x dim sums of G xh and of G, or NULL
  float2* row_sums;  // long rows: mean(u) and mean(u xh) of every row
  int32_t row_blocks;
  Shape shape;
  Ring ring;
  Patience patience;
};

struct JoinArgs {
  const float* partial;
  int32_t blocks, dim;
  void *dweight, *dbias;
  int32_t bf16, accumulate;
};

// Wait for the kernel before (programmatic dependent launch), and let the next one be launched.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;"); }

// The backward pass's producer warp: block after block of the rows that this block of
// threads takes.
template <typename TX, typename TG>
__device__ __forceinline__ void produce(RingBarriers& b, unsigned char* raw, const Ring& ring, const TX* x, int64_t x_stride, const TG* g,
                                        int64_t g_stride, int64_t rows, int32_t dim, const Patience& patience) {
  const int lane = threadIdx.x & 31;
  const TX* x_end = x + (rows - 1) * x_stride + dim;
  const TG* g_end = g + (rows - 1) * g_stride + dim;
  uint32_t k = 0;
  bool ok = true;
  for (int64_t r0 = (int64_t)blockIdx.x * ring.rows; r0 < patience.loaded && ok; r0 += (int64_t)gridDim.x * ring.rows, ++k) {
    const uint32_t slot = k % ring.slots, turn = k / ring.slots;
    if (turn > 0) ok = __all_sync(0xffffffffu, ring_wait(b, &b.empty[slot], (turn - 1) & 1, patience.limit));
    if (!ok) break;
    const int32_t count = (int32_t)min((int64_t)ring.rows, rows - r0);
    unsigned char* to = raw + (size_t)slot * ring.slot_bytes;
    uint32_t bytes = 0;
    if (ring.pitch[0] == 0) {
      if (lane == 0) bytes += copy_in(to, x + r0 * x_stride, (int64_t)count * dim, x, x_end, &b.full[slot]);
    } else {
      for (int i = lane; i < count; i += 32)
        bytes += copy_in(to + (size_t)i * ring.pitch[0], x + (r0 + i) * x_stride, (int64_t)dim, x, x_end, &b.full[slot]);
    }
    to += ring.second;
    if (ring.pitch[1] == 0) {
      if (lane == 1) bytes += copy_in(to, g + r0 * g_stride, (int64_t)count * dim, g, g_end, &b.full[slot]);
    } else {
      for (int i = lane; i < count; i += 32)
        bytes += copy_in(to + (size_t)i * ring.pitch[1], g + (r0 + i) * g_stride, (int64_t)dim, g, g_end, &b.full[slot]);
    }
    bytes = __reduce_add_sync(0xffffffffu, bytes);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_expect_tx(&b.full[slot], bytes);
  }
  // no copy is in flight when the block ends
  for (uint32_t p = k > (uint32_t)ring.slots ? k - ring.slots : 0; p < k; ++p)
    ptx::mbar_wait(&b.full[p % ring.slots], (p / ring.slots) & 1);
}

template <typename TX, typename TG, int P, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1) norm_backward(const __grid_constant__ NormGradArgs a) {
  extern __shared__ __align__(128) unsigned char raw[];
  __shared__ RingBarriers bar;
  __shared__ float2 red[2][kWarps];
  launch_next();
  const Shape sp = a.shape;
  const int warps = sp.warps * sp.groups;
  float* weight = reinterpret_cast<float*>(raw);
  unsigned char* ring = raw + a.ring.first;
  ring_init(bar, a.ring.slots, warps);
  const TX* x = static_cast<const TX*>(a.x);
  const TG* g = static_cast<const TG*>(a.grad);
  const int warp = threadIdx.x >> 5;
  const int in_warp = threadIdx.x & 31, lane = in_warp & (sp.lanes - 1);
  const int group = warp / sp.warps, w = warp - group * sp.warps, base = group * sp.warps;
  const Columns<P, ALIGNED> c(w, lane, a.dim, sp.lanes);
  uint64_t dw[4 * P], db[4 * P];
#pragma unroll
  for (int i = 0; i < 4 * P; ++i) dw[i] = db[i] = 0;
  if (warp == warps) {
    produce<TX, TG>(bar, ring, a.ring, x, a.x_stride, g, a.grad_stride, a.rows, a.dim, a.patience);
  } else {
    copy_params(weight, a.weight, a.param_bf16, a.dim, 1.f, warps * 32);
    TX* dx = static_cast<TX*>(a.dx);
    const float inv_dim = 1.f / (float)a.dim;
    // (a group's place in a slot is fixed)
    const int mine = group * (32 / sp.lanes) + in_warp / sp.lanes;
    const int64_t step = (int64_t)gridDim.x * a.ring.rows, block0 = (int64_t)blockIdx.x * a.ring.rows;
    // the row's place in a slot, and where its image begins within 16 bytes
    const uint32_t xr = mine * (a.ring.pitch[0] ? a.ring.pitch[0] : a.dim * (int32_t)sizeof(TX));
    const uint32_t gr = a.ring.second + mine * (a.ring.pitch[1] ? a.ring.pitch[1] : a.dim * (int32_t)sizeof(TG));
    uint32_t x_pad = (uint32_t)reinterpret_cast<uintptr_t>(x + (block0 + (a.ring.pitch[0] ? mine : 0)) * a.x_stride) & 15;
    uint32_t g_pad = (uint32_t)reinterpret_cast<uintptr_t>(g + (block0 + (a.ring.pitch[1] ? mine : 0)) * a.grad_stride) & 15;
    const uint32_t x_next = (uint32_t)(step * a.x_stride * (int64_t)sizeof(TX)), g_next = (uint32_t)(step * a.grad_stride * (int64_t)sizeof(TG));
    float next_mean = 0.f, next_rstd = 0.f;
    int64_t row = block0 + mine;
    const auto fetch = [&](int64_t r) {
      if (r < a.rows) {
        next_mean = a.mean[r];
        next_rstd = a.rstd[r];
      }
    };
    fetch(row);
    asm volatile("bar.sync 15, %0;" ::"r"(warps * 32) : "memory");  // the parameters are there
    int buf = 0;
    uint32_t slot = 0, phase = 0;
    bool ok = true;  // once a wait gave up the phases are not known any more: all later rows are lost
    for (; row - mine < a.rows; row += step) {
      ok = __all_sync(0xffffffffu, ok && ring_wait(bar, &bar.full[slot], phase, a.patience.limit));
      uint64_t xh[4 * P], gv[4 * P];
      const RowScale r = given_scale(next_mean, next_rstd);
      const float rstd = ok ? next_rstd : NAN;
      if (row < a.rows) {
        const TX* px = reinterpret_cast<const TX*>(ring + slot * a.ring.slot_bytes + xr + x_pad);
        const TG* pg = reinterpret_cast<const TG*>(ring + slot * a.ring.slot_bytes + gr + g_pad);
#pragma unroll
        for (int q = 0; q < 2 * P; ++q) {
          if (!c.has(4 * q)) break;
          read_four<TX, P, ALIGNED>(xh[2 * q], xh[2 * q + 1], px, q, c);
          read_four<TG, P, ALIGNED>(gv[2 * q], gv[2 * q + 1], pg, q, c);
        }
      }
      x_pad = (x_pad + x_next) & 15;
      g_pad = (g_pad + g_next) & 15;
      fetch(row + step);
      __syncwarp();
      if (in_warp == 0) ptx::mbar_arrive(&bar.empty[slot]);
      if (++slot == (uint32_t)a.ring.slots) {
        slot = 0;
        phase ^= 1;
      }
      uint64_t t1 = 0, t2 = 0;
      if (row < a.rows) {
        // xh = x rstd - mean rstd; x - mean first where the two cancel or leave fp32
        const bool apart = r.h != 1.f || !(fabsf(r.mean) * r.rstd < 16.f);
        const uint64_t h2 = both(r.h), minus_m = both(-r.mean), scale = both(ok ? r.rstd : NAN), offset = both(apart ? 0.f : -r.mean * r.rstd);
#pragma unroll
        for (int q = 0; q < 2 * P; ++q) {
          if (!c.has(4 * q)) break;
          uint64_t p[2];
          read_four<float, P, ALIGNED>(p[0], p[1], weight, q, c);
#pragma unroll
          for (int i = 2 * q; i < 2 * q + 2; ++i) {
            uint64_t &xi = xh[i], &gi = gv[i];
            if (apart) xi = lm::fma2(xi, h2, minus_m);
            xi = only(lm::fma2(xi, scale, offset), i, c);
            dw[i] = lm::fma2(gi, xi, dw[i]);
            db[i] = lm::add2(gi, db[i]);
            gi = lm::mul2(gi, p[i & 1]);
            t1 = lm::add2(gi, t1);
            t2 = lm::fma2(gi, xi, t2);
          }
        }
        if (!ok) {
#pragma unroll
          for (int i = 0; i < 4 * P; ++i) db[i] = both(NAN);
        }
      }
      float s1 = sum2(t1), s2 = sum2(t2);
      if (sp.lanes == 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
          s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
      } else {
        s1 = lanes_sum(s1, sp.lanes);
        s2 = lanes_sum(s2, sp.lanes);
      }
      if (sp.warps > 1) {
        if (in_warp == 0) red[buf][warp] = make_float2(s1, s2);
        __syncwarp();
        group_sync(group, sp.warps * 32);
        s1 = s2 = 0.f;
        for (int i = 0; i < sp.warps; ++i) {
          const float2 q = red[buf][base + i];
          s1 += q.x;
          s2 += q.y;
        }
        buf ^= 1;
      }
      if (!dx || row >= a.rows) continue;
      // rstd u - xh (rstd m2) - rstd m1
      const uint64_t scale = both(rstd), by_xh = both(-s2 * inv_dim * rstd), offset = both(-s1 * inv_dim * rstd);
      TX* to = dx + row * a.dx_stride;
#pragma unroll
      for (int q = 0; q < 2 * P; ++q) {
        if (!c.has(4 * q)) break;
        store_four<TX, P, ALIGNED>(to, lm::fma2(gv[2 * q], scale, lm::fma2(xh[2 * q], by_xh, offset)),
                                   lm::fma2(gv[2 * q + 1], scale, lm::fma2(xh[2 * q + 1], by_xh, offset)), q, c);
      }
    }
  }
  if (!a.partial) return;
  // the groups' sums, in their order, where the ring was
  float* sums = reinterpret_cast<float*>(raw);
  const int32_t width = sp.warps * sp.lanes * 8 * P, at_once = sp.groups * (32 / sp.lanes);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    if (warp < warps) {
      float* to = sums + (group * (32 / sp.lanes) + in_warp / sp.lanes) * width;
#pragma unroll
      for (int i = 0; i < 4 * P; ++i) {
        float lo, hi;
        lm::unpack2(which ? db[i] : dw[i], lo, hi);
        to[c.column(2 * i)] = lo;
        to[c.column(2 * i + 1)] = hi;
      }
    }
    __syncthreads();
    float* to = a.partial + ((int64_t)blockIdx.x * 2 + which) * a.dim;
    for (int32_t j = threadIdx.x; j < a.dim; j += blockDim.x) {
      float s = sums[j];
      for (int k = 1; k < at_once; ++k) s += sums[k * width + j];
      to[j] = s;
    }
  }
}

// Long rows, first kernel: mean(u) and mean(u xh) of every row.
template <typename TX, typename TG>
__global__ void __launch_bounds__(kThreads) norm_backward_rows(const NormGradArgs a) {
  __shared__ double red[32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride;
    const TG* g = static_cast<const TG*>(a.grad) + row * a.grad_stride;
    const RowScale r = given_scale(a.mean[row], a.rstd[row]);
    const auto u = [&](int32_t i) { return load_f32(g + i) * (a.weight ? param(a.weight, a.param_bf16, i) : 1.f); };
    const double m1 = block_sum_of(a.dim, red, u) / a.dim;
    const double m2 = block_sum_of(a.dim, red, [&](int32_t i) { return u(i) * r.xhat(load_f32(x + i)); }) / a.dim;
    if (threadIdx.x == 0) a.row_sums[row] = make_float2((float)m1, (float)m2);
  }
}

// Long rows, second kernel: a column a thread, every row_blocks-th row a block.
constexpr int kLongRows = 8;  // in flight
template <typename TX, typename TG>
__global__ void __launch_bounds__(kThreads) norm_backward_columns(const NormGradArgs a) {
  launch_next();
  const int32_t chunks = (a.dim + kThreads - 1) / kThreads;
  const int32_t part = blockIdx.x / chunks, i = (blockIdx.x - part * chunks) * kThreads + threadIdx.x;
  if (i >= a.dim) return;
  const float wt = a.weight ? param(a.weight, a.param_bf16, i) : 1.f;
  double dw = 0.0, db = 0.0;
#pragma unroll 1
  for (int64_t row0 = part; row0 < a.rows; row0 += kLongRows * (int64_t)a.row_blocks) {
    float x[kLongRows], g[kLongRows], pw = 0.f, pb = 0.f;
    // (all loads first: dx may be written over x or the gradient)
#pragma unroll
    for (int u = 0; u < kLongRows; ++u) {
      const int64_t row = row0 + u * (int64_t)a.row_blocks;
      x[u] = row < a.rows ? load_f32(static_cast<const TX*>(a.x) + row * a.x_stride + i) : 0.f;
      g[u] = row < a.rows ? load_f32(static_cast<const TG*>(a.grad) + row * a.grad_stride + i) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kLongRows; ++u) {
      const int64_t row = row0 + u * (int64_t)a.row_blocks;
      if (row >= a.rows) break;
      const float xh = given_scale(a.mean[row], a.rstd[row]).xhat(x[u]);
      pw = fmaf(g[u], xh, pw);
      pb += g[u];
      if (a.dx) {
        const float2 m = a.row_sums[row];
        store_f32(static_cast<TX*>(a.dx) + row * a.dx_stride + i, a.rstd[row] * (fmaf(g[u], wt, -m.x) - xh * m.y));
      }
    }
    dw += (double)pw;
    db += (double)pb;
  }
  if (!a.partial) return;
  a.partial[(int64_t)part * 2 * a.dim + i] = (float)dw;
  a.partial[((int64_t)part * 2 + 1) * a.dim + i] = (float)db;
}

// The blocks' sums, in a fixed order: 32 columns a block, sixteen threads each.
constexpr int kJoinThreads = 512, kJoinRows = kJoinThreads / 32;
__global__ void __launch_bounds__(kJoinThreads) norm_join(const JoinArgs a) {
  __shared__ float part[kJoinRows][33];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int32_t chunks = (a.dim + 31) / 32;
  const int which = blockIdx.x / chunks;
  const int32_t j = (blockIdx.x - which * chunks) * 32 + lane;
  wait_for_previous();
  float s = 0.f;
  if (j < a.dim) {
#pragma unroll 10
    for (int b = r; b < a.blocks; b += kJoinRows) s += a.partial[((int64_t)b * 2 + which) * a.dim + j];
  }
  part[r][lane] = s;
  __syncthreads();
  void* out = which ? a.dbias : a.dweight;
  if (r != 0 || j >= a.dim || !out) return;
#pragma unroll
  for (int k = 1; k < kJoinRows; ++k) s += part[k][lane];
  if (a.bf16) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + j;
    store_f32(o, a.accumulate ? load_f32(o) + s : s);
  } else {
    float* o = static_cast<float*>(out) + j;
    *o = a.accumulate ? *o + s : s;
  }
}

template <typename TX, typename TG>
cudaError_t launch_backward(const NormGradArgs& a, const Plan& p, bool aligned, cudaStream_t s) {
  if (p.wide) {
    const cudaError_t e = launch<norm_backward_rows<TX, TG>>((unsigned)std::min<int64_t>(a.rows, 4 * kSms), kThreads, 0, s, false, a);
    return e == cudaSuccess ? launch<norm_backward_columns<TX, TG>>(p.blocks, kThreads, 0, s, false, a) : e;
  }
  const unsigned threads = 32 * (p.shape.warps * p.shape.groups + 1);
  const size_t smem = ring_smem(p, a.ring, true, a.partial != nullptr);
  const auto go = [&](auto columns) {
    constexpr int P = decltype(columns)::value;
    return aligned ? launch<norm_backward<TX, TG, P, true>>(p.blocks, threads, smem, s, false, a)
                   : launch<norm_backward<TX, TG, P, false>>(p.blocks, threads, smem, s, false, a);
  };
  return p.p == 1   ? go(std::integral_constant<int, 1>{})
         : p.p == 2 ? go(std::integral_constant<int, 2>{})
                    : go(std::integral_constant<int, 3>{});
}

// the workspace: the blocks' sums, then (long rows) the rows' sums
size_t partial_bytes(const Plan& p, int64_t dim) { return ((size_t)p.partials * 2 * (size_t)dim * 4 + 255) / 256 * 256; }
size_t workspace_bytes_of(const Plan& p, int64_t rows, int64_t dim) {
  return partial_bytes(p, dim) + (p.wide ? (size_t)rows * sizeof(float2) : 0) + 256;
}

}  // namespace
}  // namespace dobb

using namespace dobb;

extern "C" size_t dobb_layer_norm_backward_bytes(int64_t rows, int64_t dim) {
  if (check_norm(rows, dim, 0, dim, 0, dim, 0) != DOBB_OK) return 0;
  if (rows > ((int64_t)1 << 48)) {
    fail(DOBB_ERR_UNSUPPORTED, "too many rows (%lld)", (long long)rows);
    return 0;
  }
  return workspace_bytes_of(plan(std::max<int64_t>(rows, 1), dim, true), rows, dim);
}

namespace {

// selftest: the waits' limit and the rows that are copied in, or NULL
dobb_status layer_norm_backward(const void* grad, dobb_dtype grad_dtype, int64_t grad_stride, const void* x, dobb_dtype x_dtype,
                                int64_t rows, int64_t dim, int64_t x_stride, const void* weight, dobb_dtype param_dtype,
                                const float* mean, const float* rstd, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                dobb_dtype dparam_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream,
                                const Patience* selftest) {
  dobb_status st = check_norm(rows, dim, x_dtype, x_stride, grad_dtype, grad_stride, param_dtype);
  if (st != DOBB_OK) return st;
  if (lm::bad_dtype(dparam_dtype)) return fail(DOBB_ERR_INVALID_ARG, "every dtype must be DOBB_F32 or DOBB_BF16");
  if (accumulate != 0 && accumulate != 1) return fail(DOBB_ERR_INVALID_ARG, "accumulate must be 0 or 1 (got %d)", accumulate);
  if (dx && rows > 1 && (dx_stride < dim || dx_stride > INT64_MAX / 8 / rows))
    return fail(DOBB_ERR_INVALID_ARG, "dx_stride %lld does not fit rows of %lld", (long long)dx_stride, (long long)dim);
  if (rows > 0 && (!grad || !x || !mean || !rstd))
    return fail(DOBB_ERR_INVALID_ARG, "grad, x, mean and rstd must be non-NULL");
  if (lm::misaligned(grad, lm::dtype_bytes(grad_dtype)) || lm::misaligned(x, lm::dtype_bytes(x_dtype)) ||
      lm::misaligned(dx, lm::dtype_bytes(x_dtype)) || lm::misaligned(weight, lm::dtype_bytes(param_dtype)) ||
      lm::misaligned(dweight, lm::dtype_bytes(dparam_dtype)) || lm::misaligned(dbias, lm::dtype_bytes(dparam_dtype)) ||
      lm::misaligned(mean, 4) || lm::misaligned(rstd, 4))
    return fail(DOBB_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
  const size_t need = dobb_layer_norm_backward_bytes(rows, dim);
  if (need == 0) return DOBB_ERR_UNSUPPORTED;
  if (!dx && !dweight && !dbias) return DOBB_OK;
  if (!workspace || lm::misaligned(workspace, 256))
    return fail(DOBB_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < need)
    return fail(DOBB_ERR_STATE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, need);
  const bool on_grad = dx == grad && x_dtype == grad_dtype && (rows <= 1 || dx_stride == grad_stride);
  const bool on_x = dx == x && (rows <= 1 || dx_stride == x_stride);
  lm::Extents ext;
  ext.read("grad", grad, rows, dim, grad_stride, grad_dtype, on_grad);
  ext.read("x", x, rows, dim, x_stride, x_dtype, on_x);
  ext.read("weight", weight, 1, dim, dim, param_dtype);
  ext.read("mean", mean, 1, rows, rows, DOBB_F32);
  ext.read("rstd", rstd, 1, rows, rows, DOBB_F32);
  ext.write("dx", dx, rows, dim, dx_stride, x_dtype, on_grad || on_x);
  ext.write("dweight", dweight, 1, dim, dim, dparam_dtype);
  ext.write("dbias", dbias, 1, dim, dim, dparam_dtype);
  ext.write("workspace", workspace, 1, (int64_t)(need / 4), (int64_t)(need / 4), DOBB_F32);
  if ((st = ext.check()) != DOBB_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool params = dweight || dbias;
  Plan p = plan(std::max<int64_t>(rows, 1), dim, true);
  if (selftest && p.wide) return fail(DOBB_ERR_UNSUPPORTED, "this call waits for no copies");
  float* partial = static_cast<float*>(workspace);
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    NormGradArgs a{grad,   x,      rows, grad_stride, x_stride, (int32_t)dim, weight, param_dtype == DOBB_BF16, mean, rstd, dx, dx_stride,
                   params ? partial : nullptr,
                   reinterpret_cast<float2*>(static_cast<char*>(workspace) + partial_bytes(p, dim)), p.partials, p.shape, {},
                   selftest ? *selftest : Patience{kWaitNs, rows}};
    if (!p.wide) a.ring = ring_of(p, rows, dim, x_stride, x_dtype, grad_stride, grad_dtype, true);
    const bool aligned = dim % 4 == 0 && aligned_rows(x, x_stride, x_dtype, rows) && aligned_rows(grad, grad_stride, grad_dtype, rows) &&
                         (!dx || aligned_rows(dx, dx_stride, x_dtype, rows));
    using bf16 = __nv_bfloat16;
    e = x_dtype == DOBB_F32
            ? (grad_dtype == DOBB_F32 ? launch_backward<float, float>(a, p, aligned, s) : launch_backward<float, bf16>(a, p, aligned, s))
            : (grad_dtype == DOBB_F32 ? launch_backward<bf16, float>(a, p, aligned, s) : launch_backward<bf16, bf16>(a, p, aligned, s));
  } else {
    p.partials = 0;
  }
  if (e == cudaSuccess && params) {
    const JoinArgs j{partial, p.partials, (int32_t)dim, dweight, dbias, dparam_dtype == DOBB_BF16, accumulate};
    e = launch<norm_join>((unsigned)(2 * ((dim + 31) / 32)), kJoinThreads, 0, s, rows > 0, j);
  }
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "layer norm gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

}  // namespace

extern "C" dobb_status dobb_layer_norm_backward(const void* grad, dobb_dtype grad_dtype, int64_t grad_stride, const void* x,
                                                dobb_dtype x_dtype, int64_t rows, int64_t dim, int64_t x_stride,
                                                const void* weight, dobb_dtype param_dtype, const float* mean,
                                                const float* rstd, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                                dobb_dtype dparam_dtype, int accumulate, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  return layer_norm_backward(grad, grad_dtype, grad_stride, x, x_dtype, rows, dim, x_stride, weight, param_dtype, mean, rstd, dx, dx_stride, dweight, dbias,
                             dparam_dtype, accumulate, workspace, workspace_bytes, stream, nullptr);
}

extern "C" dobb_status dobb_selftest_layer_norm_backward_timeout(
    const void* grad, dobb_dtype grad_dtype, int64_t grad_stride, const void* x, dobb_dtype x_dtype, int64_t rows, int64_t dim,
    int64_t x_stride, const void* weight, dobb_dtype param_dtype, const float* mean, const float* rstd, void* dx, int64_t dx_stride,
    void* dweight, void* dbias, dobb_dtype dparam_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream,
    int64_t loaded_rows, uint64_t timeout_ns) {
  const Patience patience{timeout_ns, loaded_rows};
  if (const dobb_status st = check_patience(patience, rows); st != DOBB_OK) return st;
  return layer_norm_backward(grad, grad_dtype, grad_stride, x, x_dtype, rows, dim, x_stride, weight, param_dtype, mean, rstd, dx, dx_stride, dweight, dbias,
                             dparam_dtype, accumulate, workspace, workspace_bytes, stream, &patience);
}
