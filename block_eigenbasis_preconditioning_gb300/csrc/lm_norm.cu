// Layer norm, forward.
#include "lm_norm.cuh"

namespace dobb {
namespace {

struct NormArgs {
  const void* x;
  int64_t rows, x_stride;
  int32_t dim;
  const void *weight, *bias;
  int32_t param_bf16;
  float eps;
  void* out;
  int64_t out_stride;
  float *mean, *rstd;
  Shape shape;
  Ring ring;
  Patience patience;
};

// The forward pass's: a lane for each group.
template <typename TX>
__device__ __forceinline__ void produce_groups(GroupBarriers& b, unsigned char* raw, const Ring& ring, const Shape& shape, const TX* x,
                                               int64_t stride, int64_t rows, int32_t dim, const Patience& patience) {
  const int group = threadIdx.x & 31, unit = 32 / shape.lanes;
  if (group >= shape.groups) return;
  const TX* end = x + (rows - 1) * stride + dim;
  uint32_t k = 0;
  bool ok = true;
  for (int64_t r0 = (int64_t)blockIdx.x * ring.rows + group * unit; r0 < patience.loaded && ok; r0 += (int64_t)gridDim.x * ring.rows, ++k) {
    const uint32_t s = group * ring.slots + k % ring.slots, turn = k / ring.slots;
    if (turn > 0 && !(ok = ring_wait(b, &b.empty[s], (turn - 1) & 1, patience.limit))) break;
    const int32_t count = (int32_t)min((int64_t)unit, rows - r0);
    unsigned char* to = raw + (size_t)s * ring.slot_bytes;
    uint32_t bytes = 0;
    if (ring.pitch[0] == 0)
      bytes = copy_in(to, x + r0 * stride, (int64_t)count * dim, x, end, &b.full[s]);
    else
      for (int i = 0; i < count; ++i)
        bytes += copy_in(to + (size_t)i * ring.pitch[0], x + (r0 + i) * stride, (int64_t)dim, x, end, &b.full[s]);
    ptx::mbar_arrive_expect_tx(&b.full[s], bytes);
  }
  for (uint32_t p = k > (uint32_t)ring.slots ? k - ring.slots : 0; p < k; ++p)
    ptx::mbar_wait(&b.full[group * ring.slots + p % ring.slots], (p / ring.slots) & 1);
}

// Two passes over the registers: a warp's mean, then its squares around it; the
// warps' pairs (n, mean, M2) join exactly.
template <typename TX, typename TO, int P, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1) norm_forward(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(128) unsigned char raw[];
  __shared__ GroupBarriers bar;
  __shared__ float2 red[2][kWarps];
  const Shape sp = a.shape;
  const int warps = sp.warps * sp.groups;
  float* weight = reinterpret_cast<float*>(raw);
  float* bias = weight + (a.dim + 3) / 4 * 4;
  unsigned char* ring = raw + a.ring.first;
  const TX* x = static_cast<const TX*>(a.x);
  const int warp = threadIdx.x >> 5;
  ring_init(bar, sp.groups * a.ring.slots, sp.warps);
  if (warp == warps) {
    produce_groups<TX>(bar, ring, a.ring, sp, x, a.x_stride, a.rows, a.dim, a.patience);
    return;
  }
  copy_params(weight, a.weight, a.param_bf16, a.dim, 1.f, warps * 32);
  copy_params(bias, a.bias, a.param_bf16, a.dim, 0.f, warps * 32);
  const int in_warp = threadIdx.x & 31, lane = in_warp & (sp.lanes - 1);
  const int group = warp / sp.warps, w = warp - group * sp.warps, base = group * sp.warps;
  const Columns<P, ALIGNED> c(w, lane, a.dim, sp.lanes);
  TO* out = static_cast<TO*>(a.out);
  // the last of a row's warps may have fewer columns
  const float inv_dim = 1.f / (float)a.dim, n_last = (float)(a.dim - (sp.warps - 1) * 256 * P), n_full = 256.f * P;
  const float inv_n = w == sp.warps - 1 ? 1.f / n_last : 1.f / n_full;
  asm volatile("bar.sync 15, %0;" ::"r"(warps * 32) : "memory");  // the parameters are there
  int buf = 0;
  const int unit = 32 / sp.lanes, mine = in_warp / sp.lanes;  // rows of the group at a time, this lane's of them
  uint32_t slot = 0, phase = 0;
  bool ok = true;  // once a wait gave up the phases are not known any more: all later rows are lost
  for (int64_t row0 = (int64_t)blockIdx.x * a.ring.rows + group * unit; row0 < a.rows; row0 += (int64_t)gridDim.x * a.ring.rows) {
    const uint32_t s = group * a.ring.slots + slot;
    ok = __all_sync(0xffffffffu, ok && ring_wait(bar, &bar.full[s], phase, a.patience.limit));
    if (++slot == (uint32_t)a.ring.slots) {
      slot = 0;
      phase ^= 1;
    }
    const int64_t row = row0 + mine;
    const bool live = row < a.rows;
    uint64_t v[4 * P];
    const TX* from = ring_row(ring + (size_t)s * a.ring.slot_bytes, a.ring.pitch[0], x + row0 * a.x_stride, a.x_stride, mine, a.dim);
#pragma unroll
    for (int q = 0; q < 2 * P; ++q) {
      v[2 * q] = v[2 * q + 1] = 0;
      if (live && c.has(4 * q)) read_four<TX, P, ALIGNED>(v[2 * q], v[2 * q + 1], from, q, c);
    }
    __syncwarp();
    if (in_warp == 0) ptx::mbar_arrive(&bar.empty[s]);
    float mean, var;
    float h = 1.f;
    bool again = false;
#pragma unroll 1
    while (true) {
      const uint64_t h2 = both(h);
      uint64_t s[2] = {0, 0}, q[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4 * P; ++i) s[i & 1] = lm::fma2(v[i], h2, s[i & 1]);
      const float m = lanes_sum(sum2(lm::add2(s[0], s[1])), sp.lanes) * inv_n;
      const uint64_t minus_m = both(-m);
#pragma unroll
      for (int k = 0; k < 2 * P; ++k) {
        if (!c.has(4 * k)) break;
#pragma unroll
        for (int i = 2 * k; i < 2 * k + 2; ++i) {
          const uint64_t d = lm::fma2(v[i], h2, minus_m);
          if (ALIGNED || c.has(2 * i)) {
            const uint64_t e = only(d, i, c);
            q[i & 1] = lm::fma2(e, e, q[i & 1]);
          }
        }
      }
      const float m2 = lanes_sum(sum2(lm::add2(q[0], q[1])), sp.lanes);
      mean = m;
      var = m2;
      if (sp.warps > 1) {
        // (a warp whose wait gave up: the whole row is lost)
        if (in_warp == 0) red[buf][warp] = ok ? make_float2(m, m2) : make_float2(NAN, NAN);
        __syncwarp();
        group_sync(group, sp.warps * 32);
        mean = 0.f;
        for (int i = 0; i < sp.warps; ++i) mean = fmaf((i == sp.warps - 1 ? n_last : n_full) * inv_dim, red[buf][base + i].x, mean);
        var = 0.f;
        for (int i = 0; i < sp.warps; ++i) {
          const float2 r = red[buf][base + i];
          const float d = r.x - mean;
          var += fmaf((i == sp.warps - 1 ? n_last : n_full) * d, d, r.y);
        }
        buf ^= 1;
      }
      var *= inv_dim;
      // again, rows whose sums left fp32 scaled down (where rows share a warp, the others once more)
      const bool left = !(finite(mean) && finite(var));
      if (again || !__any_sync(0xffffffffu, left)) break;
      if (left) h = kDown;
      again = true;
    }
    float row_mean, row_rstd;
    const RowScale r = row_scale(h, mean, var, a.eps, row_mean, row_rstd);
    if (!live) continue;
    if (w == 0 && lane == 0) {
      a.mean[row] = ok ? row_mean : NAN;
      a.rstd[row] = ok ? row_rstd : NAN;
    }
    const uint64_t minus_m = both(-r.mean), h2 = both(h), rstd = both(ok ? r.rstd : NAN);
#pragma unroll
    for (int q = 0; q < 2 * P; ++q) {
      if (!c.has(4 * q)) break;
      uint64_t w0, w1, b0, b1;
      read_four<float, P, ALIGNED>(w0, w1, weight, q, c);
      read_four<float, P, ALIGNED>(b0, b1, bias, q, c);
      // (rstd times the weight first could leave fp32 where the result does not)
      store_four<TO, P, ALIGNED>(out + row * a.out_stride, lm::fma2(lm::mul2(lm::fma2(v[2 * q], h2, minus_m), rstd), w0, b0),
                                 lm::fma2(lm::mul2(lm::fma2(v[2 * q + 1], h2, minus_m), rstd), w1, b1), q, c);
    }
  }
}

// Rows of more than kMaxForwardDim columns: a block a row, which it reads three times
// (from L2 but for the first).
template <typename TX, typename TO>
__global__ void __launch_bounds__(kThreads) norm_forward_long(const NormArgs a) {
  __shared__ double red[32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride;
    TO* out = static_cast<TO*>(a.out) + row * a.out_stride;
    float h = 1.f, mean, var;
    while (true) {
      mean = (float)(block_sum_of(a.dim, red, [&](int32_t i) { return load_f32(x + i) * h; }) / a.dim);
      var = (float)(block_sum_of(a.dim, red, [&](int32_t i) {
                      const float d = fmaf(load_f32(x + i), h, -mean);
                      return d * d;
                    }) / a.dim);
      if (h != 1.f || (finite(mean) && finite(var))) break;
      h = kDown;
    }
    float row_mean, row_rstd;
    const RowScale r = row_scale(h, mean, var, a.eps, row_mean, row_rstd);
    if (threadIdx.x == 0) {
      a.mean[row] = row_mean;
      a.rstd[row] = row_rstd;
    }
#pragma unroll 8
    for (int32_t i = threadIdx.x; i < a.dim; i += kThreads)
      store_f32(out + i, fmaf(r.xhat(load_f32(x + i)), a.weight ? param(a.weight, a.param_bf16, i) : 1.f,
                              a.bias ? param(a.bias, a.param_bf16, i) : 0.f));
  }
}

template <typename TX, typename TO>
cudaError_t launch_forward(const NormArgs& a, const Plan& p, bool aligned, cudaStream_t s) {
  if (p.wide) return launch<norm_forward_long<TX, TO>>(p.blocks, kThreads, 0, s, false, a);
  const unsigned threads = 32 * (p.shape.warps * p.shape.groups + 1);
  const size_t smem = ring_smem(p, a.ring, false, false);
  const auto go = [&](auto columns) {
    constexpr int P = decltype(columns)::value;
    return aligned ? launch<norm_forward<TX, TO, P, true>>(p.blocks, threads, smem, s, false, a)
                   : launch<norm_forward<TX, TO, P, false>>(p.blocks, threads, smem, s, false, a);
  };
  return p.p == 1   ? go(std::integral_constant<int, 1>{})
         : p.p == 2 ? go(std::integral_constant<int, 2>{})
         : p.p == 4 ? go(std::integral_constant<int, 4>{})
                    : go(std::integral_constant<int, 8>{});
}

// selftest: the waits' limit and the rows that are copied in, or NULL
dobb_status layer_norm(const void* x, dobb_dtype x_dtype, int64_t rows, int64_t dim, int64_t x_stride, const void* weight,
                       const void* bias, dobb_dtype param_dtype, float eps, void* out, dobb_dtype out_dtype, int64_t out_stride,
                       float* mean, float* rstd, void* stream, const Patience* selftest) {
  dobb_status st = check_norm(rows, dim, x_dtype, x_stride, out_dtype, out_stride, param_dtype);
  if (st != DOBB_OK) return st;
  if (!(eps >= 0x1p-126f && eps < INFINITY))
    return fail(DOBB_ERR_INVALID_ARG, "eps must be a positive normal number (got %g)", eps);
  if (rows == 0) return DOBB_OK;
  if (!x || !out || !mean || !rstd) return fail(DOBB_ERR_INVALID_ARG, "x, out, mean and rstd must be non-NULL");
  if (lm::misaligned(x, lm::dtype_bytes(x_dtype)) || lm::misaligned(out, lm::dtype_bytes(out_dtype)) || lm::misaligned(mean, 4) ||
      lm::misaligned(rstd, 4) || lm::misaligned(weight, lm::dtype_bytes(param_dtype)) ||
      lm::misaligned(bias, lm::dtype_bytes(param_dtype)))
    return fail(DOBB_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
  const bool in_place = out == x && out_dtype == x_dtype && (rows <= 1 || out_stride == x_stride);
  lm::Extents ext;
  ext.read("x", x, rows, dim, x_stride, x_dtype, in_place);
  ext.read("weight", weight, 1, dim, dim, param_dtype);
  ext.read("bias", bias, 1, dim, dim, param_dtype);
  ext.write("out", out, rows, dim, out_stride, out_dtype, in_place);
  ext.write("mean", mean, 1, rows, rows, DOBB_F32);
  ext.write("rstd", rstd, 1, rows, rows, DOBB_F32);
  if ((st = ext.check()) != DOBB_OK) return st;
  Plan p = plan(rows, dim, false);
  if (selftest && p.wide) return fail(DOBB_ERR_UNSUPPORTED, "this call waits for no copies");
  const Ring ring = p.wide ? Ring{} : forward_ring(p, rows, dim, x_stride, x_dtype);
  const NormArgs a{x,   rows,       x_stride, (int32_t)dim, weight, bias, param_dtype == DOBB_BF16, eps,
                   out, out_stride, mean,     rstd,         p.shape, ring,   selftest ? *selftest : Patience{kWaitNs, rows}};
  const bool aligned = dim % 4 == 0 && aligned_rows(x, x_stride, x_dtype, rows) && aligned_rows(out, out_stride, out_dtype, rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using bf16 = __nv_bfloat16;
  cudaError_t e = x_dtype == DOBB_F32
                      ? (out_dtype == DOBB_F32 ? launch_forward<float, float>(a, p, aligned, s) : launch_forward<float, bf16>(a, p, aligned, s))
                      : (out_dtype == DOBB_F32 ? launch_forward<bf16, float>(a, p, aligned, s) : launch_forward<bf16, bf16>(a, p, aligned, s));
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "layer norm launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

}  // namespace
}  // namespace dobb

using namespace dobb;

extern "C" dobb_status dobb_layer_norm(const void* x, dobb_dtype x_dtype, int64_t rows, int64_t dim, int64_t x_stride,
                                       const void* weight, const void* bias, dobb_dtype param_dtype, float eps, void* out,
                                       dobb_dtype out_dtype, int64_t out_stride, float* mean, float* rstd, void* stream) {
  return layer_norm(x, x_dtype, rows, dim, x_stride, weight, bias, param_dtype, eps, out, out_dtype, out_stride, mean, rstd, stream, nullptr);
}

extern "C" dobb_status dobb_selftest_layer_norm_timeout(const void* x, dobb_dtype x_dtype, int64_t rows, int64_t dim, int64_t x_stride,
                                                        const void* weight, const void* bias, dobb_dtype param_dtype, float eps,
                                                        void* out, dobb_dtype out_dtype, int64_t out_stride, float* mean, float* rstd,
                                                        void* stream, int64_t loaded_rows, uint64_t timeout_ns) {
  const Patience patience{timeout_ns, loaded_rows};
  if (const dobb_status st = check_patience(patience, rows); st != DOBB_OK) return st;
  return layer_norm(x, x_dtype, rows, dim, x_stride, weight, bias, param_dtype, eps, out, out_dtype, out_stride, mean, rstd, stream,
                    &patience);
}

extern "C" int64_t dobb_selftest_layer_norm_smem(int64_t rows, int64_t dim, dobb_dtype x_dtype, int64_t x_stride, dobb_dtype grad_dtype,
                                                 int64_t grad_stride, int backward, int64_t* most) {
  if (most) *most = lm::kMostSmem;
  if (check_norm(rows, dim, x_dtype, x_stride, grad_dtype, grad_stride, DOBB_F32) != DOBB_OK || rows < 1) return -1;
  Plan p = plan(rows, dim, backward != 0);
  if (p.wide) return 0;
  if (!backward) {
    const Ring r = forward_ring(p, rows, dim, x_stride, x_dtype);
    return (int64_t)ring_smem(p, r, false, false);
  }
  return (int64_t)ring_smem(p, ring_of(p, rows, dim, x_stride, x_dtype, grad_stride, grad_dtype, true), true, true);
}
