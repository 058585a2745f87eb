// Distillation from a teacher's top logits: the loss of a student's logits, and
// its gradient.
//
// With y = s x over a row of V logits, p = softmax(y), and the row's k teacher
// entries (id_i, t_i), those with id_i >= 0:
//   q_i = e^{s_t t_i} / sum,  loss = sum_i q_i (log q_i - log p[id_i])
//   dx_j = s g (p_j sum q - sum_{i: id_i = j} q_i)
// The dense part s g p_j is the gradient of log sum e^y; the teacher's part
// touches k entries, which are corrected after it.
// Measured, 8192 x 50257 bf16 with 64 entries a row: loss and gradient 286 us (85 % of
// the copy rate for one read and one write), the gradient alone 264 us (92 %).
#include <cooperative_groups.h>

#include <algorithm>

#include "lm_logits.cuh"
#include "tc_ptx.cuh"

namespace dobb {
namespace {

namespace cg = cooperative_groups;

struct DistillArgs {
  const void* logits;
  int64_t rows, row_stride;
  int32_t vocab;
  const void *ids, *teacher;
  int32_t id_bytes, teacher_bf16, k;
  float scale, teacher_scale;
  float *loss, *row_max, *log_sum;
  const float* g;
  void* out;
  int64_t out_stride;
  int32_t blocks, chunks;  // of the gradient alone: blocks per row, chunks per block
  uint32_t* flags;
};

// The teacher's row in shared memory.
struct Teacher {
  int32_t id[DOBB_MAX_TEACHER];  // -1: none
  float q[DOBB_MAX_TEACHER], log_q[DOBB_MAX_TEACHER];
  float sum[DOBB_MAX_TEACHER];  // of q over an id, at its first entry; -1 at the others
  int32_t state;
};
// no entries; q is a distribution; NaN or +inf among the entries; an id >= vocab
constexpr int kNone = 0, kGood = 1, kNan = 2, kBad = 3;
constexpr int kPerLane = DOBB_MAX_TEACHER / 32;

// Ids of the rounds before, three bits each (a Bloom filter of multiplicative hashes: fields of
// the product with 2^64 / golden ratio).  256 entries without a repeated id are taken for some with
// one in one row of a hundred.
constexpr int kSeenBits = 12;
struct Seen {
  uint32_t word[3][(1 << kSeenBits) / 32];
  static __device__ __forceinline__ uint32_t bit(int32_t id, int h) {
    return (uint32_t)((uint64_t)id * 0x9e3779b97f4a7c15ull >> (64 - (h + 1) * kSeenBits)) & ((1u << kSeenBits) - 1);
  }
  __device__ __forceinline__ bool has(int32_t id) const {
    bool all = true;
#pragma unroll
    for (int h = 0; h < 3; ++h) all &= word[h][bit(id, h) >> 5] >> (bit(id, h) & 31) & 1;
    return all;
  }
  __device__ __forceinline__ void add(int32_t id) {
#pragma unroll
    for (int h = 0; h < 3; ++h) atomicOr(&word[h][bit(id, h) >> 5], 1u << (bit(id, h) & 31));
  }
};

// One warp reads the teacher's row: q and log q of every entry, and with SUMS the sum
// of q over every id at its first entry.
template <bool SUMS>
__device__ __forceinline__ void load_teacher(Teacher& t, Seen* seen, const DistillArgs& a, int64_t row) {
  const int lane = threadIdx.x & 31;
  float v[kPerLane], m = -INFINITY;
  int64_t ids[kPerLane];
  // all loads first
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int i = u * 32 + lane;
    ids[u] = -1;
    v[u] = -INFINITY;
    if (i < a.k) {
      ids[u] = lm::load_token(a.ids, a.id_bytes, row * a.k + i);
      v[u] = a.teacher_bf16 ? load_f32(static_cast<const __nv_bfloat16*>(a.teacher) + row * a.k + i)
                            : static_cast<const float*>(a.teacher)[row * a.k + i];
    }
  }
  if (SUMS && a.k > 32) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Seen) / 16); i += 32) reinterpret_cast<uint4*>(seen)[i + lane] = make_uint4(0, 0, 0, 0);
    static_assert(sizeof(Seen) % 512 == 0, "cleared by a warp");
    __syncwarp();
  }
  bool any = false, bad = false, nan = false, twice = false;
  int32_t own[kPerLane];
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int i = u * 32 + lane;
    if (u * 32 >= a.k) break;
    if (ids[u] < 0) v[u] = -INFINITY;
    bad |= ids[u] >= a.vocab;
    any |= v[u] != -INFINITY;
    nan |= !(v[u] < INFINITY);
    own[u] = ids[u] < 0 || ids[u] >= a.vocab ? -1 : (int32_t)ids[u];
    if (i < a.k) t.id[i] = own[u];
    m = fmaxf(m, v[u]);
    if (SUMS) {
      // the ids of one round against each other, then against those of the rounds before, which
      // are all marked by then: no order of the lanes matters
      const uint32_t equal = __match_any_sync(0xffffffffu, own[u]);
      if (own[u] >= 0) twice |= (equal & (equal - 1)) != 0 || (u > 0 && seen->has(own[u]));
      if ((u + 1) * 32 < a.k) {
        __syncwarp();
        if (own[u] >= 0) seen->add(own[u]);
        __syncwarp();
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  any = __any_sync(0xffffffffu, any);
  bad = __any_sync(0xffffffffu, bad);
  nan = __any_sync(0xffffffffu, nan);
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    if (u * 32 >= a.k) break;
    const float d = v[u] == -INFINITY ? -INFINITY : scaled_difference(v[u], m, a.teacher_scale);
    v[u] = d;
    s += expf(d);
  }
  s = nan ? NAN : warp_sum(s);
  const float log_s = logf(s), inv = 1.f / s;
  float q[kPerLane];
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int i = u * 32 + lane;
    q[u] = 0.f;
    if (u * 32 >= a.k) break;
    q[u] = any && i < a.k ? expf(v[u]) * inv : 0.f;
    if (i < a.k) {
      t.q[i] = q[u];
      t.log_q[i] = v[u] - log_s;
    }
  }
  if (SUMS) {
    if (!__any_sync(0xffffffffu, twice)) {
#pragma unroll
      for (int u = 0; u < kPerLane; ++u)
        if (u * 32 + lane < a.k) t.sum[u * 32 + lane] = own[u] < 0 ? -1.f : q[u];
    } else {
      __syncwarp();
#pragma unroll 1
      for (int i = lane; i < a.k; i += 32) {
        const int32_t id = t.id[i];
        float sum = 0.f;
        bool first = id >= 0;
#pragma unroll 4
        for (int o = 0; o < a.k; ++o) {
          const bool same = t.id[o] == id;
          sum += same ? t.q[o] : 0.f;
          first = first && !(same && o < i);
        }
        t.sum[i] = first ? sum : -1.f;
      }
    }
  }
  if (lane == 0) t.state = bad ? kBad : nan ? kNan : any ? kGood : kNone;
  __syncwarp();
}

// log p of a logit, given its row's statistics
__device__ __forceinline__ float log_p(float x, float m, float log_sum, float scale) {
  if (m == -INFINITY && log_sum == -INFINITY) return -INFINITY;
  return scaled_difference(x, m, scale) - log_sum;
}

// The share in the loss of a logit at the end of fp32, whose log p lies beyond.  (A call, as inline it costs the
// loss and gradient of 8192 x 50257 bf16 half a percent more.)
__device__ __noinline__ float far_share(float q, float log_q, float x, float m, float log_sum, float scale) {
  return (float)((double)q * ((double)log_q - ((double)scale * ((double)x - (double)m) - (double)log_sum)));
}

// The loss of a row by one warp; the teacher's entries are in t, x_at(i) is
// the student's logit of entry i.
template <typename F>
__device__ __forceinline__ void write_loss(const DistillArgs& a, const Teacher& t, int64_t row, float m, float log_sum, F x_at) {
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  for (int i = lane; i < a.k; i += 32) {
    const float q = t.q[i];
    if (t.id[i] < 0 || q == 0.f) continue;
    const float x = x_at(i), lp = log_p(x, m, log_sum, a.scale);
    if (lp == -INFINITY && x != -INFINITY)
      s += far_share(q, t.log_q[i], x, m, log_sum, a.scale);
    else
      s = fmaf(q, t.log_q[i] - lp, s);
  }
  s = warp_sum(s);
  if (lane == 0) {
    if (t.state == kBad) {
      s = NAN;
      if (a.flags) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
    }
    a.loss[row] = t.state == kNone ? 0.f : s;
  }
}

// A warp a row, after the statistics.
constexpr int kLossWarps = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kLossWarps) distill_loss(const DistillArgs a) {
  __shared__ Teacher teachers[kLossWarps];
  const int64_t row = (int64_t)blockIdx.x * kLossWarps + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  Teacher& t = teachers[threadIdx.x >> 5];
  load_teacher<false>(t, nullptr, a, row);
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  write_loss(a, t, row, a.row_max[row], a.log_sum[row], [&](int i) { return load_f32(x + t.id[i]); });
}

// What an entry of a row becomes: p times the dense factor.
struct Dense {
  float half, minus_hm, c, minus_log2_sum, factor;
  bool zero;  // the row has no gradient
  // x - m may be beyond fp32, and its product with a small scale not: half of both
  __device__ __forceinline__ Dense(float m, float log_sum, float scale, float g, int state) {
    half = fabsf(m) >= 0x1p100f && scale < 0.5f ? 0.5f : 1.f;
    minus_hm = -half * m;
    c = scale * kLog2e / half;
    minus_log2_sum = -log_sum * kLog2e;
    factor = state == kNan ? NAN : scale * g;
    zero = state == kNone || state == kBad || (m == -INFINITY && log_sum == -INFINITY);
  }
  __device__ __forceinline__ float operator()(float x) const {
    return lm::exp2_fast(fmaf(fmaf(x, half, minus_hm), c, minus_log2_sum)) * factor;
  }
};

// The gradient alone.  A block takes a row, or where rows are few a stretch of one, in
// chunks of kGradVecs vectors per thread, aligned to the output; the logits are
// shifted into place when the two differ in alignment.  The teacher's row is read
// once, while the first chunk is on its way (a block for every chunk: 8192 x 50257
// bf16 with 64 entries 512 us, waiting for the teacher).  The rows go from the last to the
// first: the statistics right before leave the last ones in L2.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;

template <typename T>
__global__ void __launch_bounds__(kGradThreads) distill_backward(const DistillArgs a) {
  using V = lm::Vec16<T>;
  __shared__ Teacher t;
  __shared__ __align__(16) Seen seen;
  constexpr int kChunk = kGradThreads * kGradVecs;
  const int64_t row = a.rows - 1 - blockIdx.x / (unsigned)a.blocks;
  const int32_t chunk0 = blockIdx.x % (unsigned)a.blocks * a.chunks;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  T* d = static_cast<T*>(a.out) + row * a.out_stride;
  const int32_t head = (int32_t)lm::head_of(d, a.vocab), nvec = (a.vocab - head) / V::N, tail0 = head + nvec * V::N;
  const int32_t end = (int32_t)min((int64_t)nvec, (int64_t)(chunk0 + a.chunks) * kChunk);  // of this block's vectors
  const uint32_t s = (uint32_t)(reinterpret_cast<uintptr_t>(x + head) & 15);
  const int32_t tid = threadIdx.x;
  int32_t v0 = chunk0 * kChunk + tid;
  uint4 v[kGradVecs];
  const auto load = [&] {
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int32_t j = v0 + u * kGradThreads;
      if (j < end) v[u] = lm::load16(x, (int64_t)head + (int64_t)j * V::N, a.vocab, s);
    }
  };
  load();
  if (tid < 32) load_teacher<true>(t, &seen, a, row);
  __syncthreads();
  const Dense dense(a.row_max[row], a.log_sum[row], a.scale, a.g[row], t.state);
  // the teacher's entries in this stretch: their logits are read before they may be written over
  int32_t at = -1;
  float own = 0.f, q = -1.f;
  if (tid < a.k && t.id[tid] >= 0) {
    at = t.id[tid];
    const int32_t of = at < head || at >= tail0 ? 0 : (at - head) / V::N / kChunk;
    if (of >= chunk0 && of < chunk0 + a.chunks) {
      own = load_f32(x + at);
      q = t.sum[tid];
    } else {
      at = -1;
    }
  }
  const int32_t j1 = chunk0 != 0 ? -1 : tid < head ? tid : (tid >= 32 && tid - 32 < a.vocab - tail0) ? tail0 + tid - 32 : -1;
  const float single = j1 >= 0 ? load_f32(x + j1) : 0.f;
  __syncthreads();
#pragma unroll 1
  for (; v0 - tid < end; v0 += kChunk) {
    uint4 o[kGradVecs];
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      o[u] = make_uint4(0, 0, 0, 0);
      if (!dense.zero) {
#pragma unroll
        for (int i = 0; i < V::N / 2; ++i) V::put(o[u], i, dense(V::get(v[u], 2 * i)), dense(V::get(v[u], 2 * i + 1)));
      }
    }
    const int32_t was = v0;
    v0 += kChunk;
    load();
    v0 = was;
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int32_t j = v0 + u * kGradThreads;
      if (j < end) __stcs(reinterpret_cast<uint4*>(d + head) + j, o[u]);
    }
  }
  if (j1 >= 0) store_f32(d + j1, dense.zero ? 0.f : dense(single));
  if (dense.zero) return;
  __syncthreads();
  if (at >= 0 && !(q < 0.f)) store_f32(d + at, dense(own) - dense.factor * q);
}

static_assert(DOBB_MAX_TEACHER <= kGradThreads, "a thread takes one of the teacher's entries");

// ------------------------------------------------- loss and gradient in one
//
// A cluster of blocks takes a row, a stretch of it each, in shared memory, so that
// the logits cross HBM once.  The blocks are persistent and their warps have roles:
//   compute   (16) sum a row's stages while they arrive, then read them again for the
//             gradient, stage after stage;
//   producer  (1) copies the next row's stages in as they become free;
//   teacher   (1) reads the next row's teacher, and the logits of its entries, ahead;
//             when a row's dense part is written, its loss, and the entries of
//             the gradient that the teacher touches.
// Two blocks an SM: one copies or waits while the other computes.
// Shared by the blocks of a cluster are only the maxima and sums of a row, sent with
// an arrival at the receiver's barrier.
constexpr int kComputeWarps = 16;
constexpr int kComputeThreads = 32 * kComputeWarps;
constexpr int kRowThreads = kComputeThreads + 64;
constexpr int kUnroll = 4;
constexpr int kStageVecs = kUnroll * kComputeThreads;
constexpr int kMaxStages = 8;
constexpr int kMaxParts = 8;
constexpr int kSms = 152;
constexpr uint64_t kWaitNs = 2000000000ull;

// How long a wait lasts at most, and (self-test) the block of a cluster that copies in no row
// from `loaded` on.
struct Patience {
  uint64_t limit = kWaitNs;
  int64_t loaded = 0;
  int32_t late_part = -1;
};

struct RowTeacher {
  Teacher t;
  float x[DOBB_MAX_TEACHER];  // the logits of its entries
};
struct RowShared {
  uint64_t full[kMaxStages], empty[kMaxStages], ready, written, parts_in[2];
  __align__(16) Seen seen;
  RowTeacher teacher[2];
  float2 part[2][kMaxParts];  // maximum and sum of every block's stretch; a maximum of NaN: it gave up
  float2 stat[2];             // row_max and log_sum, NaN where a block gave up
  float red[2][kComputeWarps];
  int32_t late;               // a wait gave up: all others do
};

__device__ __forceinline__ bool row_wait(RowShared& sh, uint64_t* bar, uint32_t parity, uint64_t limit) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*(volatile int32_t*)&sh.late) return false;
    if (ptx::global_timer_ns() - t0 > limit) {
      *(volatile int32_t*)&sh.late = 1;
      return false;
    }
  }
  return true;
}

// the same address in the shared memory of another block of the cluster
__device__ __forceinline__ uint32_t peer_address(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void send_part(const float2* to, uint64_t* bar, int rank, float m, float s) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer_address(to, rank)), "f"(m), "f"(s) : "memory");
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_address(bar, rank)) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(ptx::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory"); }

template <typename T>
struct Stretch {  // of one row
  using V = lm::Vec16<T>;
  const T* x;
  T* d;
  int32_t head, nvec, tail0;
  int32_t stages;  // the same for every row, whatever its alignment: the last may be without a vector
  __device__ __forceinline__ Stretch(const DistillArgs& a, int64_t row, int32_t lo, int32_t n) {
    x = static_cast<const T*>(a.logits) + row * a.row_stride + lo;
    d = static_cast<T*>(a.out) + row * a.out_stride + lo;
    head = (int32_t)lm::head_of(x, n);
    nvec = (n - head) / V::N;
    tail0 = head + nvec * V::N;
    // (with fewer in a row that starts later, its entries behind the vectors would lie in a
    // stage for which the next row's copy waits for none of this row's readers)
    stages = (n / V::N + kStageVecs - 1) / kStageVecs;
  }
};

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 2) distill_rows(const DistillArgs a, int32_t per, const Patience patience) {
  using V = lm::Vec16<T>;
  extern __shared__ __align__(128) unsigned char raw[];
  RowShared& sh = *reinterpret_cast<RowShared*>(raw);
  // the vectors of a stretch from byte 16 of the image on, the entries before them ahead
  uint4* xv = reinterpret_cast<uint4*>(raw + (sizeof(RowShared) + 127) / 128 * 128 + 16);
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = blockIdx.x / (unsigned)parts, step = gridDim.x / (unsigned)parts;
  const int32_t lo = min(a.vocab, rank * per), n = min(a.vocab, lo + per) - lo;
  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      ptx::mbar_init(&sh.full[s], 1);
      ptx::mbar_init(&sh.empty[s], kComputeWarps);
    }
    ptx::mbar_init(&sh.ready, 1);
    ptx::mbar_init(&sh.written, kComputeWarps);
    ptx::mbar_init(&sh.parts_in[0], parts);
    ptx::mbar_init(&sh.parts_in[1], parts);
    sh.late = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (parts > 1) cluster.sync();
  const float c = a.scale * kLog2e;
  const uint64_t limit = patience.limit;

  if (warp == kComputeWarps) {
    // ---- producer
    if (lane == 0) {
    uint32_t issued[kMaxStages];  // copies so far, by stage
#pragma unroll
    for (int s = 0; s < kMaxStages; ++s) issued[s] = 0;
    bool ok = true;
    for (int64_t row = first; row < a.rows && ok; row += step) {
      if (rank == patience.late_part && row >= patience.loaded) break;
      const Stretch<T> r(a, row, lo, n);
#pragma unroll
      for (int s = 0; s < kMaxStages; ++s) {
        if (s >= r.stages || !ok) break;
        if (issued[s] > 0 && !(ok = row_wait(sh, &sh.empty[s], (issued[s] - 1) & 1, limit))) break;
        const uint32_t bytes = (uint32_t)max(min(r.nvec - s * kStageVecs, kStageVecs), 0) * 16;
        if (bytes > 0) {
          ptx::mbar_arrive_expect_tx(&sh.full[s], bytes);
          ptx::bulk_load(xv + s * kStageVecs, r.x + r.head + (int64_t)s * kStageVecs * V::N, bytes, &sh.full[s]);
        } else {
          ptx::mbar_arrive(&sh.full[s]);
        }
        ++issued[s];
      }
    }
    // no copy is in flight when the block ends
#pragma unroll
    for (int s = 0; s < kMaxStages; ++s)
      if (issued[s] > 0) ptx::mbar_wait(&sh.full[s], (issued[s] - 1) & 1);
    }
    __syncwarp();
  } else if (warp == kComputeWarps + 1) {
    // ---- teacher
    const auto fetch = [&](int64_t row, RowTeacher& q) {
      load_teacher<true>(q.t, &sh.seen, a, row);
      const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
      for (int i = lane; i < a.k; i += 32) q.x[i] = q.t.id[i] >= 0 ? load_f32(x + q.t.id[i]) : 0.f;
    };
    // ready(row): its teacher is there, and that of the row before last, with its
    // statistics, not needed any more
    const auto ready = [&] {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.ready);
    };
    if (first < a.rows) fetch(first, sh.teacher[0]);
    ready();
    uint32_t it = 0;
    for (int64_t row = first; row < a.rows; row += step, ++it) {
      RowTeacher& q = sh.teacher[it & 1];
      if (row + step < a.rows) fetch(row + step, sh.teacher[(it + 1) & 1]);
      const bool ok = row_wait(sh, &sh.written, it & 1, limit);
      __syncwarp();
      const float2 st = sh.stat[it & 1];
      // a wait of this block gave up, or one of another block of the cluster
      const bool lost = !ok || *(volatile int32_t*)&sh.late || !(st.x == st.x);
      if (lost && lane == 0 && a.flags) atomicOr(a.flags, DOBB_FLAG_TIMEOUT);
      if (rank == 0) {
        if (!lost) write_loss(a, q.t, row, st.x, st.y, [&](int i) { return q.x[i]; });
        if (lane == 0) {
          if (lost) a.loss[row] = NAN;
          a.row_max[row] = lost ? NAN : st.x;
          a.log_sum[row] = lost ? NAN : st.y;
        }
      }
      const Dense dense(st.x, st.y, a.scale, a.g[row], q.t.state);
      T* d = static_cast<T*>(a.out) + row * a.out_stride;
      if (!dense.zero && !lost)
        for (int i = lane; i < a.k; i += 32) {
          const int32_t id = q.t.id[i];
          if (id >= lo && id < lo + n && !(q.t.sum[i] < 0.f)) store_f32(d + id, dense(q.x[i]) - dense.factor * q.t.sum[i]);
        }
      ready();
    }
  } else {
  // ---- compute
  const uint64_t c2 = lm::pack2(c, c);
  uint32_t it = 0, turns[kMaxStages];  // rows, and uses of every stage, so far
#pragma unroll
  for (int s = 0; s < kMaxStages; ++s) turns[s] = 0;
  for (int64_t row = first; row < a.rows; row += step, ++it) {
    const Stretch<T> r(a, row, lo, n);
    T* xs = reinterpret_cast<T*>(xv) - r.head;
    // the entries before and behind the vectors: fewer than 8 each
    const int32_t outside = tid < r.head ? tid : (tid >= 16 && tid - 16 < n - r.tail0) ? r.tail0 + tid - 16 : -1;
    T kept{};
    if (outside >= 0) kept = r.x[outside];
    float own = -INFINITY, ref = -kWide;
    bool nan = false, ok = true;
    uint64_t s2 = 0, e2 = 0;
#pragma unroll
    for (int st = 0; st < kMaxStages; ++st) {
      if (st >= r.stages) break;
      ok = ok && row_wait(sh, &sh.full[st], turns[st] & 1, limit);
      ++turns[st];
      const int32_t v0 = st * kStageVecs + tid;
      if (r.nvec - st * kStageVecs >= kStageVecs) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = xv[v0 + u * kComputeThreads];
        add_vectors<T, false>(v, c, c2, own, ref, s2, e2, nan);
      } else {
#pragma unroll 1
        for (int32_t j = v0; j < r.nvec; j += kComputeThreads) {
          const uint4 v[1] = {xv[j]};
          add_vectors<T, false>(v, c, c2, own, ref, s2, e2, nan);
        }
      }
    }
    const float single = outside >= 0 ? load_f32(&kept) : -INFINITY;
    if (single == single)
      own = fmaxf(own, single);
    else
      nan = true;
    // the teacher's row is there, and so its last use of what is written next is over
    ok = row_wait(sh, &sh.ready, it & 1, limit) && ok;
    float m = own;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sh.red[0][warp] = m;
    compute_sync();  // (and the last row's entries outside its vectors are not read any more)
    if (outside >= 0) {
      xs[outside] = kept;
      ptx::fence_proxy_async_smem();  // a later row's copy may come here
    }
    m = sh.red[0][0];
#pragma unroll
    for (int w = 1; w < kComputeWarps; ++w) m = fmaxf(m, sh.red[0][w]);
    float s = 0.f;
    if (is_wide(m, c)) {
      compute_sync();
      for (int32_t i = tid; i < n; i += kComputeThreads) s += lm::exp2_fast(lm::max_nan((load_f32(xs + i) - m) * c, -200.f));
    } else {
      float hi, none = 0.f;
      lm::unpack2(s2, s, hi);
      s += hi;
      const float to = reference(m, c);
      move_by(s, none, ref - to);
      if (single == single) s += lm::exp2_fast(lm::max_nan(fmaf(single, c, -to), -200.f));
      move_to_max(s, none, to, m, c);
    }
    s = warp_sum(nan ? NAN : s);
    if (lane == 0) sh.red[1][warp] = s;
    compute_sync();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kComputeWarps; ++w) s += sh.red[1][w];
    if (parts > 1) {
      const int buf = it & 1;
      if (tid < parts) send_part(&sh.part[buf][rank], &sh.parts_in[buf], tid, *(volatile int32_t*)&sh.late ? NAN : m, s);
      const uint64_t t0 = ptx::global_timer_ns();
      while (!try_wait_cluster(&sh.parts_in[buf], (it >> 1) & 1)) {
        if (ptx::global_timer_ns() - t0 > limit) {
          *(volatile int32_t*)&sh.late = 1;
          ok = false;
          break;
        }
      }
      for (int p = 0; p < parts; ++p) {
        m = fmaxf(m, sh.part[buf][p].x);
        ok = ok && sh.part[buf][p].x == sh.part[buf][p].x;
      }
      s = 0.f;
      for (int p = 0; p < parts; ++p) {
        const float2 q = sh.part[buf][p];
        float qs = q.y, none = 0.f;
        if (q.x != m) move_by(qs, none, scaled_difference(q.x, m, c));
        s += qs;
      }
    }
    float log_sum = kLn2 * log2f(s);
    if (!ok || *(volatile int32_t*)&sh.late) m = log_sum = NAN;
    if (tid == 0) sh.stat[it & 1] = make_float2(m, log_sum);

    // ---- the gradient, in vectors on the output's boundaries
    // (in a row that is given up the teacher may be another row's)
    const Dense dense(m, log_sum, a.scale, a.g[row], m == m ? sh.teacher[it & 1].t.state : kNan);
    const int32_t dhead = (int32_t)lm::head_of(r.d, n), dvec = (n - dhead) / V::N, dtail0 = dhead + dvec * V::N;
    const uint32_t shift = (uint32_t)((dhead - r.head) * (int32_t)sizeof(T)) & 15;
    uint4* dv = reinterpret_cast<uint4*>(r.d + dhead);
    const int32_t j1 = tid < dhead ? tid : (tid >= 16 && tid - 16 < n - dtail0) ? dtail0 + tid - 16 : -1;
    if (j1 >= 0) store_f32(r.d + j1, dense.zero ? 0.f : dense(load_f32(xs + j1)));
    const auto out = [&](const uint4& v, int32_t j) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (!dense.zero) {
#pragma unroll
        for (int i = 0; i < V::N / 2; ++i) V::put(o, i, dense(V::get(v, 2 * i)), dense(V::get(v, 2 * i + 1)));
      }
      __stcs(dv + j, o);
    };
#pragma unroll 1
    for (int st = 0; st < r.stages; ++st) {
      const int32_t v0 = st * kStageVecs + tid;
      if (shift == 0) {
        const uint4* src = reinterpret_cast<const uint4*>(xs + dhead);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (v0 + u * kComputeThreads < dvec) out(src[v0 + u * kComputeThreads], v0 + u * kComputeThreads);
      } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int32_t j = v0 + u * kComputeThreads;
          if (j < dvec) out(lm::load_shifted16(xs + dhead + j * V::N, shift), j);
        }
      }
      // the output's vectors are at most one off those of the image, so a stage is
      // free when the next one has been read
      __syncwarp();
      if (lane == 0) {
        if (st > 0) ptx::mbar_arrive(&sh.empty[st - 1]);
        if (st == r.stages - 1) ptx::mbar_arrive(&sh.empty[st]);
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sh.written);
  }
  }
  // a block's shared memory stays until no other one sends to it
  if (parts > 1) cluster.sync();
}

}  // namespace
}  // namespace dobb

using namespace dobb;

namespace {

dobb_status check_distill(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride, const void* ids,
                          int id_bytes, const void* teacher, int teacher_dtype, int k, float scale, float teacher_scale,
                          bool grad, const float* g, const void* out, int64_t out_stride) {
  if (lm::bad_dtype(dtype) || lm::bad_dtype(teacher_dtype))
    return fail(DOBB_ERR_INVALID_ARG, "the dtype of logits and teacher must be DOBB_F32 or DOBB_BF16");
  if (rows < 0) return fail(DOBB_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
  if (rows > INT32_MAX) return fail(DOBB_ERR_UNSUPPORTED, "too many rows (%lld)", (long long)rows);
  if (vocab < 1 || vocab > INT32_MAX)
    return fail(DOBB_ERR_INVALID_ARG, "vocab must lie in [1, 2^31) (got %lld)", (long long)vocab);
  if (rows > 1 && row_stride < vocab)
    return fail(DOBB_ERR_INVALID_ARG, "row_stride %lld is below vocab %lld", (long long)row_stride, (long long)vocab);
  if (id_bytes != 4 && id_bytes != 8) return fail(DOBB_ERR_INVALID_ARG, "id_bytes must be 4 or 8 (got %d)", id_bytes);
  if (k < 1 || k > DOBB_MAX_TEACHER)
    return fail(DOBB_ERR_INVALID_ARG, "k must lie in [1, %d] (got %d)", DOBB_MAX_TEACHER, k);
  if (!(scale > 0.f) || scale > 0x1p127f || !(teacher_scale > 0.f) || teacher_scale > 0x1p127f)
    return fail(DOBB_ERR_INVALID_ARG, "scale and teacher_scale must lie in (0, 2^127] (got %g, %g)", scale, teacher_scale);
  if (grad && rows > 1 && out_stride < vocab)
    return fail(DOBB_ERR_INVALID_ARG, "out_stride %lld is below vocab %lld", (long long)out_stride, (long long)vocab);
  if (rows > 1 && (row_stride > INT64_MAX / 8 / rows || (grad && out_stride > INT64_MAX / 8 / rows)))
    return fail(DOBB_ERR_UNSUPPORTED, "rows times the row stride is too large");
  if (rows == 0) return DOBB_OK;
  if (!logits || !ids || !teacher) return fail(DOBB_ERR_INVALID_ARG, "logits, ids and teacher must be non-NULL");
  if (grad && (!g || !out)) return fail(DOBB_ERR_INVALID_ARG, "the gradient needs grad_loss and dlogits");
  if (lm::misaligned(logits, lm::dtype_bytes(dtype)) || lm::misaligned(ids, id_bytes) ||
      lm::misaligned(teacher, lm::dtype_bytes(teacher_dtype)) || (grad && lm::misaligned(out, lm::dtype_bytes(dtype))) ||
      (grad && lm::misaligned(g, 4)))
    return fail(DOBB_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
  return DOBB_OK;
}

void read_all(lm::Extents& ext, const DistillArgs& a, int dtype, bool in_place) {
  ext.read("logits", a.logits, a.rows, a.vocab, a.row_stride, dtype, in_place);
  ext.read("ids", a.ids, 1, a.rows * a.k * (a.id_bytes / 4), a.rows * a.k * (a.id_bytes / 4), DOBB_F32);
  ext.read("teacher", a.teacher, 1, a.rows * a.k, a.rows * a.k, a.teacher_bf16 ? DOBB_BF16 : DOBB_F32);
  ext.read("grad_loss", a.g, 1, a.rows, a.rows, DOBB_F32);
  ext.write("dlogits", a.out, a.rows, a.vocab, a.out_stride, dtype, in_place);
}

template <typename T>
cudaError_t launch_backward(DistillArgs a, cudaStream_t s) {
  const int64_t per = (int64_t)kGradThreads * kGradVecs * (16 / (int64_t)sizeof(T));
  const int64_t chunks = (a.vocab + per - 1) / per;
  // one block a row where that fills the GPU, else as many as do
  a.blocks = (int32_t)std::min<int64_t>(chunks, std::max<int64_t>(1, 8 * kSms / a.rows));
  a.chunks = (int32_t)((chunks + a.blocks - 1) / a.blocks);
  const int64_t most = ((int64_t)1 << 30) / a.blocks;
  for (int64_t end = a.rows; end > 0; end -= most) {  // the last rows first
    DistillArgs b = a;
    const int64_t r0 = end > most ? end - most : 0;
    b.rows = end - r0;
    b.logits = static_cast<const T*>(a.logits) + r0 * a.row_stride;
    b.out = static_cast<T*>(a.out) + r0 * a.out_stride;
    b.ids = static_cast<const char*>(a.ids) + r0 * a.k * a.id_bytes;
    b.teacher = static_cast<const char*>(a.teacher) + r0 * a.k * (a.teacher_bf16 ? 2 : 4);
    b.row_max = a.row_max + r0;
    b.log_sum = a.log_sum + r0;
    b.g = a.g + r0;
    distill_backward<T><<<(unsigned)(b.rows * a.blocks), kGradThreads, 0, s>>>(b);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Rows in the cluster's shared memory: blocks per row, 0 where a row does not fit.
constexpr size_t kRowImage = 100 * 1024;  // of the 113 KB that two blocks an SM have each
int row_parts(int64_t rows, int64_t vocab, size_t bytes) {
  const int64_t fit = (int64_t)(kRowImage / bytes) - 16;
  int64_t parts = (vocab + fit - 1) / fit;
  if (parts > kMaxParts) return 0;
  while (parts < kMaxParts && rows * (parts + 1) <= 2 * kSms && vocab / (parts + 1) >= 8192) ++parts;
  return (int)parts;
}

template <typename T>
cudaError_t launch_rows(const DistillArgs& a, int parts, const Patience& patience, cudaStream_t s) {
  // stretches of whole 16-byte vectors
  const int32_t per = (int32_t)(((a.vocab + parts - 1) / parts + 7) / 8 * 8);
  const size_t smem = (sizeof(RowShared) + 127) / 128 * 128 + 16 + (size_t)per * sizeof(T) + 32;
  cudaError_t e = lm::allow_smem<distill_rows<T>>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)parts, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // clusters that run at once: fewer than the SMs hold blocks, a cluster stays in one part of the GPU
  int clusters = 2 * kSms / parts;
  if (parts > 1 && a.rows > clusters / 2) {
    cfg.gridDim = dim3((unsigned)(clusters * parts));
    e = cudaOccupancyMaxActiveClusters(&clusters, distill_rows<T>, &cfg);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(a.rows, std::max(clusters, 1)) * parts));
  return cudaLaunchKernelEx(&cfg, distill_rows<T>, a, per, patience);
}

// selftest: with the waits' limit and the withheld rows of `patience`, and no other way than the clusters'
dobb_status distill(const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab,
                                    int64_t row_stride, const void* ids, int id_bytes, const void* teacher,
                                    dobb_dtype teacher_dtype, int k, float scale, float teacher_scale, float* loss,
                                    float* row_max, float* log_sum, const float* grad_loss, void* dlogits,
                                    int64_t out_stride, uint32_t* flags, void* stream, Patience patience, bool selftest) {
  dobb_status st = check_distill(logits, logits_dtype, rows, vocab, row_stride, ids, id_bytes, teacher, teacher_dtype, k, scale,
                                 teacher_scale, grad_loss || dlogits, grad_loss, dlogits, out_stride);
  if (st != DOBB_OK || rows == 0) return st;
  if (!loss || !row_max || !log_sum) return fail(DOBB_ERR_INVALID_ARG, "loss, row_max and log_sum must be non-NULL");
  if (lm::misaligned(loss, 4) || lm::misaligned(row_max, 4) || lm::misaligned(log_sum, 4) || lm::misaligned(flags, 4))
    return fail(DOBB_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
  DistillArgs a{logits, rows,    row_stride, (int32_t)vocab, ids,       teacher, id_bytes,   teacher_dtype == DOBB_BF16, k,    scale,
                teacher_scale, loss,       row_max,        log_sum, grad_loss, dlogits, out_stride, 0,    0, flags};
  const bool in_place = dlogits == logits && (rows == 1 || out_stride == row_stride);
  lm::Extents ext;
  read_all(ext, a, logits_dtype, in_place);
  ext.write("loss", loss, 1, rows, rows, DOBB_F32);
  ext.write("row_max", row_max, 1, rows, rows, DOBB_F32);
  ext.write("log_sum", log_sum, 1, rows, rows, DOBB_F32);
  if ((st = ext.check()) != DOBB_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = logits_dtype == DOBB_F32;
  const int parts = dlogits ? row_parts(rows, vocab, lm::dtype_bytes(logits_dtype)) : 0;
  if (selftest && (parts == 0 || patience.late_part < 0 || patience.late_part >= parts))
    return parts ? fail(DOBB_ERR_INVALID_ARG, "late_part must lie in [0, %d) (got %d)", parts, patience.late_part)
                 : fail(DOBB_ERR_UNSUPPORTED, "this call waits for no copies");
  if (parts) {
    const cudaError_t e = f32 ? launch_rows<float>(a, parts, patience, s) : launch_rows<__nv_bfloat16>(a, parts, patience, s);
    if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "distillation launch: %s", cudaGetErrorString(e));
    return DOBB_OK;
  }
  if ((st = log_prob_statistics(logits, logits_dtype, rows, vocab, row_stride, scale, loss, row_max, log_sum, flags, stream)) != DOBB_OK)
    return st;
  const int64_t blocks = (rows + kLossWarps - 1) / kLossWarps;
  if (f32)
    distill_loss<float><<<(unsigned)blocks, 32 * kLossWarps, 0, s>>>(a);
  else
    distill_loss<__nv_bfloat16><<<(unsigned)blocks, 32 * kLossWarps, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && dlogits) e = f32 ? launch_backward<float>(a, s) : launch_backward<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "distillation launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

}  // namespace

extern "C" dobb_status dobb_distill(const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab,
                                    int64_t row_stride, const void* ids, int id_bytes, const void* teacher,
                                    dobb_dtype teacher_dtype, int k, float scale, float teacher_scale, float* loss,
                                    float* row_max, float* log_sum, const float* grad_loss, void* dlogits,
                                    int64_t out_stride, uint32_t* flags, void* stream) {
  return distill(logits, logits_dtype, rows, vocab, row_stride, ids, id_bytes, teacher, teacher_dtype, k, scale, teacher_scale, loss,
                 row_max, log_sum, grad_loss, dlogits, out_stride, flags, stream, Patience{}, false);
}

extern "C" dobb_status dobb_selftest_distill_timeout(const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab,
                                                     int64_t row_stride, const void* ids, int id_bytes, const void* teacher,
                                                     dobb_dtype teacher_dtype, int k, float scale, float teacher_scale, float* loss,
                                                     float* row_max, float* log_sum, const float* grad_loss, void* dlogits,
                                                     int64_t out_stride, uint32_t* flags, void* stream, int64_t loaded_rows,
                                                     int late_part, uint64_t timeout_ns) {
  if (loaded_rows < 0 || loaded_rows > rows || timeout_ns == 0 || timeout_ns > 5000000000ull)
    return fail(DOBB_ERR_INVALID_ARG, "loaded_rows must lie in [0, rows], timeout_ns in [1, 5e9]");
  return distill(logits, logits_dtype, rows, vocab, row_stride, ids, id_bytes, teacher, teacher_dtype, k, scale, teacher_scale, loss,
                 row_max, log_sum, grad_loss, dlogits, out_stride, flags, stream, Patience{timeout_ns, loaded_rows, late_part}, true);
}

extern "C" dobb_status dobb_distill_backward(const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab,
                                             int64_t row_stride, const void* ids, int id_bytes, const void* teacher,
                                             dobb_dtype teacher_dtype, int k, float scale, float teacher_scale,
                                             const float* row_max, const float* log_sum, const float* grad_loss,
                                             void* dlogits, int64_t out_stride, void* stream) {
  dobb_status st = check_distill(logits, logits_dtype, rows, vocab, row_stride, ids, id_bytes, teacher, teacher_dtype, k, scale,
                                 teacher_scale, true, grad_loss, dlogits, out_stride);
  if (st != DOBB_OK || rows == 0) return st;
  if (!row_max || !log_sum) return fail(DOBB_ERR_INVALID_ARG, "row_max and log_sum must be non-NULL");
  if (lm::misaligned(row_max, 4) || lm::misaligned(log_sum, 4))
    return fail(DOBB_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
  const DistillArgs a{logits, rows, row_stride, (int32_t)vocab, ids, teacher, id_bytes, teacher_dtype == DOBB_BF16, k, scale,
                      teacher_scale, nullptr, const_cast<float*>(row_max), const_cast<float*>(log_sum), grad_loss, dlogits, out_stride,
                      0, 0, nullptr};
  const bool in_place = dlogits == logits && (rows == 1 || out_stride == row_stride);
  lm::Extents ext;
  read_all(ext, a, logits_dtype, in_place);
  ext.read("row_max", row_max, 1, rows, rows, DOBB_F32);
  ext.read("log_sum", log_sum, 1, rows, rows, DOBB_F32);
  if ((st = ext.check()) != DOBB_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == DOBB_F32 ? launch_backward<float>(a, s) : launch_backward<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "distillation gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
