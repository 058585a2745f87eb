// Embedding lookup with scaling, and its gradient by sorted tokens.
#include <cooperative_groups.h>

#include "lm_common.cuh"

namespace dobb {
namespace {

namespace cg = cooperative_groups;

// Where every row of both tensors starts on a 16-byte boundary and dim is a
// multiple of eight, rows are worked on in packets of eight values.  Of other
// rows (odd widths, odd strides) the lookup shifts the packets into place
// (9000 rows of 1601 bf16: 14 us; value by value 25 us, bound by the number of
// requests).  The gradient sums them value by value, neighbouring lanes on
// neighbouring values: every row of a run has a shift of its own, which cost
// 183 instructions a packet (32761 rows of 1601: 105 us against 51).
struct Eight {
  uint64_t v[4];  // pairs of fp32
};

template <typename T>
struct Packet {
  static constexpr int kVecs = (int)sizeof(T) / 2;
  uint4 a[kVecs];

  // NC: nothing in the kernel writes the tensor
  template <bool NC>
  __device__ __forceinline__ void load(const T* p) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) a[k] = NC ? __ldg(q + k) : q[k];
  }
  __device__ __forceinline__ Eight get() const {
    Eight r;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      r.v[k] = kVecs == 1 ? lm::Vec16<__nv_bfloat16>::pair(a[0], k) : lm::Vec16<float>::pair(a[k / 2 * (kVecs - 1)], k % 2);
    return r;
  }
  __device__ __forceinline__ void put_to(const Eight& r, T* p) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      lm::unpack2(r.v[k], lo, hi);
      if (kVecs == 1)
        lm::Vec16<__nv_bfloat16>::put(a[0], k, lo, hi);
      else
        lm::Vec16<float>::put(a[k / 2 * (kVecs - 1)], k % 2, lo, hi);
    }
    uint4* q = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) q[k] = a[k];
  }
};

__device__ __forceinline__ uint32_t misalign(const void* p) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
}

bool rows_aligned(const void* a, int64_t a_stride, size_t a_bytes, const void* b, int64_t b_stride,
                  size_t b_bytes, int64_t dim) {
  return dim % 8 == 0 && !lm::misaligned(a, 16) && !lm::misaligned(b, 16) &&
         a_stride * (int64_t)a_bytes % 16 == 0 && b_stride * (int64_t)b_bytes % 16 == 0;
}

// Wait for the kernel before (programmatic dependent launch), and let the next one be launched.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;"); }

// ------------------------------------------------------------------ lookup

constexpr int kThreads = 256;
constexpr int kPackets = 4;  // per thread, in flight together

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
  int32_t chunks;  // groups of lanes per row
  int32_t span;    // 2^span lanes work on a row together
};

// 2^span lanes take kPackets packets each of one token's row: short rows share
// a warp, long ones are split over several.  Bound by HBM: 16384 rows of 4096,
// fp32 to bf16, 42.6 us, 88 % of the copy rate on the distinct rows.
template <typename W, typename O, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) embed_forward(const EmbedArgs a) {
  const int64_t group = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> a.span;
  const int lane = threadIdx.x & ((1 << a.span) - 1);
  const int64_t t = group / a.chunks;
  const int32_t chunk = (int32_t)(group - t * a.chunks);
  if (t >= a.count) return;
  const int64_t v = lm::load_token(a.tokens, a.token_bytes, t);
  const bool live = v >= 0 && v < a.vocab;
  if (v >= a.vocab && a.flags && chunk == 0 && lane == 0) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
  const W* w = static_cast<const W*>(a.weight) + (live ? v : 0) * a.weight_stride;
  O* o = static_cast<O*>(a.out) + t * a.out_stride;
  if (ALIGNED) {
    const int64_t p0 = ((int64_t)chunk * kPackets << a.span) + lane, packets = a.dim / 8;
    Packet<W> in[kPackets];
#pragma unroll
    for (int u = 0; u < kPackets; ++u)
      if (live && p0 + (u << a.span) < packets) in[u].template load<true>(w + 8 * (p0 + (u << a.span)));
    const uint64_t scale = lm::pack2(a.scale, a.scale);
#pragma unroll
    for (int u = 0; u < kPackets; ++u) {
      if (p0 + (u << a.span) >= packets) break;
      Eight r = in[u].get();
#pragma unroll
      for (int k = 0; k < 4; ++k) r.v[k] = live ? lm::mul2(r.v[k], scale) : 0;
      Packet<O> out;
      out.put_to(r, o + 8 * (p0 + (u << a.span)));
    }
  } else {
    // packets on the output's boundaries; the input is shifted into place
    const int64_t head = lm::head_of(o, a.dim), packets = (a.dim - head) / 8, rest = a.dim - packets * 8;
    const int64_t p0 = ((int64_t)chunk * kPackets << a.span) + lane;
    const uint32_t s = misalign(w + head);
    Packet<W> in[kPackets];
#pragma unroll
    for (int u = 0; u < kPackets; ++u) {
      const int64_t p = p0 + (u << a.span);
      if (live && p < packets) {
#pragma unroll
        for (int k = 0; k < Packet<W>::kVecs; ++k) in[u].a[k] = lm::load16(w, head + 8 * p + 4 * k, a.dim, s);
      }
    }
    const uint64_t scale = lm::pack2(a.scale, a.scale);
#pragma unroll
    for (int u = 0; u < kPackets; ++u) {
      const int64_t p = p0 + (u << a.span);
      if (p >= packets) break;
      Eight r = in[u].get();
#pragma unroll
      for (int k = 0; k < 4; ++k) r.v[k] = live ? lm::mul2(r.v[k], scale) : 0;
      Packet<O> out;
      out.put_to(r, o + head + 8 * p);
    }
    if (chunk == 0) {  // fewer than 8 values on either side
      for (int64_t i = lane; i < rest; i += 1 << a.span) {
        const int64_t j = i < head ? i : packets * 8 + i;
        store_f32(o + j, live ? a.scale * load_f32(w + j) : 0.f);
      }
    }
  }
}

// -------------------------------------------------------------------- sort
// Stable least-significant-digit radix sort of (token, position) by one
// cluster of CTAs.  Every warp counts and places a contiguous run of items, so
// that equal tokens keep their order: the place of an item is the number of
// items with smaller digits, plus those with its digit in earlier CTAs,
// earlier warps, and earlier in its warp.  Tokens that take no gradient get
// the key `vocab` and end up last.
//
// A sort of a few thousand tokens is a chain of latencies (12 us for 8192) that
// one cluster works off while the zeros of the gradient are written (24 us for
// 161 MB): the fill kernel is launched before it and lets it start at once, and
// the sort ends only when the fill has.  More SMs help the passes over the
// items (32768 tokens: 4 CTAs of 1024 threads 57 us, 8 29 us, 16 of 512 17 us);
// what is left are the barriers and the exchange of totals.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kBatch = 4;  // items in flight per lane
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kMaxCluster = 16;  // above 8 the kernel has to ask for it
constexpr int kSms = 152;

struct SortArgs {
  const void* tokens;
  int32_t token_bytes;
  int32_t count, vocab;
  int32_t passes, digit_bits;
  uint2* item[2];  // (key, position): pass p reads item[p & 1], writes the other; pass 0 reads the tokens
  uint32_t* flags;
};

struct SortShared {
  uint32_t hist[kSortWarps][kMaxBins];
  uint32_t total[kMaxBins];
  uint32_t base[kMaxBins];
  uint32_t warp_sum[kSortWarps];
};

__device__ __forceinline__ uint32_t token_key(const SortArgs& a, int32_t i) {
  const int64_t v = lm::load_token(a.tokens, a.token_bytes, i);
  if (v >= a.vocab && a.flags) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
  return (v >= 0 && v < a.vocab) ? (uint32_t)v : (uint32_t)a.vocab;
}

__device__ void sort_part(const SortArgs& a, SortShared& sh, cg::cluster_group& cluster) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t warps = (int64_t)parts * kSortWarps;
  const int64_t per = ((a.count + warps - 1) / warps + 31) / 32 * 32;
  const int64_t lo = min((int64_t)a.count, per * (rank * kSortWarps + warp)), hi = min((int64_t)a.count, lo + per);
  const int bins = 1 << a.digit_bits;
  for (int p = 0; p < a.passes; ++p) {
    const uint2* item = a.item[p & 1];
    const int shift = p * a.digit_bits;
    uint32_t* hist = sh.hist[warp];
    for (int b = lane; b < bins; b += 32) hist[b] = 0;
    __syncwarp();
    uint32_t k[kBatch], from[kBatch];
    unsigned same[kBatch];
    // kBatch items of this lane and, for each, the lanes of its warp with the same digit
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int64_t i = i0 + u * 32 + lane;
        k[u] = 0xffffffffu;
        if (i < hi) {
          const uint2 it = p == 0 ? make_uint2(token_key(a, (int32_t)i), (uint32_t)i) : __ldcg(item + i);
          k[u] = it.x;
          from[u] = it.y;
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        same[u] = 0;
        if (i0 + u * 32 >= hi) continue;  // the same for the whole warp
        // one ballot per bit of the digit (match.any instead: 29 us, not 27, for 32768 tokens)
        const uint32_t digit = (k[u] >> shift) & (bins - 1);
        same[u] = __ballot_sync(0xffffffffu, i0 + u * 32 + lane < hi);
#pragma unroll
        for (int bit = 0; bit < kMaxDigitBits; ++bit) {
          const bool one = (digit >> bit) & 1;
          const unsigned who = __ballot_sync(0xffffffffu, one);
          same[u] &= one ? who : ~who;
        }
      }
    };
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i0 + u * 32 >= hi) break;
        if (k[u] != 0xffffffffu && lane == __ffs(same[u]) - 1)
          hist[(k[u] >> shift) & (bins - 1)] += __popc(same[u]);
        __syncwarp();
      }
    }
    __syncthreads();
    // within a digit, the warps in order
    uint32_t mine = 0;
    if (threadIdx.x < bins) {
      uint32_t c[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = sh.hist[w][threadIdx.x];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        sh.hist[w][threadIdx.x] = mine;
        mine += c[w];
      }
      sh.total[threadIdx.x] = mine;
    }
    cluster.sync();
    // the CTAs in order, and the digits in order
    uint32_t below = 0, all = 0;
    if (threadIdx.x < bins) {
      uint32_t c[kMaxCluster];  // the reads in flight together
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        c[r] = r < parts ? *cluster.map_shared_rank(&sh.total[threadIdx.x], r) : 0u;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        all += c[r];
        below += r < rank ? c[r] : 0u;
      }
    }
    uint32_t sum = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    __syncthreads();
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0u);
    if (threadIdx.x < bins) sh.base[threadIdx.x] = before + sum - all + below;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
      if (hi - lo > 32 * kBatch) load(i0);  // else they are still here
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i0 + u * 32 >= hi) break;
        const bool in = k[u] != 0xffffffffu;
        const uint32_t d = (k[u] >> shift) & (bins - 1);
        const uint32_t in_warp = in ? hist[d] + __popc(same[u] & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (in) {
          if (lane == 31 - __clz(same[u])) hist[d] = in_warp + 1;
          a.item[(p + 1) & 1][sh.base[d] + in_warp] = make_uint2(k[u], from[u]);
        }
        __syncwarp();
      }
    }
    cluster.sync();  // every item is in its place before the next pass reads it
  }
}

// One cluster.  The kernel before it in the stream may still be writing zeros.
__global__ void __launch_bounds__(kSortThreads) sort_tokens(const SortArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  cg::cluster_group cluster = cg::this_cluster();
  launch_next();
  sort_part(a, *reinterpret_cast<SortShared*>(raw), cluster);
  wait_for_previous();
}

// Zeros for `rows` rows of the gradient.
struct FillArgs {
  char* out;
  int64_t rows, row_bytes, stride_bytes;
};

__global__ void __launch_bounds__(kThreads) fill_rows(const FillArgs a) {
  launch_next();
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x, threads = (int64_t)gridDim.x * kThreads;
  if (a.stride_bytes == a.row_bytes) {  // one stretch of memory
    const int64_t n = a.rows * a.row_bytes;
    const int64_t head = min(n, (int64_t)((16 - misalign(a.out)) & 15)), nvec = (n - head) / 16;
    uint4* v = reinterpret_cast<uint4*>(a.out + head);
    for (int64_t i = tid; i < nvec; i += threads) v[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = tid; i < n - nvec * 16; i += threads) a.out[i < head ? i : nvec * 16 + i] = 0;
    return;
  }
  // a warp per row
  const int lane = threadIdx.x & 31;
  for (int64_t r = tid >> 5; r < a.rows; r += threads >> 5) {
    char* row = a.out + r * a.stride_bytes;
    const int64_t head = min(a.row_bytes, (int64_t)((16 - misalign(row)) & 15)), nvec = (a.row_bytes - head) / 16;
    uint4* v = reinterpret_cast<uint4*>(row + head);
    for (int64_t i = lane; i < nvec; i += 32) v[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = lane; i < a.row_bytes - nvec * 16; i += 32) row[i < head ? i : nvec * 16 + i] = 0;
  }
}

// ---------------------------------------------------------------- gradient
//
// The sorted tokens are cut into units of equal length, whatever their runs
// of equal tokens look like.  A CTA walks over one unit for a slab of columns,
// a batch of rows in flight, and writes the sum of every run that lies within
// the unit.  A run that continues in another unit leaves a partial sum in the
// workspace: slot 0 of a unit for the run that came from the unit before,
// slot 1 for the one that begins here and goes on.  join_runs adds those up in
// a fixed order.  Bound by latency, with as many rows in flight as registers
// hold: 8192 rows of 1600 bf16 9 us, 32761 of 1601 added to fp32 rows 51 us.
// Rings of shared memory per warp (cp.async or bulk copies) took 16 and 64 us:
// more instructions a row, and the chain of rows a warp has is what it waits for.
constexpr int kSumThreads = 128;
constexpr int kSlab = 8 * kSumThreads;  // columns
constexpr int kMaxUnit = 64;
constexpr uint32_t kNoToken = 0xffffffffu;

struct SumArgs {
  const void* grad;
  int64_t dim, grad_stride;
  int32_t count, vocab;
  const uint2* item;  // (token, position), sorted
  float scale;
  void* out;
  int64_t out_stride;
  float* part;   // [unit][slot][width]
  int64_t width;  // dim rounded up to 8
  int32_t unit;  // tokens per unit
  int32_t slabs;
};

// A token of a unit: its gradient's row, and the row of the sum.
template <typename G, typename O>
struct Item {
  const G* grad;
  O* out;
};

template <typename G, typename O>
struct UnitShared {
  uint32_t key[kMaxUnit + 2];  // 1 ... n; 0 and n + 1: the neighbours'
  Item<G, O> item[kMaxUnit + 1];
};

// The unit's tokens into shared memory; returns their number.
template <typename G, typename O>
__device__ __forceinline__ int32_t load_unit(const SumArgs& a, int32_t u, UnitShared<G, O>& sh) {
  const int64_t lo = (int64_t)u * a.unit;
  const int32_t n = (int32_t)min((int64_t)a.unit, a.count - lo);
  for (int32_t i = threadIdx.x; i < n + 2; i += kSumThreads) {
    const int64_t j = lo - 1 + i;
    const uint2 sorted = j >= 0 && j < a.count ? a.item[j] : make_uint2(kNoToken, 0u);
    sh.key[i] = sorted.x;
    if (i >= 1 && i <= n && sorted.x < (uint32_t)a.vocab)
      sh.item[i] = Item<G, O>{static_cast<const G*>(a.grad) + (int64_t)sorted.y * a.grad_stride,
                              static_cast<O*>(a.out) + (int64_t)sorted.x * a.out_stride};
  }
  __syncthreads();
  return n;
}

// Rows on 16-byte boundaries: a packet of columns per thread.
template <typename G, typename O, bool ADD>
__global__ void __launch_bounds__(kSumThreads) sum_runs(const SumArgs a) {
  constexpr int kRows = ADD || sizeof(G) == 4 ? 4 : 8;  // in flight
  __shared__ UnitShared<G, O> sh;
  launch_next();
  wait_for_previous();
  const int32_t u = blockIdx.x / (unsigned)a.slabs;
  const int64_t col = (int64_t)(blockIdx.x % (unsigned)a.slabs) * kSlab + 8 * threadIdx.x;
  const int32_t n = load_unit(a, u, sh);
  if (col >= a.dim) return;
  const bool came = sh.key[0] == sh.key[1];  // the first run began before this unit
  const uint64_t scale = lm::pack2(a.scale, a.scale);
  Eight sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) sum.v[k] = 0;
  for (int32_t b = 1; b <= n; b += kRows) {
    Packet<G> g[kRows];
    Packet<O> old[ADD ? kRows : 1];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (b + i <= n && sh.key[b + i] < (uint32_t)a.vocab) {
        g[i].template load<true>(sh.item[b + i].grad + col);
        // where the run ends: what its sum is added to
        if (ADD && sh.key[b + i + 1] != sh.key[b + i]) old[i].template load<false>(sh.item[b + i].out + col);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (b + i > n) break;
      const uint32_t v = sh.key[b + i], next = sh.key[b + i + 1];
      if (v >= (uint32_t)a.vocab) return;  // the rest takes no gradient
      const Eight x = g[i].get();
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.v[k] = lm::add2(sum.v[k], x.v[k]);
      const bool on = b + i == n && next == v, from = came && v == sh.key[1];
      if (next == v && !on) continue;
      if (from || on) {
        ulonglong2* q = reinterpret_cast<ulonglong2*>(a.part + ((int64_t)u * 2 + (from ? 0 : 1)) * a.width + col);
        q[0] = make_ulonglong2(sum.v[0], sum.v[1]);
        q[1] = make_ulonglong2(sum.v[2], sum.v[3]);
      } else {
        if (ADD) {
          const Eight was = old[i].get();
#pragma unroll
          for (int k = 0; k < 4; ++k) sum.v[k] = lm::fma2(sum.v[k], scale, was.v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) sum.v[k] = lm::mul2(sum.v[k], scale);
        }
        Packet<O> out;
        out.put_to(sum, sh.item[b + i].out + col);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.v[k] = 0;
    }
  }
}

// Rows anywhere: eight columns per thread, kSumThreads apart.  (Packets shifted
// into place, with a shift per row: 183 instructions a packet, 105 us, not 51.)
template <typename G, typename O, bool ADD>
__global__ void __launch_bounds__(kSumThreads) sum_runs_any(const SumArgs a) {
  constexpr int kRows = 2;  // in flight
  __shared__ UnitShared<G, O> sh;
  launch_next();
  wait_for_previous();
  const int32_t u = blockIdx.x / (unsigned)a.slabs;
  const int64_t col = (int64_t)(blockIdx.x % (unsigned)a.slabs) * kSlab + threadIdx.x;
  const int32_t n = load_unit(a, u, sh);
  if (col >= a.dim) return;
  const int cols = (int)min((int64_t)8, (a.dim - col + kSumThreads - 1) / kSumThreads);
  const bool came = sh.key[0] == sh.key[1];
  float sum[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = 0.f;
  for (int32_t b = 1; b <= n; b += kRows) {
    G g[kRows][8];
    O old[ADD ? kRows : 1][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (b + i <= n && sh.key[b + i] < (uint32_t)a.vocab) {
        const G* row = sh.item[b + i].grad + col;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cols) g[i][k] = __ldg(row + k * kSumThreads);
        if (ADD && sh.key[b + i + 1] != sh.key[b + i]) {
          const O* o = sh.item[b + i].out + col;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < cols) old[i][k] = o[k * kSumThreads];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (b + i > n) break;
      const uint32_t v = sh.key[b + i], next = sh.key[b + i + 1];
      if (v >= (uint32_t)a.vocab) return;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += load_f32(&g[i][k]);
      const bool on = b + i == n && next == v, from = came && v == sh.key[1];
      if (next == v && !on) continue;
      if (from || on) {
        float* q = a.part + ((int64_t)u * 2 + (from ? 0 : 1)) * a.width + col;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cols) q[k * kSumThreads] = sum[k];
      } else {
        O* o = sh.item[b + i].out + col;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < cols)
            store_f32(o + k * kSumThreads, ADD ? fmaf(sum[k], a.scale, load_f32(&old[i][k])) : sum[k] * a.scale);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = 0.f;
    }
  }
}

// Runs over several units: the partial sums of the units, in interleaved
// chains that are joined in order.  A run of up to kShortRun units is joined by
// the CTAs of the unit where it begins, each a slab of columns; of a longer one
// the CTAs of its first kShortRun units take a share of each slab (one token
// repeated, 1600 bf16 columns, the whole call when it adds to what is there: 32768
// tokens 48 us, 131072 tokens 167 us; with the first unit's CTAs alone 96 and 459).
constexpr int kJoinThreads = 256;
constexpr int kJoinPairs = 4;  // short: pairs of columns per thread
constexpr int kJoinRows = 4;   // chains
constexpr int kJoinLanes = kJoinThreads / kJoinRows;
constexpr int kJoinCols = 2 * kJoinLanes * kJoinPairs;
constexpr int kShortRun = 8;
constexpr int kLongLanes = kJoinCols / kShortRun / 4;  // long: four columns per thread
constexpr int kLongRows = kJoinThreads / kLongLanes;
// the CTAs that find no run to join are the most: six to an SM (131072 uniform
// tokens 201 us; 216 us with the three that the registers would allow)
constexpr int kJoinCtas = 6;

template <typename O, bool ADD>
__device__ __forceinline__ void write_joined(const SumArgs& a, uint32_t v, int64_t col, float sum) {
  if (col >= a.dim) return;
  O* o = static_cast<O*>(a.out) + (int64_t)v * a.out_stride + col;
  store_f32(o, ADD ? fmaf(sum, a.scale, load_f32(o)) : sum * a.scale);
}

template <typename O, bool ADD>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) join_runs(const SumArgs a, int32_t slabs) {
  __shared__ union {
    float2 pair[kJoinRows][kJoinPairs][kJoinLanes];
    float4 quad[kLongRows][kLongLanes];
  } red;
  wait_for_previous();
  const int32_t u = blockIdx.x / (unsigned)slabs;
  const int64_t slab = (int64_t)(blockIdx.x % (unsigned)slabs) * kJoinCols;
  // does a run go on from unit u into the next one?
  const int64_t lo = (int64_t)u * a.unit, hi = lo + a.unit;
  if (hi >= a.count) return;
  const uint32_t v = a.item[hi - 1].x;
  if (v >= (uint32_t)a.vocab || a.item[hi].x != v) return;
  // how many units before it began, when this unit lies within it
  int back = 0;
  if (lo > 0 && a.item[lo].x == v && a.item[lo - 1].x == v) {
    const int64_t j = ((int64_t)u - threadIdx.x) * a.unit - 1;
    back = __syncthreads_count(threadIdx.x < kShortRun && j >= 0 && a.item[j].x == v);
    if (back == kShortRun) return;
  }
  // it reaches the units whose first token is v
  const int32_t begin = u - back;
  int32_t last = u;
  for (int32_t at = u + 1;; at += kJoinThreads) {
    const int64_t j = ((int64_t)at + threadIdx.x) * a.unit;
    const int reached = __syncthreads_count(j < a.count && a.item[j].x == v);
    last += reached;
    if (reached < kJoinThreads) break;
  }
  const bool is_short = last - begin < kShortRun;
  if (is_short && back > 0) return;
  // slot 1 of the unit where it begins, slot 0 of the others
  auto part = [&](int32_t i) { return a.part + (2 * (int64_t)i + (i == begin)) * a.width; };
  if (is_short) {
    const int lane = threadIdx.x % kJoinLanes, row = threadIdx.x / kJoinLanes;
    const int64_t col = slab + 2 * lane;
    float2 sum[kJoinPairs];
#pragma unroll
    for (int k = 0; k < kJoinPairs; ++k) sum[k] = make_float2(0.f, 0.f);
    for (int32_t i = begin + row; i <= last; i += kJoinRows) {
#pragma unroll
      for (int k = 0; k < kJoinPairs; ++k) {
        if (col + 2 * kJoinLanes * k < a.dim) {
          const float2 x = *reinterpret_cast<const float2*>(part(i) + col + 2 * kJoinLanes * k);
          sum[k].x += x.x;
          sum[k].y += x.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kJoinPairs; ++k) red.pair[row][k][lane] = sum[k];
    __syncthreads();
    // row r of threads finishes pair r
    static_assert(kJoinPairs == kJoinRows, "a row of threads per pair");
    float2 t = red.pair[0][row][lane];
#pragma unroll
    for (int r = 1; r < kJoinRows; ++r) {
      t.x += red.pair[r][row][lane].x;
      t.y += red.pair[r][row][lane].y;
    }
    write_joined<O, ADD>(a, v, col + 2 * kJoinLanes * row, t.x);
    write_joined<O, ADD>(a, v, col + 2 * kJoinLanes * row + 1, t.y);
  } else {
    const int lane = threadIdx.x % kLongLanes, row = threadIdx.x / kLongLanes;
    const int64_t col = slab + (back * kLongLanes + lane) * 4;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < a.dim) {
#pragma unroll 4
      for (int32_t i = begin + row; i <= last; i += kLongRows) {
        const float4 x = *reinterpret_cast<const float4*>(part(i) + col);
        sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
      }
    }
    red.quad[row][lane] = sum;
    __syncthreads();
    if (row != 0) return;
    for (int r = 1; r < kLongRows; ++r) {
      const float4 x = red.quad[r][lane];
      sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
    }
    write_joined<O, ADD>(a, v, col, sum.x);
    write_joined<O, ADD>(a, v, col + 1, sum.y);
    write_joined<O, ADD>(a, v, col + 2, sum.z);
    write_joined<O, ADD>(a, v, col + 3, sum.w);
  }
}

// Tokens per unit: long units leave fewer partial sums, short ones keep the
// GPU busy when there are few tokens.  At least 3, 6 or 12 CTAs an SM for 8192
// rows of 1600: sums 12.4, 9.6, 10.5 us, joins 6.2, 7.8, 11.2.
int32_t unit_of(int64_t count, int64_t dim) {
  const int64_t slabs = (dim + kSlab - 1) / kSlab;
  int32_t unit = 4;
  while (unit < kMaxUnit && count * slabs / (2 * unit) >= 6 * kSms) unit *= 2;
  return unit;
}
int64_t width_of(int64_t dim) { return (dim + 7) / 8 * 8; }

struct Workspace {
  size_t item[2], part, total;
};

Workspace workspace(int64_t count, int64_t dim) {
  Workspace w{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t n = up((size_t)count * 8);
  const int32_t unit = unit_of(count, dim);
  w.item[1] = n;
  w.part = 2 * n;
  w.total = w.part + up(((size_t)count + unit - 1) / unit * 2 * width_of(dim) * 4) + 256;
  return w;
}

dobb_status check_grad_sizes(int64_t count, int64_t vocab, int64_t dim) {
  if (count < 0 || count > INT32_MAX)
    return fail(DOBB_ERR_INVALID_ARG, "count must lie in [0, 2^31) (got %lld)", (long long)count);
  if (vocab < 1 || vocab > (1 << 30))
    return fail(DOBB_ERR_INVALID_ARG, "vocab must lie in [1, 2^30] (got %lld)", (long long)vocab);
  if (dim < 1) return fail(DOBB_ERR_INVALID_ARG, "dim must be >= 1 (got %lld)", (long long)dim);
  // the joins have the largest grid; with that, all sizes and offsets fit 64 bits
  const int64_t join_slabs = (dim - 1) / kJoinCols + 1;
  const int64_t unit = join_slabs <= INT32_MAX ? unit_of(count, dim) : 1;
  if (join_slabs > INT32_MAX || (count + unit - 1) / unit * join_slabs > INT32_MAX)
    return fail(DOBB_ERR_UNSUPPORTED, "too many tokens times columns for one call");
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
  if (lm::rows_overlap({weight, vocab, dim, weight_stride, weight_dtype}, {out, count, dim, out_stride, out_dtype}))
    return fail(DOBB_ERR_INVALID_ARG, "out overlaps the weight");
  const bool aligned = rows_aligned(weight, weight_stride, lm::dtype_bytes(weight_dtype), out, out_stride,
                                    lm::dtype_bytes(out_dtype), dim);
  // lanes per row: enough for one packet each, at most a warp
  const int64_t packets = (dim - 1) / 8 + 1;
  int32_t span = 0;
  while (span < 5 && (1 << span) < packets) ++span;
  const int64_t per = (int64_t)kPackets << span, chunks = (packets + per - 1) / per;
  if (chunks > INT32_MAX || count > INT64_MAX / 32 / chunks)
    return fail(DOBB_ERR_UNSUPPORTED, "too many tokens times columns for one call");
  const int64_t blocks = ((count * chunks << span) + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return fail(DOBB_ERR_UNSUPPORTED, "too many tokens times columns for one call");
  const EmbedArgs a{weight, vocab, dim, weight_stride, tokens, token_bytes, count, scale, out, out_stride, flags,
                    (int32_t)chunks, span};
  const unsigned grid = (unsigned)blocks;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(a); };
  using B = __nv_bfloat16;
  switch (4 * aligned + 2 * (weight_dtype == DOBB_BF16) + (out_dtype == DOBB_BF16)) {
    case 0: launch(embed_forward<float, float, false>); break;
    case 1: launch(embed_forward<float, B, false>); break;
    case 2: launch(embed_forward<B, float, false>); break;
    case 3: launch(embed_forward<B, B, false>); break;
    case 4: launch(embed_forward<float, float, true>); break;
    case 5: launch(embed_forward<float, B, true>); break;
    case 6: launch(embed_forward<B, float, true>); break;
    case 7: launch(embed_forward<B, B, true>); break;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "embedding launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

extern "C" size_t dobb_embedding_backward_bytes(int64_t count, int64_t vocab, int64_t dim) {
  if (check_grad_sizes(count, vocab, dim) != DOBB_OK) return 0;
  return workspace(count, dim).total;
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
  const Workspace w = workspace(count, dim);
  if (!ws || lm::misaligned(ws, 256))
    return fail(DOBB_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (ws_bytes < w.total)
    return fail(DOBB_ERR_STATE, "workspace of %zu bytes is smaller than the %zu required", ws_bytes,
                w.total);
  if (count > 0 && lm::rows_overlap({grad, count, dim, grad_stride, grad_dtype},
                                    {dweight, vocab, dim, dweight_stride, dweight_dtype}))
    return fail(DOBB_ERR_INVALID_ARG, "dweight overlaps the gradient");
  if (count == 0 && accumulate) return DOBB_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(ws);
  SortArgs sa{};
  sa.tokens = tokens;
  sa.token_bytes = token_bytes;
  sa.count = (int32_t)count;
  sa.vocab = (int32_t)vocab;
  int bits = 1;
  while (vocab >> bits) ++bits;  // the largest key is vocab
  sa.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  sa.digit_bits = (bits + sa.passes - 1) / sa.passes;
  for (int i = 0; i < 2; ++i) sa.item[i] = reinterpret_cast<uint2*>(base + w.item[i]);
  sa.flags = flags;
  cudaError_t e = cudaSuccess;
  if (!accumulate) {
    const int64_t b = (int64_t)lm::dtype_bytes(dweight_dtype);
    // two small blocks per SM write at full rate and leave room for the sort
    fill_rows<<<2 * kSms, kThreads, 0, s>>>(FillArgs{static_cast<char*>(dweight), vocab, dim * b, dweight_stride * b});
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "fill launch: %s", cudaGetErrorString(e));
    if (count == 0) return DOBB_OK;
  }
  // early: may start before the kernel of this call before it has ended
  auto launch = [&](bool early, auto kernel, unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                    auto... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {cluster, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 2 : 1;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, args...);
  };
  // a warp's worth of items per warp of the cluster, or more
  unsigned parts = 1;
  while (parts < kMaxCluster && count > (int64_t)parts * kSortThreads) parts *= 2;
  e = cudaFuncSetAttribute(sort_tokens, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SortShared));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_tokens, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  // beside the fill; without one it follows the caller's work, and waits for that
  launch(!accumulate, sort_tokens, parts, kSortThreads, sizeof(SortShared), parts, sa);
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "token sort launch: %s", cudaGetErrorString(e));
  SumArgs a{};
  a.grad = grad;
  a.dim = dim;
  a.grad_stride = grad_stride;
  a.count = (int32_t)count;
  a.vocab = (int32_t)vocab;
  a.item = sa.item[sa.passes & 1];
  a.scale = scale;
  a.out = dweight;
  a.out_stride = dweight_stride;
  a.part = reinterpret_cast<float*>(base + w.part);
  a.width = width_of(dim);
  a.unit = unit_of(count, dim);
  const int64_t slabs = (dim + kSlab - 1) / kSlab, join_slabs = (dim + kJoinCols - 1) / kJoinCols;
  const int64_t units = (count + a.unit - 1) / a.unit;
  a.slabs = (int32_t)slabs;
  auto sums = [&](auto writes, auto adds) {
    launch(true, accumulate ? adds : writes, (unsigned)(units * slabs), kSumThreads, 0, 1, a);
  };
  auto joins = [&](auto writes, auto adds) {
    launch(true, accumulate ? adds : writes, (unsigned)(units * join_slabs), kJoinThreads, 0, 1, a, (int32_t)join_slabs);
  };
  using F = float;
  using B = __nv_bfloat16;
  const bool aligned = rows_aligned(grad, grad_stride, lm::dtype_bytes(grad_dtype), dweight, dweight_stride,
                                    lm::dtype_bytes(dweight_dtype), dim);
  switch (4 * aligned + 2 * (grad_dtype == DOBB_BF16) + (dweight_dtype == DOBB_BF16)) {
    case 0: sums(sum_runs_any<F, F, false>, sum_runs_any<F, F, true>); break;
    case 1: sums(sum_runs_any<F, B, false>, sum_runs_any<F, B, true>); break;
    case 2: sums(sum_runs_any<B, F, false>, sum_runs_any<B, F, true>); break;
    case 3: sums(sum_runs_any<B, B, false>, sum_runs_any<B, B, true>); break;
    case 4: sums(sum_runs<F, F, false>, sum_runs<F, F, true>); break;
    case 5: sums(sum_runs<F, B, false>, sum_runs<F, B, true>); break;
    case 6: sums(sum_runs<B, F, false>, sum_runs<B, F, true>); break;
    case 7: sums(sum_runs<B, B, false>, sum_runs<B, B, true>); break;
  }
  if (dweight_dtype == DOBB_F32)
    joins(join_runs<F, false>, join_runs<F, true>);
  else
    joins(join_runs<B, false>, join_runs<B, true>);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(DOBB_ERR_CUDA, "embedding gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
