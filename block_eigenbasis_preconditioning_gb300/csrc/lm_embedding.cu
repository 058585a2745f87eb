// Embedding lookup with scaling, and its gradient by sorted tokens.
#include <cooperative_groups.h>

#include "lm_common.cuh"

namespace dobb {
namespace {

namespace cg = cooperative_groups;

// A row is worked on in packets of eight values that start on 16-byte
// boundaries of the output.  Where every row of both tensors starts on one and
// dim is a multiple of eight (ALIGNED), that is all.  Otherwise the first and
// the last packet may be cut off by the row (edges: value by value, out of
// line), and the input's packets lie anywhere: aligned loads around them are
// shifted into place.
struct Eight {
  uint64_t v[4];  // pairs of fp32
};

__device__ __forceinline__ uint32_t misalign(const void* p) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
}

__device__ __forceinline__ Eight eight_of(const uint4& a, const uint4&, __nv_bfloat16) {
  Eight r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.v[k] = lm::Vec16<__nv_bfloat16>::pair(a, k);
  return r;
}
__device__ __forceinline__ Eight eight_of(const uint4& a, const uint4& b, float) {
  Eight r;
  r.v[0] = lm::Vec16<float>::pair(a, 0);
  r.v[1] = lm::Vec16<float>::pair(a, 1);
  r.v[2] = lm::Vec16<float>::pair(b, 0);
  r.v[3] = lm::Vec16<float>::pair(b, 1);
  return r;
}

// Values i ... i + 7 of a row of n, those outside it 0 and not read.
template <typename T>
__device__ __noinline__ Eight load_edge(const T* row, int64_t i, int64_t n) {
  Eight r;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const int64_t j = i + 2 * k;
    r.v[k] = lm::pack2(j >= 0 && j < n ? load_f32(row + j) : 0.f,
                       j + 1 >= 0 && j + 1 < n ? load_f32(row + j + 1) : 0.f);
  }
  return r;
}
template <typename T>
__device__ __noinline__ void store_edge(T* row, int64_t i, int64_t n, Eight r) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const int64_t j = i + 2 * k;
    float lo, hi;
    lm::unpack2(r.v[k], lo, hi);
    if (j >= 0 && j < n) store_f32(row + j, lo);
    if (j + 1 >= 0 && j + 1 < n) store_f32(row + j + 1, hi);
  }
}

// The memory of a tensor: aligned 16 bytes may be read where they lie inside.
struct Span {
  const char *lo, *hi;
};
template <typename T>
Span span_of(const T* base, int64_t rows, int64_t stride, int64_t dim, size_t bytes) {
  const char* p = reinterpret_cast<const char*>(base);
  return Span{p, p + (size_t)((rows - 1) * stride + dim) * bytes};
}

// Raw bytes of a packet in flight: what aligned loads around it brought, and
// its misalignment s.
template <typename T, bool ALIGNED>
struct Raw {
  static constexpr int kVecs = (int)sizeof(T) / 2;
  uint4 a[kVecs + (ALIGNED ? 0 : 1)];

  // the packet at q (first 16-byte boundary at or before it); what lies outside
  // the row is read too, but not outside the tensor
  __device__ __forceinline__ void load(const char* q, uint32_t s) {
    const uint4* v = reinterpret_cast<const uint4*>(q);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) a[k] = __ldg(v + k);
    if (!ALIGNED && s) a[kVecs] = __ldg(v + kVecs);
  }
  static __device__ __forceinline__ bool inside(const char* q, uint32_t s, const Span& m) {
    return ALIGNED || (q >= m.lo && q + 16 * (kVecs + (s ? 1 : 0)) <= m.hi);
  }
  __device__ __forceinline__ Eight get(uint32_t s) const {
    if (ALIGNED) return eight_of(a[0], a[kVecs - 1], T{});
    constexpr int N = 4 * (kVecs + 1);
    uint32_t w[N];
#pragma unroll
    for (int k = 0; k <= kVecs; ++k) {
      w[4 * k] = a[k].x;
      w[4 * k + 1] = a[k].y;
      w[4 * k + 2] = a[k].z;
      w[4 * k + 3] = a[k].w;
    }
    if (s & 8) {
#pragma unroll
      for (int i = 0; i + 2 < N; ++i) w[i] = w[i + 2];
    }
    if (s & 4) {
#pragma unroll
      for (int i = 0; i + 1 < N; ++i) w[i] = w[i + 1];
    }
    if (sizeof(T) == 2 && (s & 2)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return eight_of(make_uint4(w[0], w[1], w[2], w[3]),
                    make_uint4(w[4 * (kVecs - 1)], w[4 * (kVecs - 1) + 1], w[4 * (kVecs - 1) + 2], w[4 * (kVecs - 1) + 3]),
                    T{});
  }
};

// The same of a row that the kernel writes, i on a 16-byte boundary.
template <bool ALIGNED, typename T>
__device__ __forceinline__ Eight load8_own(const T* row, int64_t i, int64_t n) {
  if (!ALIGNED && (i < 0 || i + 8 > n)) return load_edge(row, i, n);
  const uint4* q = reinterpret_cast<const uint4*>(row + i);
  return eight_of(q[0], sizeof(T) == 4 ? q[1] : q[0], T{});
}

template <bool ALIGNED, typename T>
__device__ __forceinline__ void store8(T* row, int64_t i, int64_t n, const Eight& r) {
  if (!ALIGNED && (i < 0 || i + 8 > n)) return store_edge(row, i, n, r);
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) lm::unpack2(r.v[k], f[2 * k], f[2 * k + 1]);
  uint4* q = reinterpret_cast<uint4*>(row + i);
  if (sizeof(T) == 2) {
    uint4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k) lm::Vec16<__nv_bfloat16>::put(o, k, f[2 * k], f[2 * k + 1]);
    *q = o;
  } else {
    q[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    q[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
}

// First value of packet 0 of an output row, <= 0.
template <bool ALIGNED, typename T>
__device__ __forceinline__ int32_t first_packet(const T* row) {
  if (ALIGNED) return 0;
  const int32_t h = (int32_t)((16 - misalign(row)) & 15) / (int32_t)sizeof(T);
  return h ? h - 8 : 0;
}
// Packets of a row, whatever its alignment.
int64_t packets_of(int64_t dim, bool aligned) { return aligned ? dim / 8 : (dim + 14) / 8; }

bool rows_aligned(const void* a, int64_t a_stride, size_t a_bytes, const void* b, int64_t b_stride,
                  size_t b_bytes, int64_t dim) {
  return dim % 8 == 0 && !lm::misaligned(a, 16) && !lm::misaligned(b, 16) &&
         a_stride * (int64_t)a_bytes % 16 == 0 && b_stride * (int64_t)b_bytes % 16 == 0;
}

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
  int32_t packets;  // per row
  int32_t chunks;   // groups per row
  int32_t span;     // 2^span lanes work on a row together
  Span memory;      // of the weight
};

// 2^span lanes take kPackets packets each of one token's row: short rows share
// a warp, long ones are split over several.
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
  const int32_t p0 = ((chunk * kPackets) << a.span) + lane, i0 = first_packet<ALIGNED>(o);
  // packet p of the input begins at q + 8 p sizeof(W), s bytes after a boundary
  const uint32_t s = ALIGNED ? 0u : misalign(w + i0);
  const char* q = reinterpret_cast<const char*>(w + i0) - s;
  Raw<W, ALIGNED> raw[kPackets];
#pragma unroll
  for (int u = 0; u < kPackets; ++u) {
    const int32_t p = p0 + (u << a.span);
    const char* at = q + (int64_t)p * (8 * (int)sizeof(W));
    if (live && p < a.packets && raw[u].inside(at, s, a.memory)) raw[u].load(at, s);
  }
  const uint64_t scale = lm::pack2(a.scale, a.scale);
#pragma unroll
  for (int u = 0; u < kPackets; ++u) {
    const int32_t p = p0 + (u << a.span);
    if (p >= a.packets) break;
    Eight r = raw[u].get(s);
    if (!raw[u].inside(q + (int64_t)p * (8 * (int)sizeof(W)), s, a.memory)) r = load_edge(w, (int64_t)i0 + 8 * p, a.dim);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.v[k] = live ? lm::mul2(r.v[k], scale) : 0;
    store8<ALIGNED>(o, (int64_t)i0 + 8 * p, a.dim, r);
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
// A sort of a few thousand tokens is a chain of latencies that a few SMs can
// work off; the other CTAs of the launch write the zeros of the gradient
// meanwhile.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kBatch = 4;  // items in flight per lane
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kMaxCluster = 8;
constexpr int kSms = 152;

struct SortArgs {
  const void* tokens;
  int32_t token_bytes;
  int32_t count, vocab;
  int32_t passes, digit_bits;
  uint32_t* key[2];  // pass p reads buffer p & 1, writes the other; pass 0 reads the tokens
  uint32_t* pos[2];
  uint32_t* flags;
  // rows to fill with zeros: `fill` of `dim` values
  void* out;
  int64_t fill, dim, out_stride;
  int32_t out_bytes;
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
    const uint32_t* key = a.key[p & 1];
    const uint32_t* pos = a.pos[p & 1];
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
          k[u] = p == 0 ? token_key(a, (int32_t)i) : __ldcg(key + i);
          from[u] = p == 0 ? (uint32_t)i : __ldcg(pos + i);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const unsigned live = __ballot_sync(0xffffffffu, i0 + u * 32 + lane < hi);
        same[u] = live & __match_any_sync(0xffffffffu, k[u] == 0xffffffffu ? ~0u : (k[u] >> shift) & (bins - 1));
      }
    };
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (k[u] != 0xffffffffu && lane == __ffs(same[u]) - 1)
          hist[(k[u] >> shift) & (bins - 1)] += __popc(same[u]);
        __syncwarp();
      }
    }
    __syncthreads();
    // within a digit, the warps in order
    uint32_t mine = 0;
    if (threadIdx.x < bins) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sh.hist[w][threadIdx.x];
        sh.hist[w][threadIdx.x] = mine;
        mine += c;
      }
      sh.total[threadIdx.x] = mine;
    }
    cluster.sync();
    // the CTAs in order, and the digits in order
    uint32_t below = 0, all = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r < parts) {
          const uint32_t c = r == rank ? mine : cluster.map_shared_rank(sh.total, r)[threadIdx.x];
          all += c;
          if (r < rank) below += c;
        }
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
    if (threadIdx.x < bins) {
      uint32_t before = 0;
      for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
      sh.base[threadIdx.x] = before + sum - all + below;
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kBatch) {
      if (hi - lo > 32 * kBatch) load(i0);  // else they are still here
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const bool in = k[u] != 0xffffffffu;
        const uint32_t d = (k[u] >> shift) & (bins - 1);
        const uint32_t in_warp = in ? hist[d] + __popc(same[u] & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (in) {
          if (lane == 31 - __clz(same[u])) hist[d] = in_warp + 1;
          const uint32_t at = sh.base[d] + in_warp;
          a.key[(p + 1) & 1][at] = k[u];
          a.pos[(p + 1) & 1][at] = from[u];
        }
        __syncwarp();
      }
    }
    cluster.sync();  // every item is in its place before the next pass reads it
  }
}

// Zeros for rows [row0, row0 + rows) by `ctas` CTAs, of which this is number `cta`.
__device__ void fill_rows(const SortArgs& a, int cta, int ctas) {
  const int64_t row_bytes = a.dim * a.out_bytes, stride = a.out_stride * a.out_bytes;
  char* out = static_cast<char*>(a.out);
  const int64_t tid = (int64_t)cta * kSortThreads + threadIdx.x, threads = (int64_t)ctas * kSortThreads;
  if (stride == row_bytes) {  // one stretch of memory
    const int64_t n = a.fill * row_bytes;
    const int64_t head = min(n, (int64_t)((16 - misalign(out)) & 15)), nvec = (n - head) / 16;
    uint4* v = reinterpret_cast<uint4*>(out + head);
    for (int64_t i = tid; i < nvec; i += threads) v[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = tid; i < n - nvec * 16; i += threads) out[i < head ? i : nvec * 16 + i] = 0;
    return;
  }
  // a warp per row
  const int lane = threadIdx.x & 31;
  for (int64_t r = tid >> 5; r < a.fill; r += threads >> 5) {
    char* row = out + r * stride;
    const int64_t head = min(row_bytes, (int64_t)((16 - misalign(row)) & 15)), nvec = (row_bytes - head) / 16;
    uint4* v = reinterpret_cast<uint4*>(row + head);
    for (int64_t i = lane; i < nvec; i += 32) v[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = lane; i < row_bytes - nvec * 16; i += 32) row[i < head ? i : nvec * 16 + i] = 0;
  }
}

// The first cluster sorts, the other CTAs fill.
__global__ void __launch_bounds__(kSortThreads) sort_and_fill(const SortArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks();
  if ((int)blockIdx.x < parts)
    sort_part(a, *reinterpret_cast<SortShared*>(raw), cluster);
  else
    fill_rows(a, blockIdx.x - parts, gridDim.x - parts);
}

__global__ void __launch_bounds__(kSortThreads) fill_only(const SortArgs a) {
  fill_rows(a, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- gradient
//
// The sorted tokens are cut into units of equal length, whatever their runs
// of equal tokens look like.  A CTA walks over one unit for a slab of columns,
// a batch of rows in flight, and writes the sum of every run that lies within
// the unit.  A run that continues in another unit leaves a partial sum in the
// workspace: slot 0 of a unit for the run that came from the unit before,
// slot 1 for the one that begins here and goes on.  join_runs adds those up in
// a fixed order.
constexpr int kSumThreads = 128;
constexpr int kMaxUnit = 64;

struct SumArgs {
  const void* grad;
  int64_t dim, grad_stride;
  int32_t count, vocab;
  const uint32_t *key, *pos;  // sorted
  float scale;
  void* out;
  int64_t out_stride;
  int32_t accumulate;
  float* part;      // [unit][slot][packets * 8]
  int32_t packets;  // per row
  int32_t unit;     // tokens per unit
  int32_t slabs;    // of kSumThreads packets
  Span memory;      // of grad
};

template <bool ALIGNED, typename O>
__device__ __forceinline__ void write_sum(const SumArgs& a, O* o, int64_t i, Eight r) {
  const uint64_t scale = lm::pack2(a.scale, a.scale);
  if (a.accumulate) {
    const Eight old = load8_own<ALIGNED>(o, i, a.dim);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.v[k] = lm::fma2(r.v[k], scale, old.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.v[k] = lm::mul2(r.v[k], scale);
  }
  store8<ALIGNED>(o, i, a.dim, r);
}

// A token of a unit: where the packets of its gradient's row and of its
// output's row begin.
struct Item {
  const char* grad;  // 16-byte boundary at or before packet 0
  char* out;         // packet 0
  uint32_t s;        // packet 0 of the gradient lies at grad + s
  int32_t first;     // first value of packet 0, <= 0
};

template <typename G, typename O, bool ALIGNED, bool ADD>
__global__ void __launch_bounds__(kSumThreads) sum_runs(const SumArgs a) {
  constexpr int kRows = !ALIGNED || ADD || sizeof(G) == 4 ? 4 : 8;  // in flight
  constexpr int kGradStep = 8 * (int)sizeof(G), kOutStep = 8 * (int)sizeof(O);
  __shared__ uint32_t key[kMaxUnit + 2];
  __shared__ Item item[kMaxUnit + 1];
  const int32_t u = blockIdx.x / (unsigned)a.slabs;
  const int32_t packet = (blockIdx.x % (unsigned)a.slabs) * kSumThreads + threadIdx.x;
  const int64_t lo = (int64_t)u * a.unit;
  const int32_t n = (int32_t)min((int64_t)a.unit, a.count - lo);
  // items 1 ... n; key[0] and key[n + 1] are the neighbours' (none: a key that no token has)
  for (int32_t i = threadIdx.x; i < n + 2; i += kSumThreads) {
    const int64_t j = lo - 1 + i;
    const uint32_t v = j >= 0 && j < a.count ? a.key[j] : 0xffffffffu;
    key[i] = v;
    if (i >= 1 && i <= n && v < (uint32_t)a.vocab) {
      O* o = static_cast<O*>(a.out) + (int64_t)v * a.out_stride;
      const int32_t first = first_packet<ALIGNED>(o);
      const char* g = reinterpret_cast<const char*>(static_cast<const G*>(a.grad) + (int64_t)a.pos[j] * a.grad_stride + first);
      const uint32_t s = ALIGNED ? 0u : misalign(g);
      item[i] = Item{g - s, reinterpret_cast<char*>(o + first), s, first};
    }
  }
  __syncthreads();
  if (packet >= a.packets) return;
  const bool came = key[0] == key[1];  // the first run began before this unit
  const uint64_t scale = lm::pack2(a.scale, a.scale);
  Eight sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) sum.v[k] = 0;
  for (int32_t b = 1; b <= n; b += kRows) {
    Raw<G, ALIGNED> raw[kRows];
    Raw<O, true> old[ADD ? kRows : 1];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (b + i <= n && key[b + i] < (uint32_t)a.vocab) {
        const Item& it = item[b + i];
        const char* q = it.grad + (int64_t)packet * kGradStep;
        if (raw[i].inside(q, it.s, a.memory)) raw[i].load(q, it.s);
        if (ADD && key[b + i + 1] != key[b + i]) {  // the run ends here: what its sum is added to
          const int64_t c = it.first + 8 * (int64_t)packet;
          const uint4* o = reinterpret_cast<const uint4*>(it.out + (int64_t)packet * kOutStep);
          if (ALIGNED || (c >= 0 && c + 8 <= a.dim)) {
#pragma unroll
            for (int k = 0; k < Raw<O, true>::kVecs; ++k) old[i].a[k] = o[k];
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (b + i > n) break;
      const uint32_t v = key[b + i], next = key[b + i + 1];
      if (v >= (uint32_t)a.vocab) return;  // the rest takes no gradient
      const Item& it = item[b + i];
      Eight g = raw[i].get(it.s);
      if (!raw[i].inside(it.grad + (int64_t)packet * kGradStep, it.s, a.memory))
        g = load_edge(reinterpret_cast<const G*>(it.grad + it.s) - it.first, it.first + 8 * (int64_t)packet, a.dim);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.v[k] = lm::add2(sum.v[k], g.v[k]);
      const bool on = b + i == n && next == v;
      if (next == v && !on) continue;
      const bool from = came && v == key[1];
      if (from || on) {
        ulonglong2* q = reinterpret_cast<ulonglong2*>(
            a.part + (((int64_t)u * 2 + (from ? 0 : 1)) * a.packets + packet) * 8);
        q[0] = make_ulonglong2(sum.v[0], sum.v[1]);
        q[1] = make_ulonglong2(sum.v[2], sum.v[3]);
      } else {
        O* o = reinterpret_cast<O*>(it.out) - it.first;
        const int64_t c = it.first + 8 * (int64_t)packet;
        if (ADD) {
          Eight was = old[i].get(0u);
          if (!ALIGNED && (c < 0 || c + 8 > a.dim)) was = load_edge(o, c, a.dim);
#pragma unroll
          for (int k = 0; k < 4; ++k) sum.v[k] = lm::fma2(sum.v[k], scale, was.v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) sum.v[k] = lm::mul2(sum.v[k], scale);
        }
        store8<ALIGNED>(o, c, a.dim, sum);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.v[k] = 0;
    }
  }
}

// Runs over several units: the partial sums of the units, in eight interleaved
// chains that are joined in order.
constexpr int kJoinPackets = 32;  // of a CTA
constexpr int kJoinRows = 8;
constexpr int kJoinThreads = kJoinPackets * kJoinRows;

template <typename O, bool ALIGNED>
__global__ void __launch_bounds__(kJoinThreads) join_runs(const SumArgs a, int32_t units, int32_t slabs) {
  __shared__ ulonglong2 red[kJoinRows][kJoinPackets][2];
  const int32_t u = blockIdx.x / (unsigned)slabs;
  const int lane = threadIdx.x % kJoinPackets, row = threadIdx.x / kJoinPackets;
  const int32_t packet = (blockIdx.x % (unsigned)slabs) * kJoinPackets + lane;
  // does a run begin in unit u and go on in the next one?
  const int64_t lo = (int64_t)u * a.unit, hi = lo + a.unit;
  if (hi >= a.count) return;
  const uint32_t v = a.key[hi - 1], next = a.key[hi], first = a.key[lo], before = lo > 0 ? a.key[lo - 1] : 0xffffffffu;
  if (v >= (uint32_t)a.vocab || next != v || (first == v && before == v)) return;
  // it reaches the units whose first token is v
  int32_t last = u;
  for (int32_t at = u + 1;; at += kJoinThreads) {
    const int64_t j = ((int64_t)at + threadIdx.x) * a.unit;
    const int reached = __syncthreads_count(j < a.count && a.key[j] == v);
    last += reached;
    if (reached < kJoinThreads) break;
  }
  Eight sum;
#pragma unroll
  for (int k = 0; k < 4; ++k) sum.v[k] = 0;
  if (packet < a.packets) {
    for (int32_t i = u + row; i <= last; i += kJoinRows) {
      const ulonglong2* q = reinterpret_cast<const ulonglong2*>(
          a.part + ((2 * (int64_t)i + (i == u)) * a.packets + packet) * 8);
      const ulonglong2 x = q[0], y = q[1];
      sum.v[0] = lm::add2(sum.v[0], x.x);
      sum.v[1] = lm::add2(sum.v[1], x.y);
      sum.v[2] = lm::add2(sum.v[2], y.x);
      sum.v[3] = lm::add2(sum.v[3], y.y);
    }
  }
  red[row][lane][0] = make_ulonglong2(sum.v[0], sum.v[1]);
  red[row][lane][1] = make_ulonglong2(sum.v[2], sum.v[3]);
  __syncthreads();
  if (row != 0 || packet >= a.packets) return;
#pragma unroll
  for (int r = 1; r < kJoinRows; ++r) {
    const ulonglong2 x = red[r][lane][0], y = red[r][lane][1];
    sum.v[0] = lm::add2(sum.v[0], x.x);
    sum.v[1] = lm::add2(sum.v[1], x.y);
    sum.v[2] = lm::add2(sum.v[2], y.x);
    sum.v[3] = lm::add2(sum.v[3], y.y);
  }
  O* o = static_cast<O*>(a.out) + (int64_t)v * a.out_stride;
  write_sum<ALIGNED>(a, o, first_packet<ALIGNED>(o) + 8 * (int64_t)packet, sum);
}

// Tokens per unit: long units leave fewer partial sums, short ones keep the
// GPU busy when there are few tokens.
int32_t unit_of(int64_t count, int64_t dim) {
  const int64_t slabs = (packets_of(dim, false) + kSumThreads - 1) / kSumThreads;
  int32_t unit = 4;
  while (unit < kMaxUnit && count * slabs / (2 * unit) >= 6 * kSms) unit *= 2;
  return unit;
}

struct Workspace {
  size_t key[2], pos[2], part, total;
};

Workspace workspace(int64_t count, int64_t dim) {
  Workspace w{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t n = up((size_t)count * 4);
  const int32_t unit = unit_of(count, dim);
  w.key[1] = n;
  w.pos[0] = 2 * n;
  w.pos[1] = 3 * n;
  w.part = 4 * n;
  w.total = w.part + up(((size_t)count + unit - 1) / unit * 2 * packets_of(dim, false) * 8 * 4) + 256;
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
  const bool aligned = rows_aligned(weight, weight_stride, lm::dtype_bytes(weight_dtype), out, out_stride,
                                    lm::dtype_bytes(out_dtype), dim);
  const int32_t packets = (int32_t)packets_of(dim, aligned);
  // lanes per row: enough for one packet each, at most a warp
  int32_t span = 0;
  while (span < 5 && (1 << span) < packets) ++span;
  const int32_t chunks = (packets + (kPackets << span) - 1) / (kPackets << span);
  const EmbedArgs a{weight, vocab, dim,        weight_stride, tokens,  token_bytes, count,
                    scale,  out,   out_stride, flags,         packets, chunks,      span,
                    span_of(static_cast<const char*>(weight), vocab, weight_stride, dim, lm::dtype_bytes(weight_dtype))};
  const int64_t blocks = (((count * chunks) << span) + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return fail(DOBB_ERR_UNSUPPORTED, "too many tokens for one call");
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
  for (int i = 0; i < 2; ++i) {
    sa.key[i] = reinterpret_cast<uint32_t*>(base + w.key[i]);
    sa.pos[i] = reinterpret_cast<uint32_t*>(base + w.pos[i]);
  }
  sa.flags = flags;
  sa.out = dweight;
  sa.fill = accumulate ? 0 : vocab;
  sa.dim = dim;
  sa.out_stride = dweight_stride;
  sa.out_bytes = (int32_t)lm::dtype_bytes(dweight_dtype);
  cudaError_t e = cudaSuccess;
  if (count == 0) {
    fill_only<<<2 * kSms, kSortThreads, 0, s>>>(sa);
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "fill launch: %s", cudaGetErrorString(e));
    return DOBB_OK;
  }
  // a warp's worth of items per warp of the cluster, or more
  int parts = 1;
  while (parts < kMaxCluster && count > (int64_t)parts * kSortThreads) parts *= 2;
  e = cudaFuncSetAttribute(sort_and_fill, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SortShared));
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(accumulate ? parts : kSms / parts * parts));
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sizeof(SortShared);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)parts, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sort_and_fill, sa);
  }
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "token sort launch: %s", cudaGetErrorString(e));
  SumArgs a{};
  a.grad = grad;
  a.dim = dim;
  a.grad_stride = grad_stride;
  a.count = (int32_t)count;
  a.vocab = (int32_t)vocab;
  a.key = sa.key[sa.passes & 1];
  a.pos = sa.pos[sa.passes & 1];
  a.scale = scale;
  a.out = dweight;
  a.out_stride = dweight_stride;
  a.accumulate = accumulate;
  a.part = reinterpret_cast<float*>(base + w.part);
  const bool aligned = rows_aligned(grad, grad_stride, lm::dtype_bytes(grad_dtype), dweight, dweight_stride,
                                    lm::dtype_bytes(dweight_dtype), dim);
  a.packets = (int32_t)packets_of(dim, aligned);
  a.unit = unit_of(count, dim);
  a.slabs = (a.packets + kSumThreads - 1) / kSumThreads;
  a.memory = span_of(static_cast<const char*>(grad), count, grad_stride, dim, lm::dtype_bytes(grad_dtype));
  const int64_t units = (count + a.unit - 1) / a.unit;
  const int32_t join_slabs = (a.packets + kJoinPackets - 1) / kJoinPackets;
  if (units * a.slabs > INT32_MAX || units * join_slabs > INT32_MAX)
    return fail(DOBB_ERR_UNSUPPORTED, "too many tokens times columns for one call");
  const unsigned grid = (unsigned)(units * a.slabs), join = (unsigned)(units * join_slabs);
  auto launch = [&](auto writes, auto adds, auto joins) {
    if (accumulate)
      adds<<<grid, kSumThreads, 0, s>>>(a);
    else
      writes<<<grid, kSumThreads, 0, s>>>(a);
    joins<<<join, kJoinThreads, 0, s>>>(a, (int32_t)units, join_slabs);
  };
  using F = float;
  using B = __nv_bfloat16;
  switch (4 * aligned + 2 * (grad_dtype == DOBB_BF16) + (dweight_dtype == DOBB_BF16)) {
    case 0: launch(sum_runs<F, F, false, false>, sum_runs<F, F, false, true>, join_runs<F, false>); break;
    case 1: launch(sum_runs<F, B, false, false>, sum_runs<F, B, false, true>, join_runs<B, false>); break;
    case 2: launch(sum_runs<B, F, false, false>, sum_runs<B, F, false, true>, join_runs<F, false>); break;
    case 3: launch(sum_runs<B, B, false, false>, sum_runs<B, B, false, true>, join_runs<B, false>); break;
    case 4: launch(sum_runs<F, F, true, false>, sum_runs<F, F, true, true>, join_runs<F, true>); break;
    case 5: launch(sum_runs<F, B, true, false>, sum_runs<F, B, true, true>, join_runs<B, true>); break;
    case 6: launch(sum_runs<B, F, true, false>, sum_runs<B, F, true, true>, join_runs<F, true>); break;
    case 7: launch(sum_runs<B, B, true, false>, sum_runs<B, B, true, true>, join_runs<B, true>); break;
  }
  e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(DOBB_ERR_CUDA, "embedding gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
