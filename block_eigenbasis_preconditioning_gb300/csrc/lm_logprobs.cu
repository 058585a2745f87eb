// Log probabilities of given tokens, entropies, the most likely alternatives,
// and their gradient with respect to the logits.
//
// With y = scale * x over a row of V logits, M = max x, u_j = scale (x_j - M):
//   S = sum e^{u_j},  E = sum e^{u_j} u_j
//   log_sum = log S,  logp = u_t - log S,  entropy = log S - E / S.
// (M, S, E) of two parts join exactly: with M' the larger maximum and
// d = scale (M - M'), a part's S becomes S e^d and its E becomes
// (E + S d) e^d.  An entry -inf adds nothing to either sum.
#include <cooperative_groups.h>

#include <type_traits>

#include "lm_common.cuh"
#include "tc_ptx.cuh"

namespace dobb {
namespace {

namespace cg = cooperative_groups;

struct LpArgs {
  const void* logits;
  int64_t row_stride;
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
  int32_t chunks;  // blocks per row
};

// ---------------------------------------------------------------- forward
//
// A row is read once.  A thread takes 16-byte vectors, kUnroll at a time, and
// keeps its own maximum M and sums S, E; the exponentials are 2^v, and E is
// summed in units of log 2.  v = x c - R, c = scale log2(e), is one fused
// multiply-add: the reference R is M c rounded, and taken as exact from there
// on, so the rounding costs nothing.  An entry far below M is clamped to
// v = -200, where 2^v is 0, so that -inf adds 0 * -200 and not 0 * -inf.
// R is kept above -2^31, and rounds by at most 64 below 2^31, so no sum
// overflows for it.  Where the maximum of a whole slice lies beyond (a row of
// masks like -1e30 or the type's lowest value, and nothing else) the slice is
// summed again as 2^{(x - M) c}.  In the end the sums refer to M c itself.
//
// The alternatives cost no second pass: the k-th largest of the segments'
// maxima (a segment: the entries of one thread) is a lower bound
// of the k-th largest entry, so only segments whose maximum reaches it are
// read again (about k of them, from L2), and their entries that reach it are
// ranked by counting.  Among many equal logits, those above the bound are taken
// and then the first ones equal to it.

constexpr int kFwdThreads = 256;
constexpr int kFwdWarps = kFwdThreads / 32;
constexpr int kSmallThreads = 64;
constexpr int kUnroll = 4;
constexpr int kPieces = 8;  // parts of a thread's entries that have a maximum of their own
constexpr int kList = 128;
constexpr int kHits = 64;
constexpr int kCand = 128;
constexpr int kMaxCluster = 8;
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Sums {
  float m;     // the maximum
  float s, e;  // relative to it, e in units of log 2
};

struct TopScratch {
  unsigned long long best[DOBB_MAX_TOP_K];  // the largest keys, descending; 0 for none
  unsigned long long cand[kCand];
  unsigned long long warp_best[kFwdWarps];
  uint32_t bound;
  int32_t above, nlist, nhit, ncand;
  int32_t list[2][kList];  // first vectors of the segments, and of their pieces, to be read again
  int32_t hit_at[kHits];
  uint4 hit[kHits];
};

template <int NT>
struct FwdShared {
  Sums part;  // of this CTA's slice of the row
  float warp_m[NT / 32], warp_s[NT / 32], warp_e[NT / 32];
  uint32_t seg[NT];  // key of every thread's maximum
  TopScratch top;
};

// The upper half of a float that is not below x (NaN for NaN).
__device__ __forceinline__ uint16_t upper_half(float x) {
  if (!(x == x)) return 0x7fffu;
  const uint32_t u = __float_as_uint(x);
  return (uint16_t)((u + ((u & 0x80000000u) ? 0u : 0xffffu)) >> 16);
}

// Unsigned integers in the order of the floats; -0 equals 0, every NaN is
// the largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x == x)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kNegInfKey = 0x007fffffu;

// larger logit first, then lower index
__device__ __forceinline__ unsigned long long full_key(float x, int32_t j) {
  return ((unsigned long long)order_key(x) << 32) | (uint32_t)(0x7fffffff - j);
}
__device__ __forceinline__ int32_t key_index(unsigned long long k) {
  return 0x7fffffff - (int32_t)(uint32_t)k;
}

// R of a maximum, kept in a range where a sum relative to it cannot overflow;
// wide: the maximum of a slice lies outside it
constexpr float kWide = 2147483648.f;
__device__ __forceinline__ float reference(float m, float c) { return fmaxf(m * c, -kWide); }
__device__ __forceinline__ bool is_wide(float m, float c) {
  return fabsf(m) != INFINITY && !(fabsf(m * c) < kWide);
}

// scale (x - m) for x <= m, where x - m may be beyond fp32 and the product not
__device__ __forceinline__ float scaled_difference(float x, float m, float scale) {
  const float d = x - m;
  return d == -INFINITY ? 2.f * (scale * (0.5f * x - 0.5f * m)) : scale * d;
}

// the sums relative to a reference that is d larger (-d)
__device__ __forceinline__ void move_by(float& s, float& e, float d) {
  d = lm::max_nan(d, -1000.f);
  const float f = lm::exp2_fast(d);
  e = (e + s * d) * f;
  s *= f;
}

// from relative to R = reference(m, c) to relative to m c
__device__ __forceinline__ void move_to_max(float& s, float& e, float r, float m, float c) {
  if (fabsf(m) != INFINITY) move_by(s, e, -fmaf(m, c, -r));
}

__device__ __forceinline__ void order_desc(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}

// The largest top_k keys of the slice x[0 .. n), which starts at index j0 of
// the row, into sh.best; seg: the key of every segment's maximum, visible to
// all.  Segment s of kSegs holds the vectors s, s + kSegs, ...; the first
// warp's lanes hold the entries outside the vectors (sval at sat, sat < 0 for
// none).
// pieces, if given: for every piece_vecs vectors of a segment (piece p of
// segment s at p * kSegs + s) the upper half of a number that none of them
// exceeds; then only the pieces that may hold something are read again.  Runs
// on NW warps (the whole block, or one warp of it).
template <typename T, int kSegs, int NW>
__device__ __forceinline__ void slice_top(TopScratch& sh, const uint32_t* seg, const T* x, int32_t n,
                                          int32_t j0, int32_t head, int32_t nvec, int32_t sat,
                                          float sval, const uint16_t* pieces, int32_t piece_vecs,
                                          int top_k) {
  using V = lm::Vec16<T>;
  auto sync = [] {
    if (NW == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5, tid = warp * 32 + lane;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  if (warp == 0) {
    constexpr int P = kSegs / 32;
    static_assert(P == 2 || P == 8, "the sorting network below sorts 2 or 8 values");
    uint32_t s[P], keep[P];
#pragma unroll
    for (int i = 0; i < P; ++i) keep[i] = s[i] = seg[i * 32 + lane];
    // every lane's values in descending order (Batcher's odd-even merge), then
    // the largest of the lanes' first values is taken away top_k times
#pragma unroll
    for (int i = 0; i < P; i += 2) order_desc(s[i], s[i + 1]);
    if constexpr (P == 8) {
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        order_desc(s[i], s[i + 2]);
        order_desc(s[i + 1], s[i + 3]);
        order_desc(s[i + 1], s[i + 2]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) order_desc(s[i], s[i + 4]);
      order_desc(s[2], s[4]);
      order_desc(s[3], s[5]);
#pragma unroll
      for (int i = 1; i < P - 1; i += 2) order_desc(s[i], s[i + 1]);
    }
    uint32_t bound = kNegInfKey;
    for (int r = 0; r < top_k; ++r) {
      bound = __reduce_max_sync(0xffffffffu, s[0]);
      if (bound <= kNegInfKey) break;
      const unsigned who = __ballot_sync(0xffffffffu, s[0] == bound);
      if (lane == __ffs(who) - 1) {
#pragma unroll
        for (int i = 0; i < P - 1; ++i) s[i] = s[i + 1];
        s[P - 1] = 0;
      }
    }
    bound = max(bound, kNegInfKey);
    // The entries that reach the bound are wanted.  Where it is -inf (fewer
    // than top_k segments hold more), or where many segments' maxima equal it,
    // those above it are, and then the first entries equal to it.
    int reach = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) reach += __popc(__ballot_sync(0xffffffffu, keep[i] >= bound));
    const bool above = bound == kNegInfKey || reach > top_k + 8;
    int at = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = keep[i] > bound || (!above && keep[i] == bound);
      const unsigned who = __ballot_sync(0xffffffffu, in);
      // at most top_k + 8 segments: see `above`
      if (in) sh.list[0][at + __popc(who & ((1u << lane) - 1u))] = i * 32 + lane;
      at += __popc(who);
    }
    sh.best[lane] = 0;
    if (lane == 0) {
      sh.bound = bound;
      sh.above = above;
      sh.nlist = at;
      sh.nhit = sh.ncand = 0;
    }
  }
  sync();
  const uint32_t bound = sh.bound;
  const int32_t* list = sh.list[0];
  int nlist = sh.nlist;
  int32_t count = (nvec + kSegs - 1) / kSegs;  // vectors per entry of the list, kSegs apart
  if (NW == 1 && pieces) {
    const float low = key_value(bound);
    const int np = (count + piece_vecs - 1) / piece_vecs;
    int at = 0;
    for (int i0 = 0; i0 < nlist * kPieces; i0 += 32) {
      const int i = i0 + lane, p = i % kPieces;
      int32_t first = 0;
      bool in = i < nlist * kPieces && p < np;
      if (in) {
        const int32_t s = list[i / kPieces];
        in = !(__uint_as_float((uint32_t)pieces[p * kSegs + s] << 16) < low);
        first = s + p * piece_vecs * kSegs;
      }
      const unsigned who = __ballot_sync(0xffffffffu, in);
      const int mine = at + __popc(who & ((1u << lane) - 1u));
      if (in && mine < kList) sh.list[1][mine] = first;
      at += __popc(who);
    }
    if (at <= kList) {
      list = sh.list[1];
      nlist = at;
      count = piece_vecs;
    }
    __syncwarp();
  }
  // Place of this lane among those of its warp that bring something.
  auto place = [&](int* count, bool brings) {
    const unsigned who = __ballot_sync(0xffffffffu, brings);
    int first = 0;
    if (who && lane == __ffs(who) - 1) first = atomicAdd(count, __popc(who));
    return __shfl_sync(0xffffffffu, first, who ? __ffs(who) - 1 : 0) + __popc(who & ((1u << lane) - 1u));
  };
  // All entries whose key is at least `from`: first the vectors that hold one
  // (2^span lanes take an entry of the list, kGroups loads in flight), then
  // their entries.
  auto collect = [&](uint32_t from) {
    const float low = key_value(from);  // NaN where only NaN reaches `from`
    constexpr int kGroups = NW == 1 ? 1 : 4;
    const int span = count >= 32 ? 5 : 32 - __clz(count - 1), per = 32 >> span;
    for (int32_t w0 = 0; w0 < count; w0 += 32) {
      for (int q0 = warp * per; q0 < nlist; q0 += NW * kGroups * per) {
        uint4 v[kGroups];
        int32_t at[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const int q = q0 + u * NW * per + (lane >> span);
          const int32_t w = w0 + (lane & ((1 << span) - 1));
          at[u] = q < nlist && w < count ? list[q] + w * kSegs : INT32_MAX;
          if (at[u] < nvec) v[u] = __ldg(xv + at[u]);
        }
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const uint4 one[1] = {v[u]};
          const bool hit = at[u] < nvec && !(V::max_of(one) < low);
          if (__any_sync(0xffffffffu, hit)) {
            const int p = place(&sh.nhit, hit);
            if (hit && p < kHits) {
              sh.hit[p] = v[u];
              sh.hit_at[p] = head + at[u] * V::N;
            }
          }
        }
      }
    }
    sync();
    const int hits = sh.nhit;
    for (int i0 = warp * 32; i0 < min(hits, kHits) * V::N; i0 += 32 * NW) {
      const int i = i0 + lane;
      const bool in = i < min(hits, kHits) * V::N;
      const float v = in ? load_f32(reinterpret_cast<const T*>(sh.hit) + i) : 0.f;
      const bool brings = in && order_key(v) >= from;
      const int p = place(&sh.ncand, brings);
      if (brings && p < kCand) sh.cand[p] = full_key(v, j0 + sh.hit_at[i / V::N] + i % V::N);
    }
    // the entries before and after the vectors
    if (warp == 0) {
      const bool brings = sat >= 0 && order_key(sval) >= from;
      const int p = place(&sh.ncand, brings);
      if (brings && p < kCand) sh.cand[p] = full_key(sval, j0 + sat);
    }
    sync();
    const int found = hits > kHits ? kCand + 1 : sh.ncand;
    sync();
    if (tid == 0) sh.nhit = sh.ncand = 0;
    sync();
    return found;
  };
  bool above = sh.above;
  int found = bound == 0xffffffffu && above ? 0 : collect(bound + (above ? 1 : 0));
  if (found > kCand && !above) {  // many equal entries in few segments
    above = true;
    found = bound == 0xffffffffu ? 0 : collect(bound + 1);
  }
  if (found <= kCand) {
    for (int i = tid; i < found; i += 32 * NW) {
      const unsigned long long mine = sh.cand[i];
      int rank = 0;
      for (int o = 0; o < found; ++o) rank += sh.cand[o] > mine;
      if (rank < top_k) sh.best[rank] = mine;
    }
    if (above && warp == 0) {
      int at = found;
      for (int32_t i = 0; i < n && at < top_k; i += 128) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = i + u * 32 + lane < n ? load_f32(x + i + u * 32 + lane) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool is = i + u * 32 + lane < n && order_key(v[u]) == bound;
          const unsigned who = __ballot_sync(0xffffffffu, is);
          const int mine = at + __popc(who & ((1u << lane) - 1u));
          if (is && mine < top_k) sh.best[mine] = full_key(v[u], j0 + i + u * 32 + lane);
          at += __popc(who);
        }
      }
    }
  } else {
    // hundreds of different entries above the bound within fewer than top_k
    // segments: the largest key below the last one, top_k times
    unsigned long long last = ~0ull;
    for (int r = 0; r < top_k; ++r) {
      unsigned long long b = 0;
      for (int32_t j = tid; j < n; j += 32 * NW) {
        const unsigned long long key = full_key(load_f32(x + j), j0 + j);
        if (key < last && key > b) b = key;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long c = __shfl_xor_sync(0xffffffffu, b, o);
        b = c > b ? c : b;
      }
      if (NW > 1) {
        if (lane == 0) sh.warp_best[warp] = b;
        __syncthreads();
        b = sh.warp_best[0];
        for (int w = 1; w < NW; ++w) b = sh.warp_best[w] > b ? sh.warp_best[w] : b;
      }
      last = b;
      if (tid == 0) sh.best[r] = b;
      sync();
    }
  }
  sync();
}

// The vectors v of a thread onto its maximum and sums (s2, e2: two sums each,
// for the even and the odd entries); returns their largest value, NaN for NaN
template <typename T, bool ENT, int U>
__device__ __forceinline__ float add_vectors(const uint4 (&v)[U], float c, uint64_t c2, float& m,
                                             float& r, uint64_t& s2, uint64_t& e2, bool& nan) {
  using V = lm::Vec16<T>;
  const float largest = V::max_of(v);
  float b = largest;
  if (!(b == b)) {  // the maximum of the others
    nan = true;
    b = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V::N; ++i) b = fmaxf(b, V::get(v[u], i));
  }
  if (b > m) {
    m = b;
    const float to = reference(b, c), d = lm::max_nan(r - to, -1000.f), f = lm::exp2_fast(d);
    const uint64_t f2 = lm::pack2(f, f);
    if (ENT) e2 = lm::mul2(lm::fma2(s2, lm::pack2(d, d), e2), f2);
    s2 = lm::mul2(s2, f2);
    r = to;
  }
  const uint64_t minus_r = lm::pack2(-r, -r);
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < V::N / 2; ++i) {
      uint64_t w = lm::fma2(V::pair(v[u], i), c2, minus_r);
      float lo, hi;
      lm::unpack2(w, lo, hi);
      if (ENT) {
        lo = lm::max_nan(lo, -200.f);
        hi = lm::max_nan(hi, -200.f);
        w = lm::pack2(lo, hi);
      }
      const uint64_t p = lm::pack2(lm::exp2_fast(lo), lm::exp2_fast(hi));
      s2 = lm::add2(s2, p);
      if (ENT) e2 = lm::fma2(p, w, e2);
    }
  }
  return largest;
}

// Maximum, sums and the largest keys of one slice, into sh.part and sh.best
template <typename T, bool ENT, int NT>
__device__ __forceinline__ void slice_forward(FwdShared<NT>& sh, const T* x, int32_t n, int32_t j0, float c, int top_k) {
  using V = lm::Vec16<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t head = (int32_t)lm::head_of(x, n), nvec = (n - head) / V::N;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  float own = -INFINITY, r = -kWide, s, e;
  bool nan = false;
  uint64_t s2 = 0, e2 = 0;
  const uint64_t c2 = lm::pack2(c, c);
  int32_t j = tid;
  for (; j + (kUnroll - 1) * NT < nvec; j += kUnroll * NT) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = __ldg(xv + j + u * NT);
    add_vectors<T, ENT>(v, c, c2, own, r, s2, e2, nan);
  }
  for (; j < nvec; j += NT) {
    const uint4 v[1] = {__ldg(xv + j)};
    add_vectors<T, ENT>(v, c, c2, own, r, s2, e2, nan);
  }
  {
    float lo, hi;
    lm::unpack2(s2, lo, hi);
    s = lo + hi;
    lm::unpack2(e2, lo, hi);
    e = lo + hi;
  }
  // the entries before and after the vectors: fewer than 8 each
  const int32_t tail0 = head + nvec * V::N;
  const int32_t sat = tid < head ? tid : (tid >= 16 && tid - 16 < n - tail0) ? tail0 + tid - 16 : -1;
  float sval = -INFINITY;
  if (sat >= 0) {
    sval = load_f32(x + sat);
    nan |= !(sval == sval);
    if (sval > own) {
      const float to = reference(sval, c);
      move_by(s, e, r - to);
      own = sval;
      r = to;
    }
    const float w = lm::max_nan(fmaf(sval, c, -r), -200.f), p = lm::exp2_fast(w);
    s += p;
    e += p * w;
  }
  // the slice's maximum, then the sums relative to it
  float m = own;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sh.warp_m[warp] = m;
  __syncthreads();
  m = sh.warp_m[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) m = fmaxf(m, sh.warp_m[w]);
  if (is_wide(m, c)) {
    s = e = 0.f;
#pragma unroll 4
    for (int32_t i = tid; i < n; i += NT) {
      const float w = lm::max_nan((load_f32(x + i) - m) * c, -200.f), p = lm::exp2_fast(w);
      s += p;
      e += p * w;
    }
  } else {
    const float to = reference(m, c);
    move_by(s, e, r - to);
    move_to_max(s, e, to, m, c);
  }
  if (nan) s = NAN;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    if (ENT) e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  if (lane == 0) {
    sh.warp_s[warp] = s;
    sh.warp_e[warp] = e;
  }
  __syncthreads();
  if (tid == 0) {
    Sums t{m, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      t.s += sh.warp_s[w];
      t.e += sh.warp_e[w];
    }
    sh.part = t;
  }
  if (top_k > 0) {
    sh.seg[tid] = order_key(nan ? NAN : own);
    __syncthreads();
    slice_top<T, NT, NT / 32>(sh.top, sh.seg, x, n, j0, head, nvec, sat, sval, nullptr, 0, top_k);
  }
}

// The row's results but the alternatives; returns log_sum.
template <bool ENT>
__device__ __forceinline__ float write_row(const LpArgs& a, int64_t row, const Sums& r, int64_t tok,
                                           float given) {
  const bool empty = r.m == -INFINITY && r.s == 0.f;
  const float log2_sum = log2f(r.s), log_sum = kLn2 * log2_sum;
  float lp = 0.f;
  if (tok >= a.vocab) {
    lp = NAN;
    if (a.flags) atomicOr(a.flags, DOBB_FLAG_BAD_TOKEN);
  } else if (tok >= 0) {
    lp = empty ? -INFINITY : scaled_difference(given, r.m, a.scale) - log_sum;
  }
  a.logp[row] = lp;
  a.row_max[row] = r.m;
  a.log_sum[row] = log_sum;
  if (a.lse) a.lse[row] = empty ? -INFINITY : a.scale * r.m + log_sum;
  if (ENT) a.entropy[row] = empty ? 0.f : kLn2 * (log2_sum - r.e / r.s);
  return log_sum;
}

// One cluster of CTAs per row (one CTA when the rows fill the GPU): every CTA
// takes a slice of the row, the first one joins the slices.
template <typename T, bool ENT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) lp_forward(const LpArgs a) {
  __shared__ FwdShared<NT> sh;
  __shared__ unsigned long long all[kMaxCluster * DOBB_MAX_TOP_K];
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / (unsigned)parts;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  const int32_t per = (int32_t)(((int64_t)a.vocab + parts - 1) / parts);
  const int32_t lo = (int32_t)min((int64_t)a.vocab, (int64_t)per * rank);
  const int32_t n = min(a.vocab - lo, per);
  // the given token's logit is on its way while the row is read
  int64_t tok = -1;
  float given = 0.f;
  if (rank == 0 && threadIdx.x == 0) {
    tok = lm::load_token(a.tokens, a.token_bytes, row);
    if (tok >= 0 && tok < a.vocab) given = load_f32(x + tok);
  }
  slice_forward<T, ENT, NT>(sh, x + lo, n, lo, a.scale * kLog2e, a.top_k);
  if (parts > 1) cluster.sync();
  if (rank == 0) {
    if (threadIdx.x == 0) {
      Sums r = sh.part;
      const float c = a.scale * kLog2e;
      if (parts > 1) {
        for (int p = 1; p < parts; ++p) r.m = fmaxf(r.m, cluster.map_shared_rank(&sh, p)->part.m);
        const float m = r.m;
        r = Sums{m, 0.f, 0.f};
        for (int p = 0; p < parts; ++p) {
          Sums q = cluster.map_shared_rank(&sh, p)->part;
          if (q.m != m) move_by(q.s, q.e, scaled_difference(q.m, m, c));
          r.s += q.s;
          r.e += q.e;
        }
      }
      const float log_sum = write_row<ENT>(a, row, r, tok, given);
      const bool empty = r.m == -INFINITY && r.s == 0.f;
      sh.part = Sums{r.m, log_sum, empty ? 1.f : 0.f};
    }
    if (a.top_k > 0) {
      // the slices' keys: a key's rank among them is its place
      const int num = parts * a.top_k;
      for (int i = threadIdx.x; i < num; i += NT)
        all[i] = parts > 1 ? cluster.map_shared_rank(&sh, i / a.top_k)->top.best[i % a.top_k] : sh.top.best[i];
      __syncthreads();
      for (int i = threadIdx.x; i < num; i += NT) {
        const unsigned long long mine = all[i];
        int at = i;
        if (parts > 1) {
          at = 0;
          for (int o = 0; o < num; ++o) at += all[o] > mine;
        }
        if (mine != 0 && at < a.top_k) {
          const bool empty = sh.part.e != 0.f;
          a.top_ids[row * a.top_k + at] = key_index(mine);
          a.top_logp[row * a.top_k + at] =
              empty ? -INFINITY : scaled_difference(key_value((uint32_t)(mine >> 32)), sh.part.m, a.scale) - sh.part.s;
        }
      }
    }
  }
  if (parts > 1) cluster.sync();  // the slices' shared memory stays until it was read
}

// ------------------------------------------------ forward, many long rows
//
// Persistent blocks take the rows in turn.  One thread streams them through a
// ring of shared memory with bulk copies, so that the next rows are on their
// way whatever the other warps do; eight warps keep the maxima and sums, each
// at its own pace; three more warps, row about, join them, find the alternatives
// and write the row while the eight are in the next ones.
//
// Bound by HBM without alternatives (8192 x 50257 bf16: 124 us with the entropy,
// 119 without: the copy rate); with 5 alternatives 139 us, the issue slots 69 %
// busy, with 20 155 us.  One block a row, without the ring: 191 us.  What was
// tried, for 5 and 20 alternatives: 2 stages 144, 155; 2 blocks an SM with 4
// joining warps 143, 151; 2 joining warps, and code for 4 loads at once in
// them, 159, 204: the joining warps wait for instructions as much as for data.
constexpr int kStageVecs = kUnroll * kFwdThreads;
constexpr int kStages = 3;
constexpr int kJoinWarps = 3;  // take the rows in turn
constexpr int kRingThreads = kFwdThreads + 32 + 32 * kJoinWarps;
constexpr int kRingBlocks = 3;  // per SM

struct RingShared {
  uint64_t full[kStages], empty[kStages], row_full[kJoinWarps], row_empty[kJoinWarps];
  int32_t abort;
  uint64_t wait_ns;  // the limit of a wait
  float4 stat[kJoinWarps][kFwdWarps];  // maximum, reference, and the sums relative to that
  uint32_t seg[kJoinWarps][kFwdThreads];  // key of every thread's maximum
  uint16_t pieces[kJoinWarps][kPieces * kFwdThreads];
  TopScratch top[kJoinWarps];
};

constexpr uint64_t kWaitNs = 2000000000ull;

// Wait for a phase; false once a wait of this block has run out of time.
__device__ __forceinline__ bool ring_wait(RingShared& sh, uint64_t* bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*(volatile int32_t*)&sh.abort) return false;
    if (ptx::global_timer_ns() - t0 > sh.wait_ns) {
      *(volatile int32_t*)&sh.abort = 1;
      return false;
    }
  }
  return true;
}

// the same for a whole warp: all of it goes on, or none
__device__ __forceinline__ bool ring_wait_warp(RingShared& sh, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, ring_wait(sh, bar, parity));
}

// loaded: the rows that are copied in, all of them but in the self-test, where
// the waits for the others run out.  A joining warp that gives up writes its
// other rows as rows of NaN.
template <typename T, bool ENT>
__global__ void __launch_bounds__(kRingThreads, kRingBlocks)
    lp_forward_ring(const LpArgs a, int64_t rows, int64_t loaded, uint64_t wait_ns) {
  using V = lm::Vec16<T>;
  extern __shared__ __align__(128) unsigned char raw[];
  uint4* ring = reinterpret_cast<uint4*>(raw);
  RingShared& sh = *reinterpret_cast<RingShared*>(raw + (size_t)kStages * kStageVecs * 16);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&sh.full[s], 1);
      ptx::mbar_init(&sh.empty[s], kFwdWarps);
    }
    for (int s = 0; s < kJoinWarps; ++s) {
      ptx::mbar_init(&sh.row_full[s], kFwdWarps);
      ptx::mbar_init(&sh.row_empty[s], 1);
    }
    sh.abort = 0;
    sh.wait_ns = wait_ns;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  const T* logits = static_cast<const T*>(a.logits);
  const float c = a.scale * kLog2e;
  uint32_t it = 0;  // stages so far
  if (warp > kJoinWarps) {
    const int mtid = tid - 32 * (kJoinWarps + 1), mwarp = warp - kJoinWarps - 1;
    const uint64_t c2 = lm::pack2(c, c);
    uint32_t i = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, ++i) {
      const T* x = logits + row * a.row_stride;
      const int32_t head = (int32_t)lm::head_of(x, a.vocab), nvec = (a.vocab - head) / V::N;
      float own = -INFINITY, r = -kWide, piece = -INFINITY;
      bool nan = false;
      uint64_t s2 = 0, e2 = 0;
      const uint32_t buf = i % kJoinWarps;
      const int fold = nvec / kStageVecs / kPieces + 1;  // stages per piece
      int left = fold;
      uint16_t* pieces = sh.pieces[buf] + mtid;
      if (i >= kJoinWarps && !ring_wait_warp(sh, &sh.row_empty[buf], ((i / kJoinWarps) & 1) ^ 1)) return;
      for (int32_t v0 = 0; v0 < nvec; v0 += kStageVecs, ++it) {
        const uint32_t st = it % kStages;
        if (!ring_wait_warp(sh, &sh.full[st], (it / kStages) & 1)) return;
        const uint4* src = ring + st * kStageVecs + mtid;
        if (nvec - v0 >= kStageVecs) {
          uint4 v[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) v[u] = src[u * kFwdThreads];
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.empty[st]);
          piece = lm::max_nan(piece, add_vectors<T, ENT>(v, c, c2, own, r, s2, e2, nan));
        } else {
          for (int32_t j = v0 + mtid; j < nvec; j += kFwdThreads) {
            const uint4 v[1] = {src[j - v0 - mtid]};
            piece = lm::max_nan(piece, add_vectors<T, ENT>(v, c, c2, own, r, s2, e2, nan));
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.empty[st]);
        }
        if (a.top_k > 0 && (--left == 0 || v0 + kStageVecs >= nvec)) {
          *pieces = upper_half(piece);
          pieces += kFwdThreads;
          piece = -INFINITY;
          left = fold;
        }
      }
      float m = own, s, e, hi;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      lm::unpack2(s2, s, hi);
      s += hi;
      lm::unpack2(e2, e, hi);
      e += hi;
      const float to = reference(m, c);
      move_by(s, e, r - to);
      if (nan) s = NAN;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (ENT) e += __shfl_xor_sync(0xffffffffu, e, o);
      }
      if (a.top_k > 0) sh.seg[buf][mtid] = order_key(nan ? NAN : own);
      if (lane == 0) sh.stat[buf][mwarp] = make_float4(m, to, s, e);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.row_full[buf]);
    }
  } else if (warp == kJoinWarps) {
    if (lane != 0) return;
    bool ok = true;
    for (int64_t row = blockIdx.x; row < loaded && ok; row += gridDim.x) {
      const T* x = logits + row * a.row_stride;
      const int32_t head = (int32_t)lm::head_of(x, a.vocab), nvec = (a.vocab - head) / V::N;
      const uint4* src = reinterpret_cast<const uint4*>(x + head);
      for (int32_t v0 = 0; v0 < nvec; v0 += kStageVecs, ++it) {
        const uint32_t st = it % kStages;
        if (it >= kStages && !(ok = ring_wait(sh, &sh.empty[st], ((it / kStages) & 1) ^ 1))) break;
        const uint32_t bytes = (uint32_t)min(nvec - v0, kStageVecs) * 16;
        ptx::mbar_arrive_expect_tx(&sh.full[st], bytes);
        ptx::bulk_load(ring + st * kStageVecs, src + v0, bytes, &sh.full[st]);
      }
    }
    // no copy is in flight when the block ends, whatever ended the rows
    for (uint32_t p = it > kStages ? it - kStages : 0; p < it; ++p)
      ptx::mbar_wait(&sh.full[p % kStages], (p / kStages) & 1);
  } else {
    const int buf = warp;
    TopScratch& top = sh.top[buf];
    bool ok = true;
    uint32_t i = 0;
    for (int64_t row = blockIdx.x + (int64_t)buf * gridDim.x; row < rows; row += (int64_t)kJoinWarps * gridDim.x, ++i) {
      const T* x = logits + row * a.row_stride;
      const int32_t head = (int32_t)lm::head_of(x, a.vocab), nvec = (a.vocab - head) / V::N;
      const int32_t tail0 = head + nvec * V::N;
      // the given token's logit, and the entries before and after the vectors
      const int64_t tok = lm::load_token(a.tokens, a.token_bytes, row);
      const float given = tok >= 0 && tok < a.vocab ? load_f32(x + tok) : 0.f;
      const int32_t at = lane < head ? lane : (lane >= 16 && lane - 16 < a.vocab - tail0) ? tail0 + lane - 16 : -1;
      const float single = at >= 0 ? load_f32(x + at) : -INFINITY;
      ok = ok && ring_wait_warp(sh, &sh.row_full[buf], i & 1);  // not again once it has run out
      if (!ok && lane == 0 && a.flags) atomicOr(a.flags, DOBB_FLAG_TIMEOUT);
      float4 q = make_float4(-INFINITY, -kWide, 0.f, 0.f);
      if (lane < kFwdWarps) q = sh.stat[buf][lane];
      float m = ok ? fmaxf(q.x, single) : NAN;  // (NaN is wide, and stays)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      Sums t{m, 0.f, 0.f};
      if (is_wide(m, c)) {
#pragma unroll 8
        for (int32_t j = lane; j < a.vocab; j += 32) {
          const float w = lm::max_nan((load_f32(x + j) - m) * c, -200.f), p = lm::exp2_fast(w);
          t.s += p;
          t.e += p * w;
        }
      } else {
        const float to = reference(m, c);
        const float w = lm::max_nan(fmaf(single, c, -to), -200.f), p = lm::exp2_fast(w);
        t.s = q.z;
        t.e = q.w;
        move_by(t.s, t.e, q.y - to);
        t.s += p;
        t.e += p * w;
        move_to_max(t.s, t.e, to, m, c);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t.s += __shfl_xor_sync(0xffffffffu, t.s, o);
        if (ENT) t.e += __shfl_xor_sync(0xffffffffu, t.e, o);
      }
      float log_sum = 0.f;
      if (lane == 0) log_sum = write_row<ENT>(a, row, t, tok, given);
      if (a.top_k > 0) {
        log_sum = __shfl_sync(0xffffffffu, log_sum, 0);
        const bool empty = m == -INFINITY && t.s == 0.f;
        if (ok)
          slice_top<T, kFwdThreads, 1>(top, sh.seg[buf], x, a.vocab, 0, head, nvec, at, single, sh.pieces[buf],
                                       (nvec / kStageVecs / kPieces + 1) * kUnroll, a.top_k);
        if (lane < a.top_k) {
          const unsigned long long key = top.best[lane];
          a.top_ids[row * a.top_k + lane] = ok ? key_index(key) : -1;
          a.top_logp[row * a.top_k + lane] =
              empty ? -INFINITY : scaled_difference(key_value((uint32_t)(key >> 32)), m, a.scale) - log_sum;
        }
      }
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(&sh.row_empty[buf]);
    }
  }
}

// --------------------------------------------------------------- gradient
//
// In units of log 2, u_j = scale log2(e) (x_j - M) - log2(S):
//   p_j = 2^{u_j},  dx_j = p_j (A + B u_j) + scale g [j = t]
//   A = scale (l - g - h entropy),  B = -scale h ln 2
// (B = 0 without h).  Bound by HBM: 8192 x 50257 bf16 247 us, 6.7 TB/s read and
// written.  One block takes kGradVecs vectors per thread of one
// row, aligned to the output; the logits are shifted into place when the two
// differ in alignment.  The rows go from the last to the first: a forward
// call right before leaves the last ones in L2.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;

template <typename T, bool ENT>
__global__ void __launch_bounds__(kGradThreads) lp_backward(const LpGradArgs a) {
  using V = lm::Vec16<T>;
  const int64_t row = a.rows - 1 - blockIdx.x / (unsigned)a.chunks;
  const int32_t chunk = blockIdx.x % (unsigned)a.chunks;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  T* d = static_cast<T*>(a.out) + row * a.out_stride;
  const int32_t head = (int32_t)lm::head_of(d, a.vocab), nvec = (a.vocab - head) / V::N;
  const uint32_t s = (uint32_t)(reinterpret_cast<uintptr_t>(x + head) & 15);
  const int32_t v0 = chunk * (kGradThreads * kGradVecs) + threadIdx.x;
  uint4 v[kGradVecs];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int32_t j = v0 + u * kGradThreads;
    if (j < nvec) v[u] = lm::load16(x, (int64_t)head + (int64_t)j * V::N, a.vocab, s);
  }
  const float m = a.row_max[row], log_sum = a.log_sum[row];
  const int64_t tok = lm::load_token(a.tokens, a.token_bytes, row);
  const bool empty = m == -INFINITY && log_sum == -INFINITY;
  const float g = (tok >= 0 && tok < a.vocab) ? a.scale * a.g[row] : 0.f;
  const float h = ENT ? a.scale * a.h[row] : 0.f;
  const float l = a.l ? a.scale * a.l[row] : 0.f;
  const float A = ENT ? l - g - h * a.entropy[row] : l - g, B = -h * kLn2;
  // x - m may be beyond fp32, and its product with a small scale not: half of both
  const float half = fabsf(m) >= 0x1p100f && a.scale < 0.5f ? 0.5f : 1.f, minus_hm = -half * m;
  const float c = a.scale * kLog2e / half, log2_sum = log_sum * kLog2e;
  const uint64_t half2 = lm::pack2(half, half), minus_m = lm::pack2(minus_hm, minus_hm), c2 = lm::pack2(c, c),
                 minus_s = lm::pack2(-log2_sum, -log2_sum), A2 = lm::pack2(A, A), B2 = lm::pack2(B, B);
  const int32_t tok_vec = (tok >= head && tok < a.vocab) ? (int32_t)((tok - head) / V::N) : -1;
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int32_t j = v0 + u * kGradThreads;
    if (j >= nvec) break;
    uint4 o = make_uint4(0, 0, 0, 0);
    if (!empty) {
#pragma unroll
      for (int i = 0; i < V::N / 2; ++i) {
        uint64_t w = lm::fma2(lm::fma2(V::pair(v[u], i), half2, minus_m), c2, minus_s);
        float lo, hi;
        lm::unpack2(w, lo, hi);
        if (ENT) {  // p u is 0, not 0 * -inf, where p is 0
          lo = lm::max_nan(lo, -200.f);
          hi = lm::max_nan(hi, -200.f);
          w = lm::pack2(lo, hi);
        }
        const uint64_t p = lm::pack2(lm::exp2_fast(lo), lm::exp2_fast(hi));
        lm::unpack2(lm::mul2(p, ENT ? lm::fma2(B2, w, A2) : A2), lo, hi);
        if (j == tok_vec) {
          if (head + j * V::N + 2 * i == tok) lo += g;
          if (head + j * V::N + 2 * i + 1 == tok) hi += g;
        }
        V::put(o, i, lo, hi);
      }
    }
    __stcs(reinterpret_cast<uint4*>(d + head) + j, o);
  }
  if (chunk == 0) {  // the entries before and after the vectors: fewer than 8 each
    const int32_t tail0 = head + nvec * V::N;
    const int32_t tid = threadIdx.x;
    const int32_t j = tid < head ? tid : (tid >= 32 && tid - 32 < a.vocab - tail0) ? tail0 + tid - 32 : -1;
    if (j >= 0) {
      float r = 0.f;
      if (!empty) {
        const float w = lm::max_nan(fmaf(fmaf(load_f32(x + j), half, minus_hm), c, -log2_sum), -200.f);
        r = lm::exp2_fast(w) * fmaf(B, w, A) + (j == tok ? g : 0.f);
      }
      store_f32(d + j, r);
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
  if (!(scale > 0.f) || scale > 0x1p127f)  // scale log2(e) is finite, too
    return fail(DOBB_ERR_INVALID_ARG, "scale must lie in (0, 2^127] (got %g)", scale);
  if (rows == 0) return DOBB_OK;
  if (!logits || !tokens) return fail(DOBB_ERR_INVALID_ARG, "logits and tokens must be non-NULL");
  if (lm::misaligned(logits, lm::dtype_bytes(dtype)) || lm::misaligned(tokens, token_bytes))
    return fail(DOBB_ERR_INVALID_ARG, "logits or tokens not aligned to their element size");
  return DOBB_OK;
}

// loaded, wait_ns: of the ring form; selftest: no other form will do
dobb_status log_probs(const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                      const void* tokens, int token_bytes, float scale, int top_k, float* logp, float* lse,
                      float* row_max, float* log_sum, float* entropy, int32_t* top_ids, float* top_logp,
                      uint32_t* flags, void* stream, int64_t loaded, uint64_t wait_ns, bool selftest) {
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Which form, measured (us; bf16 rows with 5 alternatives unless said):
  //   4000 rows of 24 KB   ring 32, blocks of 64 threads 38, of 256 threads 47
  //   4000 rows of 12 KB (fp32)  ring 22, 64 threads 24, 256 threads 35
  //   400 rows of 24 KB    ring 7.8, 256 threads 7.5 (20 alternatives: 11.2, 9.0)
  //   150 rows of 100 KB   one block a row 9.9, two 16.6
  //   64 fp32 rows of 513 KB  clusters of 4 11.3, of 8 11.0
  const int64_t row_bytes = vocab * (int64_t)lm::dtype_bytes(logits_dtype);
  // (the ring's waits are bounded; one warp searches a whole row when nearly
  // all of it ties, which stays below the limit for rows of 2^20 entries)
  if (vocab <= (1 << 20) &&
      ((rows >= 2 * kSms && row_bytes >= 32768) || (rows >= 4 * kSms && row_bytes >= 8192))) {
    const LpArgs a{logits, row_stride, (int32_t)vocab, tokens,  token_bytes, scale,    top_k, logp,
                   lse,    row_max,    log_sum,        entropy, top_ids,     top_logp, flags};
    const size_t smem = (size_t)kStages * kStageVecs * 16 + sizeof(RingShared);
    const unsigned grid = (unsigned)(rows < kSms * kRingBlocks ? rows : kSms * kRingBlocks);
    auto launch = [&](auto kernel) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      kernel<<<grid, kRingThreads, smem, s>>>(a, rows, loaded, wait_ns);
      return cudaGetLastError();
    };
    cudaError_t e = logits_dtype == DOBB_F32
                        ? (entropy ? launch(lp_forward_ring<float, true>) : launch(lp_forward_ring<float, false>))
                        : (entropy ? launch(lp_forward_ring<__nv_bfloat16, true>)
                                   : launch(lp_forward_ring<__nv_bfloat16, false>));
    if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "log-probability launch: %s", cudaGetErrorString(e));
    return DOBB_OK;
  }
  if (selftest) return fail(DOBB_ERR_UNSUPPORTED, "this call waits for no copies");
  int parts = 1;
  while (parts < kMaxCluster && rows * parts < kSms && vocab / parts > 4096) parts *= 2;
  const bool small = rows >= 4 * kSms && row_bytes < 8192;
  // a launch holds up to 2^31 - 1 blocks
  const int64_t most = ((int64_t)1 << 30) / parts;
  cudaError_t e = cudaSuccess;
  for (int64_t r0 = 0; r0 < rows && e == cudaSuccess; r0 += most) {
    const int64_t nr = rows - r0 < most ? rows - r0 : most;
    LpArgs a{static_cast<const char*>(logits) + r0 * row_stride * (int64_t)lm::dtype_bytes(logits_dtype),
             row_stride, (int32_t)vocab,
             static_cast<const char*>(tokens) + r0 * token_bytes, token_bytes, scale, top_k, logp + r0,
             lse ? lse + r0 : nullptr, row_max + r0, log_sum + r0, entropy ? entropy + r0 : nullptr,
             top_ids ? top_ids + r0 * top_k : nullptr, top_logp ? top_logp + r0 * top_k : nullptr, flags};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(nr * parts));
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)parts, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto launch = [&](auto threads) {
      constexpr int NT = decltype(threads)::value;
      cfg.blockDim = dim3(NT);
      if (logits_dtype == DOBB_F32)
        return entropy ? cudaLaunchKernelEx(&cfg, lp_forward<float, true, NT>, a)
                       : cudaLaunchKernelEx(&cfg, lp_forward<float, false, NT>, a);
      return entropy ? cudaLaunchKernelEx(&cfg, lp_forward<__nv_bfloat16, true, NT>, a)
                     : cudaLaunchKernelEx(&cfg, lp_forward<__nv_bfloat16, false, NT>, a);
    };
    e = small ? launch(std::integral_constant<int, kSmallThreads>{}) : launch(std::integral_constant<int, kFwdThreads>{});
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "log-probability launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}

}  // namespace

extern "C" dobb_status dobb_log_probs(const void* logits, dobb_dtype logits_dtype, int64_t rows,
                                      int64_t vocab, int64_t row_stride, const void* tokens,
                                      int token_bytes, float scale, int top_k, float* logp,
                                      float* lse, float* row_max, float* log_sum, float* entropy,
                                      int32_t* top_ids, float* top_logp, uint32_t* flags,
                                      void* stream) {
  return log_probs(logits, logits_dtype, rows, vocab, row_stride, tokens, token_bytes, scale, top_k, logp, lse, row_max,
                   log_sum, entropy, top_ids, top_logp, flags, stream, rows, kWaitNs, false);
}

extern "C" dobb_status dobb_selftest_log_probs_timeout(
    const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab, int64_t row_stride, const void* tokens,
    int token_bytes, float scale, int top_k, float* logp, float* lse, float* row_max, float* log_sum, float* entropy,
    int32_t* top_ids, float* top_logp, uint32_t* flags, void* stream, int64_t loaded_rows, uint64_t timeout_ns) {
  if (loaded_rows < 0 || loaded_rows > rows || timeout_ns == 0 || timeout_ns > 5000000000ull)
    return fail(DOBB_ERR_INVALID_ARG, "loaded_rows must lie in [0, rows], timeout_ns in [1, 5e9]");
  return log_probs(logits, logits_dtype, rows, vocab, row_stride, tokens, token_bytes, scale, top_k, logp, lse, row_max,
                   log_sum, entropy, top_ids, top_logp, flags, stream, loaded_rows, timeout_ns, true);
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
  // (blocks would read logits that others have written over)
  if (dlogits != logits && lm::rows_overlap({logits, rows, vocab, row_stride, logits_dtype},
                                            {dlogits, rows, vocab, out_stride, logits_dtype}))
    return fail(DOBB_ERR_INVALID_ARG, "dlogits overlaps the logits without being them");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t per = (int64_t)kGradThreads * kGradVecs * (16 / (int64_t)lm::dtype_bytes(logits_dtype));
  const int64_t chunks = (vocab + per - 1) / per, most = ((int64_t)1 << 30) / chunks;
  const size_t bytes = lm::dtype_bytes(logits_dtype);
  cudaError_t e = cudaSuccess;
  for (int64_t end = rows; end > 0 && e == cudaSuccess; end -= most) {  // the last rows first
    const int64_t r0 = end > most ? end - most : 0;
    const LpGradArgs a{static_cast<const char*>(logits) + r0 * row_stride * (int64_t)bytes,
                       end - r0,
                       row_stride,
                       (int32_t)vocab,
                       static_cast<const char*>(tokens) + r0 * token_bytes,
                       token_bytes,
                       scale,
                       row_max + r0,
                       log_sum + r0,
                       entropy ? entropy + r0 : nullptr,
                       grad_logp + r0,
                       grad_entropy ? grad_entropy + r0 : nullptr,
                       grad_lse ? grad_lse + r0 : nullptr,
                       static_cast<char*>(dlogits) + r0 * out_stride * (int64_t)bytes,
                       out_stride,
                       (int32_t)chunks};
    const unsigned grid = (unsigned)((end - r0) * chunks);
    if (logits_dtype == DOBB_F32) {
      if (grad_entropy)
        lp_backward<float, true><<<grid, kGradThreads, 0, s>>>(a);
      else
        lp_backward<float, false><<<grid, kGradThreads, 0, s>>>(a);
    } else {
      if (grad_entropy)
        lp_backward<__nv_bfloat16, true><<<grid, kGradThreads, 0, s>>>(a);
      else
        lp_backward<__nv_bfloat16, false><<<grid, kGradThreads, 0, s>>>(a);
    }
    e = cudaGetLastError();
  }
  if (e != cudaSuccess)
    return fail(DOBB_ERR_CUDA, "log-probability gradient launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
