// Sampling of tokens from rows of logits with temperature, top-k, top-p and
// min-p, from given random numbers.
//
// With y = s x over a row of V logits, ordered from the largest (equal ones by
// the lowest index), every filter keeps a prefix of that order, so what is kept
// is given by one entry, the last one: its key and its index (the cut).
//   top-k: the k-th entry.  top-p: the last entry before which less than
//   top_p of the mass sum e^y lies.  min-p: y >= max y + log min_p.
// Where the cut lies is bounded first, from maxima of the threads' entries (top-k) or
// from the masses in bins of the exponent (top-p); what lies above the bounds is kept, the
// entries between them go to a list in shared memory that is searched exactly, in whole
// numbers, whose sums do not depend on any order.  What that does not decide (sample_generic
// says what) is found digit by digit of the key, over the row in memory.  A row is a
// cluster's of one to eight blocks.
//
// Measured (in a graph): 512 x 128256 bf16 unfiltered 74 us (78 % of the copy rate),
// min_p 0.05 68, top_k 50 42; 509 x 50257 bf16 39, 32 and 25, top_p 0.9 93 (issue slots:
// 71 instructions an entry for the sum, the bins and the choice, 4700 kept of a row);
// one row of 50257 with top_k 50 and top_p 0.95 11 (a chain of eight cluster
// barriers and shared-memory rounds).  A top_k above 1024 goes the general way:
// 509 x 50257 with top_k 2000 322 us.
//
// The token is the kept one with the largest y - log E, E ~ Exp(1): token j with
// probability e^{y_j} / sum over the kept.  The entries within a margin of the
// largest fp32 value are compared again in fp64.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>

#include "lm_logits.cuh"

namespace dobb {
namespace {

namespace cg = cooperative_groups;

struct SampleArgs {
  const void* logits;
  int64_t rows, row_stride;
  int32_t vocab;
  const float* noise;
  int64_t noise_stride;
  // per row, or NULL: the one value
  const float* scales;
  const int32_t* top_ks;
  const float *top_ps, *min_ps;
  float scale;
  int32_t top_k;
  float top_p, min_p;
  int32_t* tokens;
  float* logp;
};

constexpr int kSms = 152;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 8;
constexpr int kDigitBits = 11, kBins = 1 << kDigitBits;
constexpr int kList = 4096;       // entries among which a border is looked for
constexpr int kListBins = 1024;   // and the bins that they are put in
constexpr int kFew = 128;         // as many are compared each with each
constexpr int kFastK = 1024;      // the largest top_k that is found through the threads' maxima
constexpr int kPieces = 8;        // parts of a thread's entries that have a maximum of their own
constexpr int kBatch = 4;         // vectors of a thread in flight
constexpr float kNear = 65536.f;  // |log2 e^{max y}| from which a row takes the general way
constexpr float kFar = 0x1p100f;  // and |max|: a difference from it may leave fp32, its product with a small scale not

struct Cut {
  uint32_t key;
  int32_t index;  // the last one kept of the entries with this key
  __device__ __forceinline__ bool keeps(uint32_t k, int32_t j) const { return k > key || (k == key && j <= index); }
};

// The largest y - log E seen, in units of log 2, and the largest but one (whose
// index does not matter unless it is close).
struct Best {
  float best = -INFINITY, second = -INFINITY;
  int32_t at = -1;
  __device__ __forceinline__ void add(float score, int32_t j) {
    if (score > second) {
      if (score > best) {
        second = best;
        best = score;
        at = j;
      } else {
        second = score;
      }
    }
  }
};

// A sum of fp32 numbers in a pair of them (Knuth's two-sum).
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = hi + v, z = t - hi;
    lo += (hi - (t - z)) + (v - z);
    hi = t;
  }
  __device__ __forceinline__ void add(const Pair& v) {
    add(v.hi);
    lo += v.lo;
  }
  __device__ __forceinline__ void scale(float f) {
    hi *= f;
    lo *= f;
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
};

// What a block of the cluster tells the first one: its candidate for the token.
struct Part {
  float score, x, e;  // y - log E, the logit, the random number
  int32_t at;         // index; -1: none
  int32_t again;      // two entries of one thread are close
  float2 mass;        // of what it keeps, a pair
};

struct SampleShared {
  union {
    unsigned long long list[kList];
    struct {
      uint32_t own[2 * kBins], all[kBins];  // own: twice, for the even and the odd lanes
    } bins;
    struct {
      float max[kPieces * kThreads];
      uint32_t bins[kBins];
    } pieces;
    struct {
      unsigned long long mass[kBins];
      uint32_t count[kBins];
    } digits;
  };
  uint32_t list_bins[3][kListBins];  // counts, and the halves of the masses
  unsigned long long few[kFew], few_mass[kFew];
  unsigned long long cut;
  Part part[kMaxParts];
  float max[kMaxParts], ref[kMaxParts];
  float2 sum[kMaxParts];  // a pair
  float bound[kMaxParts][2];
  int32_t border[2];
  int32_t nlist, nfew;
  unsigned long long warp_mass[2 * kWarps];
  uint32_t warp_count[2 * kWarps];
  float red[32];
  float2 pairs[kWarps];
  double best[kWarps];
  int32_t best_at[kWarps];
  unsigned long long found_mass;  // of the entries above the digit's bin
  uint32_t found_count;
  int32_t found_bin;
  int32_t index;
};

// A row and its settings.
struct Row {
  float m, scale;
  float c, half, minus_hm;  // log2(e^{y - max}) = (x half - hm) c
  int shift;
  const float* noise;
  __device__ __forceinline__ float exponent(float x) const { return fmaf(x, half, minus_hm) * c; }
  // the same in rows near zero (a product beyond fp32 gives -inf)
  __device__ __forceinline__ float near_exponent(float x) const { return (x - m) * c; }
  static __device__ __forceinline__ bool near_zero(float m, float c) { return fabsf(m * c) < kNear && fabsf(m) < kFar; }
  __device__ __forceinline__ unsigned long long mass(float x) const {
    return (unsigned long long)__float2ull_rn(ldexpf(lm::exp2_fast(exponent(x)), shift));
  }
  // log2(e^{y - max}) - log2 E.  A random number of 0 wins, whatever the exponent (it may be
  // -inf, and -inf + inf no number); NaN and negative ones lose.
  static __device__ __forceinline__ float score(float exponent, float e) {
    return e > 0.f ? exponent - __log2f(e) : e == 0.f ? INFINITY : -INFINITY;
  }
  // y - log E relative to a reference logit, in 64 bits (as slow as 100 fp32
  // entries: only for what fp32 leaves open)
  static __device__ __noinline__ double exact(float x, float e, float scale, float ref) {
    return e >= 0.f ? (double)scale * ((double)x - (double)ref) - log((double)e) : -INFINITY;
  }
};

// log2 without a case for subnormal numbers, which read as 0: an infinite score
// sends the row the general way
__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Scores this far below the largest one may still be the largest in 64 bits:
// |x c| is off by 2^-22 of itself, the logarithm by 2^-22 and 2^-21 of itself.
__device__ __forceinline__ float near(float best) { return fabsf(best) < INFINITY ? best - 0x1p-11f - 0x1p-19f * fabsf(best) : best; }

template <typename F>
__device__ __forceinline__ float block_max(float v, float* red, F op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = op(v, red[w]);
  return v;
}
__device__ __forceinline__ float larger(float p, float q) { return fmaxf(p, q); }
__device__ __forceinline__ float larger_nan(float p, float q) { return lm::max_nan(p, q); }

__device__ __forceinline__ Pair block_pair_sum(Pair v, SampleShared& sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, v.hi, o), l = __shfl_xor_sync(0xffffffffu, v.lo, o);
    v.add(Pair{h, l});
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.pairs[threadIdx.x >> 5] = make_float2(v.hi, v.lo);
  __syncthreads();
  Pair t;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t.add(Pair{sh.pairs[w].x, sh.pairs[w].y});
  return t;
}

// the larger of two 64-bit scores, the lower index if they are equal
__device__ __forceinline__ void join(double& d, int32_t& j, double d2, int32_t j2) {
  if (j2 >= 0 && (j < 0 || d2 > d || (d2 == d && j2 < j))) {
    d = d2;
    j = j2;
  }
}
__device__ __noinline__ int32_t block_join(double d, int32_t j, SampleShared& sh) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const double d2 = __shfl_xor_sync(0xffffffffu, d, o);
    const int32_t j2 = __shfl_xor_sync(0xffffffffu, j, o);
    join(d, j, d2, j2);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.best[threadIdx.x >> 5] = d;
    sh.best_at[threadIdx.x >> 5] = j;
  }
  __syncthreads();
  d = sh.best[0];
  j = sh.best_at[0];
  for (int w = 1; w < kWarps; ++w) join(d, j, sh.best[w], sh.best_at[w]);
  return j;
}

// The smallest logit that min_p keeps: m + log(min_p) / scale, rounded up.  Sums and
// products of pairs of fp32 numbers, log(min_p) to about 2^-32: min_p = f 2^e with f near 1,
// log f = 2 (s + s^3 / 3 + ...), s = (f - 1) / (f + 1).
__device__ __forceinline__ float min_p_logit(float m, float scale, float min_p) {
  if (!(min_p > 0.f)) return -FLT_MAX;
  if (min_p >= 1.f) return m;
  int e;
  float f = frexpf(min_p, &e);  // [0.5, 1)
  if (f < 0.70710678f) {
    f *= 2.f;
    --e;
  }
  const float a = f - 1.f, b = f + 1.f, bl = (f - (b - 1.f)), q = a / b;
  const float ql = (fmaf(-q, b, a) - q * bl) / b;  // s = q + ql
  const float z = q * q;
  const float poly = z * (0.33333333f + z * (0.2f + z * (0.14285714f + z * (0.11111111f + z * (0.09090909f + z * 0.07692308f)))));
  // log 2 = ch + cl, ch with 16 bits: e ch is exact
  const float ch = 0.693145751953125f, cl = 1.4286068203094172e-06f, ef = (float)e;
  Pair log_p;
  log_p.add(ef * ch);
  log_p.add(2.f * q);
  log_p.add(2.f * fmaf(q, poly, ql));
  log_p.add(ef * cl);
  const float d = log_p.hi / scale, dl = (fmaf(-d, scale, log_p.hi) + log_p.lo) / scale;
  if (!(fabsf(d) < FLT_MAX)) return -FLT_MAX;  // far below every logit
  Pair x;
  x.add(m);
  x.add(d);
  x.add(dl);
  const float r = x.hi + x.lo;
  if (!(r > -FLT_MAX)) return -FLT_MAX;
  const float rest = (x.hi - r) + x.lo;
  return fminf(m, rest > 0.f ? nextafterf(r, INFINITY) : r);
}

// ------------------------------------------------------- the general way
//
// One block, any settings and numbers, every pass over the row in memory.  It
// takes the rows that the ways below leave: a top_k above kFastK, more equal or
// nearly equal logits at a border than the list holds, |scale max| beyond 2^16 or |max| beyond 2^100, two
// close candidates in one thread, random numbers that leave no candidate.
// f(logit, index) of the row's entries, each thread's eight at a time loaded first (one
// after the other: 509 x 50257 bf16 with top_k 2000 334 us against 317).
template <typename T, typename F>
__device__ __forceinline__ void each_entry(const T* x, int32_t n, const F& f) {
  constexpr int U = 8;
#pragma unroll 1
  for (int32_t j0 = threadIdx.x; j0 < n; j0 += U * kThreads) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = j0 + u * kThreads < n ? load_f32(x + j0 + u * kThreads) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j0 + u * kThreads < n) f(v[u], j0 + u * kThreads);
  }
}

// The entry at which the count (want_count > 0) or the mass (else) of the ordered
// entries that `cut` keeps reaches what is wanted; false if all of them are kept.
template <typename T>
__device__ bool find_cut(SampleShared& sh, const T* x, int32_t n, const Row& r, Cut& cut, uint32_t want_count, float top_p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t known = 0, prefix = 0;
  unsigned long long mass = 0;  // of the entries above the prefix
  uint32_t count = 0;
  double want_mass = 0.0;
  bool first = true;
  for (int at = 32; at > 0;) {
    const int bits = min(kDigitBits, at);
    at -= bits;
    const uint32_t bins = 1u << bits;
    for (uint32_t b = tid; b < bins; b += kThreads) {
      sh.digits.mass[b] = 0;
      sh.digits.count[b] = 0;
    }
    __syncthreads();
    each_entry(x, n, [&](float v, int32_t j) {
      const uint32_t key = order_key(v);
      if (key <= kNegInfKey || (key & known) != prefix || !cut.keeps(key, j)) return;
      const uint32_t b = (key >> at) & (bins - 1);
      // (one addition for the lanes that share a digit, by match.any: 345 us against 317)
      atomicAdd(&sh.digits.count[b], 1u);
      if (want_count == 0) atomicAdd(&sh.digits.mass[b], r.mass(v));
    });
    __syncthreads();
    // bins from the largest, kBins / kThreads a thread: what lies above each
    constexpr int kEach = kBins / kThreads;
    unsigned long long own_mass = 0;
    uint32_t own_count = 0;
    for (int i = 0; i < kEach; ++i) {
      const int b = (int)bins - 1 - (tid * kEach + i);
      if (b >= 0) {
        own_mass += sh.digits.mass[b];
        own_count += sh.digits.count[b];
      }
    }
    unsigned long long in_mass = own_mass;
    uint32_t in_count = own_count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long pm = __shfl_up_sync(0xffffffffu, in_mass, o);
      const uint32_t pc = __shfl_up_sync(0xffffffffu, in_count, o);
      if (lane >= o) {
        in_mass += pm;
        in_count += pc;
      }
    }
    if (lane == 31) {
      sh.warp_mass[warp] = in_mass;
      sh.warp_count[warp] = in_count;
    }
    if (tid == 0) sh.found_bin = -1;
    __syncthreads();
    unsigned long long before_mass = mass + in_mass - own_mass, all_mass = mass;
    uint32_t before_count = count + in_count - own_count, all_count = count;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        before_mass += sh.warp_mass[w];
        before_count += sh.warp_count[w];
      }
      all_mass += sh.warp_mass[w];
      all_count += sh.warp_count[w];
    }
    if (first) {
      want_mass = (double)top_p * (double)all_mass;
      if (want_count ? all_count <= want_count : !(top_p < 1.f)) return false;
      first = false;
    }
    for (int i = 0; i < kEach; ++i) {
      const int b = (int)bins - 1 - (tid * kEach + i);
      if (b < 0) break;
      const unsigned long long m2 = before_mass + sh.digits.mass[b];
      const uint32_t c2 = before_count + sh.digits.count[b];
      const bool here = want_count ? before_count < want_count && want_count <= c2
                                   : (double)before_mass < want_mass && want_mass <= (double)m2;
      if (here) {
        sh.found_bin = b;
        sh.found_mass = before_mass;
        sh.found_count = before_count;
      }
      before_mass = m2;
      before_count = c2;
    }
    __syncthreads();
    if (sh.found_bin < 0) return false;
    mass = sh.found_mass;
    count = sh.found_count;
    prefix |= (uint32_t)sh.found_bin << at;
    known |= (bins - 1) << at;
  }
  // entries equal to the key: the first `need` of them
  const uint32_t ties = sh.digits.count[sh.found_bin];
  uint32_t need;
  if (want_count) {
    need = want_count - count;
  } else {
    const double each = (double)(sh.digits.mass[sh.found_bin] / ties);
    need = (uint32_t)fmin((double)ties, fmax(1.0, ceil((want_mass - (double)mass) / each)));
  }
  __syncthreads();
  Cut found{prefix, prefix == cut.key ? cut.index : INT32_MAX};
  if (need < ties) {
    // warps take stretches of the row in order
    const int32_t per = (n / 32 / kWarps + 1) * 32, lo = min(n, warp * per), hi = min(n, lo + per);
    const auto is = [&](int32_t j) { return j < hi && order_key(load_f32(x + j)) == prefix && cut.keeps(prefix, j); };
    uint32_t mine = 0;
    for (int32_t j = lo; j < hi; j += 32) mine += __popc(__ballot_sync(0xffffffffu, is(j + lane)));
    if (lane == 0) sh.warp_count[warp] = mine;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sh.warp_count[w];
    if (before < need && need <= before + mine) {
      for (int32_t j = lo; j < hi; j += 32) {
        const unsigned who = __ballot_sync(0xffffffffu, is(j + lane));
        if (before + __popc(who) >= need) {
          if (lane == 0) sh.index = j + (int32_t)__fns(who, 0, (int)(need - before));
          break;
        }
        before += __popc(who);
      }
    }
    __syncthreads();
    found.index = sh.index;
  }
  __syncthreads();
  cut = found;
  return true;
}


template <typename T>
__device__ __noinline__ void sample_generic(SampleShared& sh, const SampleArgs& a, const T* x, const Row& r, int64_t row,
                                            int32_t top_k, float top_p, float min_p) {
  const int tid = threadIdx.x;
  Cut cut{kNegInfKey, -1};
  if (top_k > 0) find_cut(sh, x, a.vocab, r, cut, (uint32_t)top_k, 0.f);
  if (top_p < 1.f) find_cut(sh, x, a.vocab, r, cut, 0, top_p);
  const uint32_t key = order_key(min_p_logit(r.m, r.scale, min_p));
  if (key > cut.key) cut = Cut{key, INT32_MAX};
  const auto score = [&](float v, int32_t j) { return Row::score(r.exponent(v), r.noise[j]); };
  float best = -INFINITY, sum = 0.f;
  each_entry(x, a.vocab, [&](float v, int32_t j) {
    if (!cut.keeps(order_key(v), j)) return;
    sum += lm::exp2_fast(r.exponent(v));
    best = fmaxf(best, score(v, j));
  });
  best = block_max(best, sh.red, larger);
  sum = block_sum(sum, sh.red);
  const float from = near(best);
  double d = -INFINITY;
  int32_t at = -1;
  each_entry(x, a.vocab, [&](float v, int32_t j) {
    if (cut.keeps(order_key(v), j) && score(v, j) >= from) join(d, at, Row::exact(v, r.noise[j], r.scale, r.m), j);
  });
  at = block_join(d, at, sh);
  if (tid == 0) {
    a.tokens[row] = at;
    a.logp[row] = scaled_difference(load_f32(x + at), r.m, r.scale) - logf(sum);
  }
}

// ------------------------------------------------------------ the list
//
// (key, index) pairs in the first block's shared memory, in no order.  What is asked
// of them are counts and sums of whole numbers, which no order changes.

// e^{y - max y} in units of 2^-38, in two halves: those of the whole list fit 32 bits
constexpr int kHalf = 19, kUnit = 2 * kHalf;
__device__ __forceinline__ void whole_mass(float log2_mass, uint32_t& hi, uint32_t& lo) {
  const float f = lm::exp2_fast(log2_mass) * (float)(1 << kHalf);
  hi = (uint32_t)f;
  lo = (uint32_t)((f - (float)hi) * (float)(1 << kHalf));
}
__device__ __forceinline__ unsigned long long join_halves(uint32_t hi, uint32_t lo) {
  return ((unsigned long long)hi << kHalf) + lo;
}
__device__ __forceinline__ float list_logit(unsigned long long k) { return key_value((uint32_t)(k >> 32)); }

// ceil(p s) for p in (0, 1), s < 2^62
__device__ __forceinline__ unsigned long long share_of(unsigned long long s, float p) {
  int e;
  const unsigned long long digits = (unsigned long long)(uint32_t)(frexpf(p, &e) * 0x1p24f);
  const int shift = 24 - e;  // p = digits / 2^shift, shift >= 24
  const unsigned long long hi = __umul64hi(s, digits), lo = s * digits;
  if (shift >= 64) return 1 + (shift < 128 ? hi >> (shift - 64) : 0);
  const unsigned long long whole = (hi << (64 - shift)) | (lo >> shift);
  return whole + ((lo & ((1ull << shift) - 1)) != 0 ? 1 : 0);
}

// a mass of up to 2^15 in units of 2^-38; 0 for what is not above 0, the largest
// number beyond
__device__ __forceinline__ unsigned long long whole_mass(const Pair& v) {
  const float f = v.hi + v.lo, rest = (v.hi - f) + v.lo;
  if (!(f > 0.f)) return 0;
  if (!(f < 32768.f)) return ~0ull;
  const uint32_t i = (uint32_t)f;
  const float q = (f - (float)i) * (float)(1 << kHalf);
  const uint32_t hi = (uint32_t)q, lo = (uint32_t)((q - (float)hi) * (float)(1 << kHalf));
  const long long total = ((long long)i << kUnit) + (long long)join_halves(hi, lo) + (long long)(int32_t)(rest * 0x1p38f);
  return total > 0 ? (unsigned long long)total : 0;
}

// the mass of the list's entries from `cut` up
__device__ __forceinline__ unsigned long long list_mass(SampleShared& sh, int n, unsigned long long cut, const Row& r) {
  uint32_t hi = 0, lo = 0;
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (sh.list[i] >= cut) {
      uint32_t h, l;
      whole_mass(r.near_exponent(list_logit(sh.list[i])), h, l);
      hi += h;
      lo += l;
    }
  hi = __reduce_add_sync(0xffffffffu, hi);
  lo = __reduce_add_sync(0xffffffffu, lo);
  if ((threadIdx.x & 31) == 0) sh.warp_mass[threadIdx.x >> 5] = join_halves(hi, lo);
  __syncthreads();
  unsigned long long s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sh.warp_mass[w];
  __syncthreads();
  return s;
}

// What list_border looks for: the smallest key T such that the entries from T up are
// `count` many, or (count 0) have at least the mass `want`, which all of them have.

// Bit by bit, until one entry is left in question.
__device__ __noinline__ unsigned long long list_search(SampleShared& sh, int n, int count, unsigned long long want, const Row& r) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long t = 0;
  int with = n, above = 0;  // entries from t up, and from the next candidate above the question up
#pragma unroll 1
  for (int bit = 63, round = 0; bit >= 0; --bit) {
    const unsigned long long cand = t | (1ull << bit);
    uint32_t c = 0, hi = 0, lo = 0;
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = sh.list[i];
      if (k < cand) continue;
      ++c;
      if (count == 0) {
        uint32_t h, l;
        whole_mass(r.near_exponent(list_logit(k)), h, l);
        hi += h;
        lo += l;
      }
    }
    c = __reduce_add_sync(0xffffffffu, c);
    const int at = (round & 1) * kWarps;
    round ^= 1;
    if (count == 0) {
      hi = __reduce_add_sync(0xffffffffu, hi);
      lo = __reduce_add_sync(0xffffffffu, lo);
      if (lane == 0) sh.warp_mass[at + warp] = join_halves(hi, lo);
    }
    if (lane == 0) sh.warp_count[at + warp] = c;
    __syncthreads();
    int all = 0;
    unsigned long long s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      all += (int)sh.warp_count[at + w];
      s += count == 0 ? sh.warp_mass[at + w] : 0;
    }
    if (count ? all >= count : s >= want) {
      t = cand;
      with = all;
      if (count && all == count) break;
    } else {
      above = all;
    }
    if (with - above <= 1) break;
  }
  __syncthreads();
  return t;
}

// The first of kListBins bins up to which `count` entries or the mass `want` lie
// (count 0); what lies before it.
struct ListBin {
  int bin;
  uint32_t before, here;
  unsigned long long mass;
};
__device__ __forceinline__ ListBin find_list_bin(SampleShared& sh, uint32_t count, unsigned long long want) {
  constexpr int kEach = kListBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t c = 0;
  unsigned long long s = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    c += sh.list_bins[0][b];
    s += join_halves(sh.list_bins[1][b], sh.list_bins[2][b]);
  }
  uint32_t ic = c;
  unsigned long long is = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t pc = __shfl_up_sync(0xffffffffu, ic, o);
    const unsigned long long ps = __shfl_up_sync(0xffffffffu, is, o);
    if (lane >= o) {
      ic += pc;
      is += ps;
    }
  }
  if (lane == 31) {
    sh.warp_count[warp] = ic;
    sh.warp_mass[warp] = is;
  }
  __syncthreads();
  c = ic - c;
  s = is - s;
  for (int w = 0; w < warp; ++w) {
    c += sh.warp_count[w];
    s += sh.warp_mass[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    const uint32_t here = sh.list_bins[0][b];
    const unsigned long long mass = join_halves(sh.list_bins[1][b], sh.list_bins[2][b]);
    if (count ? c < count && count <= c + here : s < want && want <= s + mass) {
      sh.found_bin = b;
      sh.found_count = c;
      sh.found_mass = s;
      sh.border[0] = (int32_t)here;
    }
    c += here;
    s += mass;
  }
  __syncthreads();
  const ListBin f{sh.found_bin, sh.found_count, (uint32_t)sh.border[0], sh.found_mass};
  __syncthreads();
  return f;
}

// The border among up to kFew entries of sh.few, each compared with each.
__device__ __forceinline__ unsigned long long few_border(SampleShared& sh, int n, uint32_t before, unsigned long long mass, uint32_t count,
                                                         unsigned long long want) {
  const int tid = threadIdx.x;
  if (tid < n) {
    const unsigned long long mine = sh.few[tid], own = sh.few_mass[tid];
#pragma unroll 4
    for (int o = 0; o < n; ++o) {
      const bool ahead = sh.few[o] > mine;
      before += ahead;
      mass += ahead ? sh.few_mass[o] : 0;
    }
    if (count ? before + 1 == count : mass < want && want <= mass + own) sh.cut = mine;
  }
  __syncthreads();
  const unsigned long long t = sh.cut;
  __syncthreads();
  return t;
}

// All entries lie in [lo, hi].  Bins by their logits; the entries of the border's
// bin each with each, or, where they are equal, bins by their indices.
__device__ __noinline__ unsigned long long list_border(SampleShared& sh, int n, uint32_t count, unsigned long long want, const Row& r,
                                                       float lo, float hi, int32_t vocab) {
  const int tid = threadIdx.x;
  const auto clear = [&] {
    for (int b = tid; b < 3 * kListBins; b += kThreads) sh.list_bins[0][b] = 0;
    if (tid == 0) sh.nfew = 0;
    __syncthreads();
  };
  // the entries for which in(key) holds go to sh.few
  const auto collect = [&](auto in) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = sh.list[i];
      if (!in(k)) continue;
      const int at = atomicAdd(&sh.nfew, 1);
      if (at >= kFew) continue;  // (never: they were counted)
      uint32_t h, l;
      whole_mass(r.near_exponent(list_logit(k)), h, l);
      sh.few[at] = k;
      sh.few_mass[at] = join_halves(h, l);
    }
    __syncthreads();
  };
  if (n <= kFew) {
    if (tid == 0) sh.nfew = 0;
    __syncthreads();
    collect([](unsigned long long) { return true; });
    return few_border(sh, n, 0, 0, count, want);
  }
  if (!(hi - lo < 64.f)) {  // a wide bound: the smallest entry
    float least = INFINITY;
    for (int i = tid; i < n; i += kThreads) least = fminf(least, list_logit(sh.list[i]));
    lo = -block_max(-least, sh.red, larger);
  }
  const float per = (float)(kListBins - 1) / (hi - lo);
  const auto bin_of = [&](unsigned long long k) {
    return (int)fminf(fmaxf((hi - list_logit(k)) * per, 0.f), (float)(kListBins - 1));  // (not a number: 0)
  };
  clear();
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long k = sh.list[i];
    const int b = bin_of(k);
    uint32_t h, l;
    whole_mass(r.near_exponent(list_logit(k)), h, l);
    atomicAdd(&sh.list_bins[0][b], 1u);
    atomicAdd(&sh.list_bins[1][b], h);
    atomicAdd(&sh.list_bins[2][b], l);
  }
  __syncthreads();
  ListBin f = find_list_bin(sh, count, want);
  if (f.here <= kFew) {
    collect([&](unsigned long long k) { return bin_of(k) == f.bin; });
    return few_border(sh, (int)f.here, f.before, f.mass, count, want);
  }
  // are they equal?
  if (tid == 0) {
    sh.few[0] = 0;
    sh.few[1] = ~0ull;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads)
    if (bin_of(sh.list[i]) == f.bin) {
      atomicMax(reinterpret_cast<uint32_t*>(&sh.few[0]), (uint32_t)(sh.list[i] >> 32));
      atomicMin(reinterpret_cast<uint32_t*>(&sh.few[1]), (uint32_t)(sh.list[i] >> 32));
    }
  __syncthreads();
  const uint32_t key = *reinterpret_cast<const uint32_t*>(&sh.few[0]);
  const bool equal = key == *reinterpret_cast<const uint32_t*>(&sh.few[1]);
  __syncthreads();
  if (!equal) return list_search(sh, n, (int)count, want, r);
  uint32_t h, l;
  whole_mass(r.near_exponent(key_value(key)), h, l);
  const float per_index = (float)kListBins / (float)vocab;
  const auto index_bin = [&](unsigned long long k) { return min((int)((float)key_index(k) * per_index), kListBins - 1); };
  clear();
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long k = sh.list[i];
    if ((uint32_t)(k >> 32) != key) continue;
    const int b = index_bin(k);
    atomicAdd(&sh.list_bins[0][b], 1u);
    atomicAdd(&sh.list_bins[1][b], h);
    atomicAdd(&sh.list_bins[2][b], l);
  }
  __syncthreads();
  const ListBin g = find_list_bin(sh, count ? count - f.before : 0, want - f.mass);
  if (g.here > kFew) return list_search(sh, n, (int)count, want, r);
  collect([&](unsigned long long k) { return (uint32_t)(k >> 32) == key && index_bin(k) == g.bin; });
  return few_border(sh, (int)g.here, f.before + g.before, f.mass + g.mass, count, want);
}

struct Listed {
  unsigned long long mass;
  Part best;
};

// What is kept of the list: the entries from `cut` up whose logit is at least min_x.
__device__ __forceinline__ Listed take_list(SampleShared& sh, int n, unsigned long long cut, float min_x, const Row& r) {
  const int tid = threadIdx.x;
  Listed out{};
  Best best;
  uint32_t hi = 0, lo = 0;
  const auto kept = [&](unsigned long long k) { return k >= cut && list_logit(k) >= min_x; };
  const auto score = [&](float x, float e) { return Row::score(r.near_exponent(x), e); };
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long k = sh.list[i];
    if (!kept(k)) continue;
    const float x = list_logit(k);
    uint32_t h, l;
    whole_mass(r.near_exponent(x), h, l);
    hi += h;
    lo += l;
    best.add(score(x, r.noise[key_index(k)]), i);
  }
  hi = __reduce_add_sync(0xffffffffu, hi);
  lo = __reduce_add_sync(0xffffffffu, lo);
  if ((tid & 31) == 0) sh.warp_mass[tid >> 5] = join_halves(hi, lo);
  const float top = block_max(best.best, sh.red, larger), from = near(top);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) out.mass += sh.warp_mass[w];
  const bool in = best.at >= 0 && best.best >= from;
  if (tid == 0) sh.index = -1;
  // one thread's one entry, or what 64 bits say (also where no score is above -inf)
  const int two = __syncthreads_or(in && best.second >= from), one = __syncthreads_count(in);
  int32_t at = -1;
  if (one == 1 && !two) {
    if (in) sh.index = best.at;
    __syncthreads();
    at = sh.index;
  } else {
    double d = -INFINITY;
    int32_t j = -1;
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long k = sh.list[i];
      if (!kept(k)) continue;
      const float x = list_logit(k), e = r.noise[key_index(k)];
      if (score(x, e) >= from) join(d, j, Row::exact(x, e, r.scale, r.m), key_index(k));
    }
    j = block_join(d, j, sh);
    if (j >= 0)
      for (int i = tid; i < n; i += kThreads)
        if (key_index(sh.list[i]) == j) sh.index = i;
    __syncthreads();
    at = sh.index;
  }
  out.best.at = -1;
  if (at >= 0) {
    const unsigned long long k = sh.list[at];
    out.best.at = key_index(k);
    out.best.x = list_logit(k);
    out.best.e = r.noise[out.best.at];
    out.best.score = score(out.best.x, out.best.e);
  }
  out.best.again = 0;
  return out;
}

// ----------------------------------------------------------------- slices
//
// The row's vectors go round the cluster's blocks kThreads at a time; the entries
// before and behind them (fewer than 8 each) are the first block's.
template <typename T>
struct Slice {
  using V = lm::Vec16<T>;
  const uint4* xv;
  int32_t head, nvec, at0, step, single;  // single: the entry outside the vectors of this thread, or -1
  __device__ __forceinline__ Slice(const T* x, int32_t vocab, int parts, int rank) {
    head = (int32_t)lm::head_of(x, vocab);
    nvec = (vocab - head) / V::N;
    xv = reinterpret_cast<const uint4*>(x + head);
    at0 = rank * kThreads + threadIdx.x;
    step = parts * kThreads;
    const int32_t tail0 = head + nvec * V::N, tid = threadIdx.x;
    single = rank != 0 ? -1 : tid < head ? tid : (tid >= 16 && tid - 16 < vocab - tail0) ? tail0 + tid - 16 : -1;
  }
  __device__ __forceinline__ int32_t index(int32_t v) const { return head + v * V::N; }
  __device__ __forceinline__ void load(uint4 (&v)[kBatch], int32_t v0) const {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) v[u] = v0 + u * step < nvec ? __ldg(xv + v0 + u * step) : V::fill_neg_inf();
  }
  // f(vector, its number) of the thread's vectors whose largest entry reaches
  // `low`, which is above -inf
  template <typename F>
  __device__ __forceinline__ void each_from(float low, const F& f) const {
#pragma unroll 1
    for (int32_t v0 = at0; v0 < nvec; v0 += kBatch * step) {
      uint4 v[kBatch];
      load(v, v0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint4 one[1] = {v[u]};
        if (V::max_of(one) >= low) f(v[u], v0 + u * step);
      }
    }
  }
};

// The same with the random numbers: groups of four entries on their 16-byte
// boundaries; the logits (8 bytes of bf16) are shifted into place where the rows
// differ in alignment.  (On the logits' boundaries eight bf16 entries have 32 bytes of
// random numbers, twice as many requests: 512 x 128256 84 us against 74.)
template <typename T>
struct Groups {
  static constexpr int kWords = (int)sizeof(T);
  struct Four {
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int i) const {
      return sizeof(T) == 4 ? __uint_as_float(w[i % kWords]) : (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
    static __device__ __forceinline__ float bf16_lo(uint32_t v) { return lm::bf16_lo(v); }
    static __device__ __forceinline__ float bf16_hi(uint32_t v) { return lm::bf16_hi(v); }
  };
  const T* x;
  const float* noise;
  int32_t vocab, head, n, at0, step, single;
  uint32_t shift;
  __device__ __forceinline__ Groups(const T* x, const float* noise, int32_t vocab, int parts, int rank)
      : x(x), noise(noise), vocab(vocab) {
    head = (int32_t)lm::head_of(noise, vocab);
    n = (vocab - head) / 4;
    at0 = rank * kThreads + threadIdx.x;
    step = parts * kThreads;
    const int32_t tail0 = head + 4 * n, tid = threadIdx.x;
    single = rank != 0 ? -1 : tid < head ? tid : (tid >= 16 && tid - 16 < vocab - tail0) ? tail0 + tid - 16 : -1;
    shift = (uint32_t)(reinterpret_cast<uintptr_t>(x + head) & (4 * sizeof(T) - 1));
  }
  __device__ __forceinline__ int32_t index(int32_t g) const { return head + 4 * g; }
  __device__ __forceinline__ float4 random(int32_t g) const { return __ldg(reinterpret_cast<const float4*>(noise + index(g))); }
  __device__ __forceinline__ Four none() const {
    Four f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) f.w[i] = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    return f;
  }
  __device__ __forceinline__ Four load(int32_t g) const {
    Four f;
    const int32_t j = index(g);
    if constexpr (sizeof(T) == 4) {
      const uint4 v = lm::load16(x, (int64_t)j, vocab, shift);
      f.w[0] = v.x;
      f.w[1] = v.y;
      f.w[2] = v.z;
      f.w[3] = v.w;
    } else if (shift == 0) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(x + j));
      f.w[0] = v.x;
      f.w[1] = v.y;
    } else {
      const int32_t before = (int32_t)(shift / 2);
      if (j >= before && (int64_t)j - before + 8 <= vocab) {
        const uint2* q = reinterpret_cast<const uint2*>(x + j - before);
        const uint2 a = __ldg(q), b = __ldg(q + 1);
        uint32_t w0 = a.x, w1 = a.y, w2 = b.x;
        if (shift & 4) {
          w0 = a.y;
          w1 = b.x;
          w2 = b.y;
        }
        f.w[0] = (shift & 2) ? __funnelshift_r(w0, w1, 16) : w0;
        f.w[1] = (shift & 2) ? __funnelshift_r(w1, w2, 16) : w1;
      } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(x + j);
        f.w[0] = h[0] | ((uint32_t)h[1] << 16);
        f.w[1] = h[2] | ((uint32_t)h[3] << 16);
      }
    }
    return f;
  }
};
constexpr int kGroups = 4;  // of a thread in flight

// The largest y - log E of a thread's batches of kGroups groups, in units of log 2,
// the batch's first group (-2 - j: entry j, outside the groups), and the largest of
// the other batches.
struct BestBatch {
  float best = -INFINITY, second = -INFINITY;
  int32_t at = -1;
  __device__ __forceinline__ void add(float score, int32_t where) {
    second = fmaxf(second, fminf(best, score));
    at = score > best ? where : at;
    best = fmaxf(best, score);
  }
};

// Lower bounds of the rank0-th and rank1-th largest of the block's numbers (kPieces
// a thread, m the largest): by bins from m down, over the range that they span
// (64 at most).
__device__ __forceinline__ void bounds(SampleShared& sh, const float (&piece)[kPieces], float m, int rank0, int rank1, float& t0, float& t1) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kEach = kBins / kThreads;
  uint32_t* bins = sh.pieces.bins;
  float least = INFINITY;
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    bins[q * kThreads + tid] = 0;
    if (piece[q] > -INFINITY) least = fminf(least, piece[q]);
  }
  static_assert(kBins == kPieces * kThreads, "cleared above");
  least = -block_max(-least, sh.red, larger);
  const float range = fminf(fmaxf(m - least, 0.f), 64.f), per = range > 0.f ? (float)(kBins - 1) / range : 0.f;
#pragma unroll
  for (int q = 0; q < kPieces; ++q)
    if (piece[q] > -INFINITY) atomicAdd(&bins[(int)fminf((m - piece[q]) * per, (float)(kBins - 1))], 1u);
  if (tid == 0) sh.border[0] = sh.border[1] = kBins - 1;
  __syncthreads();
  uint32_t b[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += b[i] = bins[tid * kEach + i];
  uint32_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t p = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += p;
  }
  if (lane == 31) sh.warp_count[warp] = upto;
  __syncthreads();
  upto -= sum;
  for (int w = 0; w < warp; ++w) upto += sh.warp_count[w];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t before = upto;
    upto += b[i];
    if (before < (uint32_t)rank0 && (uint32_t)rank0 <= upto) sh.border[0] = tid * kEach + i;
    if (before < (uint32_t)rank1 && (uint32_t)rank1 <= upto) sh.border[1] = tid * kEach + i;
  }
  __syncthreads();
  // the bin's lower edge, and a little below it
  const auto edge = [&](int bin) {
    if (bin >= kBins - 1) return -FLT_MAX;
    const float x = per > 0.f ? m - (float)(bin + 1) / per : m;
    return fmaxf(x - 0x1p-20f * (fabsf(m) + fabsf(x)), -FLT_MAX);
  };
  t0 = edge(sh.border[0]);
  t1 = edge(sh.border[1]);
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_rows(const SampleArgs a) {
  using V = lm::Vec16<T>;
  __shared__ SampleShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  // (the others' shared memory is there once all of them have started)
  cg::cluster_group::arrival_token started{};
  if (parts > 1) started = cluster.barrier_arrive();
  const auto all_started = [&] {
    if (parts > 1) cluster.barrier_wait(static_cast<cg::cluster_group::arrival_token&&>(started));
  };
  const int64_t row = blockIdx.x / (unsigned)parts;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  Row r;
  r.noise = a.noise + row * a.noise_stride;
  r.scale = a.scales ? a.scales[row] : a.scale;
  int32_t top_k = a.top_ks ? a.top_ks[row] : a.top_k;
  float top_p = a.top_ps ? a.top_ps[row] : a.top_p;
  const float min_p = a.min_ps ? a.min_ps[row] : a.min_p;
  if (top_p <= 0.f) top_k = 1;
  if (!(top_p < 1.f) || top_k == 1) top_p = 1.f;
  if (top_k < 0 || top_k >= a.vocab) top_k = 0;
  const bool usable = r.scale > 0.f && r.scale <= 0x1p127f;
  r.c = r.scale * kLog2e;
  const Slice<T> sl(x, a.vocab, parts, rank);
  const float single = sl.single >= 0 ? load_f32(x + sl.single) : -INFINITY;
  SampleShared* lead = parts > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
  const auto sync = [&] {
    if (parts > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  const auto each = [&](int p) { return parts > 1 ? cluster.map_shared_rank(&sh, p) : &sh; };
  if (tid == 0) sh.nlist = 0;
  const auto put = [&](float v, int32_t j) {
    const int32_t at = atomicAdd(&lead->nlist, 1);
    if (at < kList) lead->list[at] = full_key(v, j);
  };
  const auto finish = [&](int32_t at, float logp) {
    if (tid == 0) {
      a.tokens[row] = at;
      a.logp[row] = logp;
    }
  };
  bool general = false;
  // whether the row ends here: no token can occur, or a number is none
  const auto ended = [&](float m) {
    if (m < INFINITY && m > -INFINITY && usable) return false;
    if (rank == 0) finish(-1, m == -INFINITY && usable ? -INFINITY : NAN);
    return true;
  };
  float m = -INFINITY;

  if (top_k > 0) {
    // ---- top-k: a bound of the k-th largest entry from the pieces' maxima (a piece: every
    // eighth batch of a thread), then the entries that reach it on the first block's list
#pragma unroll
    for (int q = 0; q < kPieces; ++q) sh.pieces.max[q * kThreads + tid] = q == 0 ? single : -INFINITY;
    int q = 0;
#pragma unroll 1
    for (int32_t v0 = sl.at0; v0 < sl.nvec; v0 += kBatch * sl.step, q = (q + 1) % kPieces) {
      uint4 v[kBatch];
      sl.load(v, v0);
      float* piece = sh.pieces.max + q * kThreads + tid;
      *piece = lm::max_nan(*piece, V::max_of(v));
    }
    float piece[kPieces];
    uint32_t hot = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      piece[i] = sh.pieces.max[i * kThreads + tid];
      m = lm::max_nan(m, piece[i]);
    }
    m = block_max(m, sh.red, larger_nan);
    const bool fast = top_k <= kFastK;
    float b0 = -FLT_MAX, b1 = -FLT_MAX;
    if (fast && m > -INFINITY) bounds(sh, piece, m, top_k, (top_k + parts - 1) / parts, b0, b1);
    all_started();
    if (tid < parts) {
      SampleShared* o = each(tid);
      o->max[rank] = m;
      o->bound[rank][0] = b0;
      o->bound[rank][1] = b1;
    }
    sync();
    float most = -FLT_MAX, least = FLT_MAX;
    for (int p = 0; p < parts; ++p) {
      m = lm::max_nan(m, sh.max[p]);
      most = fmaxf(most, sh.bound[p][0]);
      least = fminf(least, sh.bound[p][1]);
    }
    if (ended(m)) return;
    // every block has k / parts entries that reach the smallest of those bounds
    const float low = fmaxf(most, least);
    if (fast) {
      if (single >= low) put(single, sl.single);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) hot |= (piece[i] >= low ? 1u : 0u) << i;
      q = 0;
#pragma unroll 1
      for (int32_t v0 = sl.at0; v0 < sl.nvec; v0 += kBatch * sl.step, q = (q + 1) % kPieces) {
        if (!((hot >> q) & 1)) continue;
        uint4 v[kBatch];
        sl.load(v, v0);
        uint32_t asked = 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int i = 0; i < V::N; ++i) asked |= (V::get(v[u], i) >= low ? 1u : 0u) << (u * V::N + i);
        while (asked) {
          const int i = __ffs(asked) - 1;
          asked &= asked - 1;
          const int32_t j = sl.index(v0 + i / V::N * sl.step) + i % V::N;
          put(load_f32(x + j), j);
        }
      }
    }
    sync();
    if (rank != 0) return;
    const int n = sh.nlist;
    r.m = m;
    if (fast && n <= kList && Row::near_zero(m, r.c)) {
      unsigned long long cut = n > top_k ? list_border(sh, n, top_k, 0, r, low, m, a.vocab) : 0;
      if (top_p < 1.f) {
        // the mass of the first k, then the border within them
        const unsigned long long at =
            list_border(sh, n, 0, share_of(list_mass(sh, n, cut, r), top_p), r, low, m, a.vocab);
        cut = at > cut ? at : cut;
      }
      const Listed t = take_list(sh, n, cut, min_p_logit(m, r.scale, min_p), r);
      if (t.best.at >= 0) return finish(t.best.at, kLn2 * (r.near_exponent(t.best.x) - log2f((float)t.mass * 0x1p-38f)));
    }
    general = true;
  }

  // ---- all others: the maximum and the sum of e^y, and without filters the best score
  const bool plain = top_p == 1.f && !(min_p > 0.f);
  if (!general) {
    const uint64_t c2 = lm::pack2(r.c, r.c);
    const Groups<T> gr(x, r.noise, a.vocab, parts, rank);
    float own = -INFINITY, ref = -kWide;
    bool nan = false;
    uint64_t s2 = 0, e2 = 0;
    // top_p's total: a batch's sum goes to a pair at once, as a plain fp32 sum over a thread's
    // entries would be off by up to their number times 2^-25 of itself (131072 nearly equal
    // entries a row: 2^-19; half a million: 2^-17).  Costs 509 x 50257 bf16 with top_p 115 -> 116 us
    Pair pair;
    const auto flush = [&](float before) {  // the reference that the pair is relative to
      if (ref != before) pair.scale(lm::exp2_fast(lm::max_nan(before - ref, -1000.f)));
      float lo, hi;
      lm::unpack2(s2, lo, hi);
      pair.add(lo + hi);
      s2 = 0;
    };
    BestBatch best;
    float outside = single;  // this thread's entry outside the vectors or groups
    if (plain) {
#pragma unroll 1
      for (int32_t g0 = gr.at0; g0 < gr.n; g0 += kGroups * gr.step) {
        typename Groups<T>::Four f[kGroups];
        float4 e[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const int32_t g = g0 + u * gr.step;
          f[u] = g < gr.n ? gr.load(g) : gr.none();
          e[u] = g < gr.n ? gr.random(g) : make_float4(1.f, 1.f, 1.f, 1.f);
        }
        uint4 v[kGroups * 4 / V::N];
#pragma unroll
        for (int u = 0; u < kGroups * 4 / V::N; ++u) {
          if constexpr (sizeof(T) == 4)
            v[u] = make_uint4(f[u].w[0], f[u].w[1], f[u].w[2], f[u].w[3]);
          else
            v[u] = make_uint4(f[2 * u].w[0], f[2 * u].w[1], f[2 * u + 1].w[0], f[2 * u + 1].w[1]);
        }
        add_vectors<T, false>(v, r.c, c2, own, ref, s2, e2, nan);
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          top = fmaxf(top, fmaxf(fmaf(f[u].get(0), r.c, -log2_fast(e[u].x)), fmaf(f[u].get(1), r.c, -log2_fast(e[u].y))));
          top = fmaxf(top, fmaxf(fmaf(f[u].get(2), r.c, -log2_fast(e[u].z)), fmaf(f[u].get(3), r.c, -log2_fast(e[u].w))));
        }
        best.add(top, g0);
      }
      flush(ref);
      outside = -INFINITY;
      if (gr.single >= 0) {
        outside = load_f32(x + gr.single);
        best.add(fmaf(outside, r.c, -log2_fast(r.noise[gr.single])), -2 - gr.single);
      }
    } else {
      int32_t v0 = sl.at0;
#pragma unroll 1
      for (; v0 + (kBatch - 1) * sl.step < sl.nvec; v0 += kBatch * sl.step) {
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = __ldg(sl.xv + v0 + u * sl.step);
        const float before = ref;
        add_vectors<T, false>(v, r.c, c2, own, ref, s2, e2, nan);
        flush(before);
      }
      const float before = ref;
#pragma unroll 1
      for (; v0 < sl.nvec; v0 += sl.step) {
        const uint4 v[1] = {__ldg(sl.xv + v0)};
        add_vectors<T, false>(v, r.c, c2, own, ref, s2, e2, nan);
      }
      flush(before);
    }
    // the block's maximum, reference and sum
    m = block_max(lm::max_nan(nan ? NAN : own, outside), sh.red, larger_nan);
    const float block_ref = reference(m, r.c);
    pair.scale(lm::exp2_fast(lm::max_nan(ref - block_ref, -1000.f)));
    pair.add(lm::exp2_fast(lm::max_nan(fmaf(outside, r.c, -block_ref), -200.f)));
    pair = block_pair_sum(pair, sh);
    all_started();
    if (tid < parts) {
      SampleShared* o = each(tid);
      o->max[rank] = m;
      o->ref[rank] = block_ref;
      o->sum[rank] = make_float2(pair.hi, pair.lo);
    }
    // the block's candidate goes to the first block
    // (score: of a kept entry, -inf of others)
    const auto tell = [&](Pair mass, float block_m, auto score) {
      const float top = block_max(best.best, sh.red, larger), from = near(top);
      const bool in = best.at != -1 && best.best >= from;
      Part mine;
      mine.again = __syncthreads_or(in && best.second >= from) || top == INFINITY;
      mine.mass = make_float2(mass.hi, mass.lo);
      mine.at = -1;
      // the entries of this thread's batch that may be the largest
      int many = 0;
      double d = -INFINITY;
      int32_t at = -1;
      if (in) {
        const auto found = [&](int32_t j) {
          if (++many == 1) {
            at = j;
          } else {  // 64 bits decide
            if (many == 2) d = Row::exact(load_f32(x + at), r.noise[at], r.scale, block_m);
            join(d, at, Row::exact(load_f32(x + j), r.noise[j], r.scale, block_m), j);
          }
        };
        if (best.at < -1) {
          found(-2 - best.at);
        } else {
          uint32_t close = 0;
#pragma unroll
          for (int u = 0; u < kGroups; ++u) {
            const int32_t g = best.at + u * gr.step;
            if (g >= gr.n) break;
            const typename Groups<T>::Four f = gr.load(g);
            const float4 e = gr.random(g);
            close |= ((score(f.get(0), e.x) >= from ? 1u : 0u) | (score(f.get(1), e.y) >= from ? 2u : 0u) |
                      (score(f.get(2), e.z) >= from ? 4u : 0u) | (score(f.get(3), e.w) >= from ? 8u : 0u))
                     << (4 * u);
          }
          for (; close; close &= close - 1) {
            const int i = __ffs(close) - 1;
            found(gr.index(best.at + (i >> 2) * gr.step) + (i & 3));
          }
        }
      }
      const int one = __syncthreads_count(at >= 0);
      if (one > 1) {
        if (many == 1) d = Row::exact(load_f32(x + at), r.noise[at], r.scale, block_m);
        const int32_t which = block_join(d, at, sh);
        if (at == which) mine.at = at;
      } else {
        mine.at = at;
      }
      if (mine.at >= 0) {
        mine.x = load_f32(x + mine.at);
        mine.e = r.noise[mine.at];
        mine.score = score(mine.x, mine.e);
        lead->part[rank] = mine;
      } else if (one == 0 && tid == 0) {
        lead->part[rank] = mine;
      }
    };
    if (plain) tell(Pair{}, m, [&](float f, float e) { return fmaf(f, r.c, -log2_fast(e)); });
    sync();
    for (int p = 0; p < parts; ++p) m = lm::max_nan(m, sh.max[p]);
    if (ended(m)) return;
    const float row_ref = reference(m, r.c);
    // the row's sum relative to m c itself (asked for twice: two registers less in the last pass)
    const auto total = [&] {
      Pair t;
      for (int p = 0; p < parts; ++p) {
        Pair q{sh.sum[p].x, sh.sum[p].y};
        q.scale(lm::exp2_fast(fmaxf(sh.ref[p] - row_ref, -1000.f)));
        t.add(q);
      }
      t.scale(lm::exp2_fast(-fmaf(m, r.c, -row_ref)));
      return t;
    };
    r.m = m;
    general = !Row::near_zero(m, r.c);
    // the first block joins the candidates; false: the general way has to
    const auto decide = [&](const Part& listed, Pair kept) {
      Part q = listed;
      int again = 0;
      for (int p = 0; p < parts; ++p) {
        again |= sh.part[p].again;
        if (sh.part[p].at >= 0 && (q.at < 0 || sh.part[p].score > q.score)) q = sh.part[p];
      }
      if (again || q.at < 0) return false;
      const float from = near(q.score);
      int close = listed.at >= 0 && listed.score >= from;
      for (int p = 0; p < parts; ++p) close += sh.part[p].at >= 0 && sh.part[p].score >= from;
      if (close > 1) {
        double d = -INFINITY;
        int32_t at = -1;
        for (int p = -1; p < parts; ++p) {
          const Part& o = p < 0 ? listed : sh.part[p];
          if (o.at < 0 || o.score < from) continue;
          const int32_t was = at;
          join(d, at, Row::exact(o.x, o.e, r.scale, m), o.at);
          if (at != was) q = o;
        }
      }
      finish(q.at, kLn2 * (r.near_exponent(q.x) - log2f(fmaxf(kept.value(), 1.f))));
      return true;
    };
    if (plain) {
      if (rank != 0) return;
      Part none_listed;
      none_listed.at = -1;
      if (!general && decide(none_listed, total())) return;
      general = true;
    }
    if (!general) {
      // ---- top-p: the masses in bins by their logarithm, as shares of the total, tell near
      // which logits the border lies
      float min_x = min_p_logit(m, r.scale, min_p);
      float above_x = -FLT_MAX, list_x = -FLT_MAX;  // kept: x >= above_x; in question: list_x <= x < above_x
      bool ranked = top_p < 1.f;
      if (ranked) {
        for (int b = tid; b < 2 * kBins; b += kThreads) sh.bins.own[b] = 0;
        // entries below (1 - top_p) / V of the total cannot hold the border: with a bit to
        // spare, the lowest bin
        const float lowest = fmaxf(log2f((1.f - top_p) / (float)a.vocab) - 1.f, -60.f);
        const float per_bin = (float)(kBins - 1) / -lowest;  // bins per unit of log 2
        const float total_ref = fmaf(m, r.c, log2f(total().value()));
        const float low_x = fmaxf((total_ref + lowest) / r.c, -FLT_MAX);
        __syncthreads();
        const auto count = [&](float f) {
          const float v = fminf(fmaf(f, r.c, -total_ref), 0.f);
          // (a number from 2^23 on: its last bits are the bin, rounded)
          if (v >= lowest)
            atomicAdd(&sh.bins.own[2 * (__float_as_uint(fmaf(v, -per_bin, 8388608.f)) & (kBins - 1)) + (tid & 1)],
                      __float2uint_rn(lm::exp2_fast(v + 31.f)));
        };
        if (single >= low_x) count(single);
        sl.each_from(low_x, [&](const uint4& v, int32_t) {
#pragma unroll
          for (int i = 0; i < V::N; ++i) count(V::get(v, i));
        });
        sync();
        {
          // the blocks add up a stretch of the bins each, for all
          const int per = kBins / parts;
          for (int b = rank * per + tid; b < (rank + 1) * per; b += kThreads) {
            uint32_t sum = 0;
            for (int p = 0; p < parts; ++p) {
              const uint2 two = *reinterpret_cast<const uint2*>(each(p)->bins.own + 2 * b);
              sum += two.x + two.y;
            }
            for (int p = 0; p < parts; ++p) each(p)->bins.all[b] = sum;
          }
          sync();
        }
        {
          const uint32_t* bins = sh.bins.all + tid * (kBins / kThreads);
          constexpr int kEach = kBins / kThreads;
          uint32_t b[kEach], sum = 0;
#pragma unroll
          for (int i = 0; i < kEach; ++i) sum += b[i] = bins[i];
          uint32_t upto = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t p = __shfl_up_sync(0xffffffffu, upto, o);
            if ((tid & 31) >= o) upto += p;
          }
          if ((tid & 31) == 31) sh.warp_count[tid >> 5] = upto;
          if (tid == 0) sh.border[0] = sh.border[1] = kBins;
          __syncthreads();
          upto -= sum;
          for (int w = 0; w < (tid >> 5); ++w) upto += sh.warp_count[w];
          // a share's rounding is half a unit of 2^-31 at most, the sums' a few of 2^-24
          const float slack = 0.5f * (float)a.vocab + 0x1p10f, want = top_p * 0x1p31f;
          const uint32_t want0 = (uint32_t)fmaxf(want - slack, 0.f), want1 = (uint32_t)fminf(want + slack, 4.2e9f);
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            upto += b[i];
            if (upto >= want0) atomicMin(&sh.border[0], tid * kEach + i);
            if (upto >= want1) atomicMin(&sh.border[1], tid * kEach + i);
          }
        }
        sync();  // the list comes where the bins are
        // the bins' edges, a little apart from them: what lies near an edge is in question
        const float b0 = (float)sh.border[0] - 0.5f, b1 = (float)sh.border[1] + 0.5f, off = 0x1p-18f * (fabsf(total_ref) + 64.f);
        above_x = fmaxf(fminf((total_ref - b0 / per_bin + off) / r.c, FLT_MAX), -FLT_MAX);
        list_x = sh.border[1] >= kBins ? -FLT_MAX : fmaxf((total_ref - b1 / per_bin - off) / r.c, -FLT_MAX);
        if (min_x >= above_x) ranked = false;  // min-p ends before
      }
      if (!ranked) above_x = list_x = min_x;

      // ---- the last pass
      Pair mass;
      float sum = 0.f;
      const float low = list_x;
      const auto score = [&](float f, float e) { return f >= above_x ? r.near_exponent(f) - log2_fast(e) : -INFINITY; };
      if (gr.single >= 0) {
        outside = load_f32(x + gr.single);
        if (outside >= above_x) {
          sum = lm::exp2_fast(r.near_exponent(outside));
          best.add(score(outside, r.noise[gr.single]), -2 - gr.single);
        } else if (outside >= low) {
          put(outside, gr.single);
        }
      }
#pragma unroll 1
      for (int32_t g0 = gr.at0; g0 < gr.n; g0 += kGroups * gr.step) {
        typename Groups<T>::Four f[kGroups];
        float4 e[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; ++u) f[u] = g0 + u * gr.step < gr.n ? gr.load(g0 + u * gr.step) : gr.none();
        uint32_t asked = 0;  // entries in question
        float most = -INFINITY;
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const float m4 = fmaxf(fmaxf(f[u].get(0), f[u].get(1)), fmaxf(f[u].get(2), f[u].get(3)));
          e[u] = m4 >= above_x ? gr.random(g0 + u * gr.step) : make_float4(1.f, 1.f, 1.f, 1.f);
          most = fmaxf(most, m4);
        }
        if (most < low) continue;
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const float n4[4] = {e[u].x, e[u].y, e[u].z, e[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = r.near_exponent(f[u].get(i));
            const bool in = f[u].get(i) >= above_x;
            sum += in ? lm::exp2_fast(w) : 0.f;
            top = fmaxf(top, in ? w - log2_fast(n4[i]) : -INFINITY);
            asked |= (!in && f[u].get(i) >= low ? 1u : 0u) << (4 * u + i);
          }
        }
        best.add(top, g0);
        mass.add(sum);
        sum = 0.f;
        while (asked) {
          const int i = __ffs(asked) - 1;
          asked &= asked - 1;
          const int32_t j = gr.index(g0 + (i >> 2) * gr.step) + (i & 3);
          put(load_f32(x + j), j);
        }
      }
      mass.add(sum);
      mass = block_pair_sum(mass, sh);
      tell(mass, m, score);
      sync();
      if (rank != 0) return;
      Pair kept;
      for (int p = 0; p < parts; ++p) kept.add(Pair{sh.part[p].mass.x, sh.part[p].mass.y});
      Part listed;
      listed.at = -1;
      general = false;
      if (top_p < 1.f) {
        // what is kept so far lies below top_p's share, so none of it is too much: the bins are
        // as exact as fp32 is at the maximum, and min-p may have ended in a gap at the border
        Pair rest;
        const Pair all = total();
        const float share = top_p * all.hi;
        rest.add(share);
        rest.add(-kept.hi);
        rest.add(fmaf(top_p, all.hi, -share));
        rest.add(fmaf(top_p, all.lo, -kept.lo));
        const unsigned long long want = whole_mass(rest);
        const int n = sh.nlist;
        general = n > kList || want == 0;
        if (ranked && !general) {
          // the border lies in the list, or the list goes to the row's end
          unsigned long long cut = 0;
          if (list_mass(sh, n, 0, r) >= want)
            cut = list_border(sh, n, 0, want, r, list_x, fminf(above_x, m), a.vocab);
          else
            general = list_x > -FLT_MAX;
          if (!general) {
            const Listed t = take_list(sh, n, cut, min_x, r);
            listed = t.best;
            kept.add((float)t.mass * 0x1p-38f);
          }
        }
      }
      if (!general && decide(listed, kept)) return;
      general = true;
    }
    if (rank != 0) return;
  }
  // the general way: the first block alone
  r.m = m;
  r.half = fabsf(m) >= 0x1p100f && r.scale < 0.5f ? 0.5f : 1.f;
  r.minus_hm = -r.half * m;
  r.c = r.scale * kLog2e / r.half;
  r.shift = min(40, 31 + __clz(a.vocab));  // V masses add up below 2^63
  __syncthreads();
  sample_generic<T>(sh, a, x, r, row, top_k, top_p, min_p);
}

}  // namespace
}  // namespace dobb

using namespace dobb;

extern "C" dobb_status dobb_sample(const void* logits, dobb_dtype logits_dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                   const float* noise, int64_t noise_stride, float scale, int top_k, float top_p, float min_p,
                                   const float* scales, const int32_t* top_ks, const float* top_ps, const float* min_ps,
                                   int32_t* tokens, float* logp, void* stream) {
  if (lm::bad_dtype(logits_dtype)) return fail(DOBB_ERR_INVALID_ARG, "logits dtype must be DOBB_F32 or DOBB_BF16");
  if (rows < 0) return fail(DOBB_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
  if (rows > INT32_MAX) return fail(DOBB_ERR_UNSUPPORTED, "too many rows (%lld)", (long long)rows);
  if (vocab < 1 || vocab > INT32_MAX - 4096)
    return fail(DOBB_ERR_INVALID_ARG, "vocab must lie in [1, 2^31 - 4096) (got %lld)", (long long)vocab);
  if (rows > 1 && (row_stride < vocab || noise_stride < vocab))
    return fail(DOBB_ERR_INVALID_ARG, "a row stride is below vocab %lld", (long long)vocab);
  if (rows > 1 && (row_stride > INT64_MAX / 8 / rows || noise_stride > INT64_MAX / 8 / rows))
    return fail(DOBB_ERR_UNSUPPORTED, "rows times the row stride is too large");
  if (!scales && !(scale > 0.f && scale <= 0x1p127f))
    return fail(DOBB_ERR_INVALID_ARG, "scale must lie in (0, 2^127] (got %g)", scale);
  if (!top_ks && top_k < 0) return fail(DOBB_ERR_INVALID_ARG, "top_k must be >= 0 (got %d)", top_k);
  if (!top_ps && !(top_p > 0.f && top_p <= 1.f)) return fail(DOBB_ERR_INVALID_ARG, "top_p must lie in (0, 1] (got %g)", top_p);
  if (!min_ps && !(min_p >= 0.f && min_p <= 1.f)) return fail(DOBB_ERR_INVALID_ARG, "min_p must lie in [0, 1] (got %g)", min_p);
  if (rows == 0) return DOBB_OK;
  if (!logits || !noise || !tokens || !logp) return fail(DOBB_ERR_INVALID_ARG, "logits, noise, tokens and logp must be non-NULL");
  if (lm::misaligned(logits, lm::dtype_bytes(logits_dtype)) || lm::misaligned(noise, 4) || lm::misaligned(tokens, 4) ||
      lm::misaligned(logp, 4) || lm::misaligned(scales, 4) || lm::misaligned(top_ks, 4) || lm::misaligned(top_ps, 4) ||
      lm::misaligned(min_ps, 4))
    return fail(DOBB_ERR_INVALID_ARG, "a tensor is not aligned to its element size");
  lm::Extents ext;
  ext.read("logits", logits, rows, vocab, row_stride, logits_dtype);
  ext.read("noise", noise, rows, vocab, noise_stride, DOBB_F32);
  ext.read("scale", scales, 1, rows, rows, DOBB_F32);
  ext.read("top_k", top_ks, 1, rows, rows, DOBB_F32);
  ext.read("top_p", top_ps, 1, rows, rows, DOBB_F32);
  ext.read("min_p", min_ps, 1, rows, rows, DOBB_F32);
  ext.write("tokens", tokens, 1, rows, rows, DOBB_F32);
  ext.write("logp", logp, 1, rows, rows, DOBB_F32);
  const dobb_status st = ext.check();
  if (st != DOBB_OK) return st;
  // blocks per row: as many as fill the GPU once, 4096 entries each at least
  int parts = 1;
  while (parts < kMaxParts && rows * parts * 2 <= 4 * kSms && vocab / (parts * 2) >= 4096) parts *= 2;
  const int64_t most = ((int64_t)1 << 30) / parts;
  cudaError_t e = cudaSuccess;
  for (int64_t r0 = 0; r0 < rows && e == cudaSuccess; r0 += most) {
    const int64_t nr = std::min<int64_t>(rows - r0, most);
    const auto from = [&](auto* p) { return p ? p + r0 : p; };
    const SampleArgs a{static_cast<const char*>(logits) + r0 * row_stride * (int64_t)lm::dtype_bytes(logits_dtype),
                       nr, row_stride, (int32_t)vocab, noise + r0 * noise_stride, noise_stride,
                       from(scales), from(top_ks), from(top_ps), from(min_ps), scale, top_k, top_p, min_p, tokens + r0, logp + r0};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(nr * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)parts, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = logits_dtype == DOBB_F32 ? cudaLaunchKernelEx(&cfg, sample_rows<float>, a)
                                 : cudaLaunchKernelEx(&cfg, sample_rows<__nv_bfloat16>, a);
  }
  if (e != cudaSuccess) return fail(DOBB_ERR_CUDA, "sampling launch: %s", cudaGetErrorString(e));
  return DOBB_OK;
}
