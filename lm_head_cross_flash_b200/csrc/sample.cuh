// sample.cuh — one token per row of logits: temperature, top-k, top-p and
// min-p from given uniform numbers, and the token's log-probability.
//
// Order.  The live logits of a row (neither -inf nor NaN) are ranked by value,
// equal ones by index.  As one unsigned number, "value key, then inverted
// index", ranks are strict, and each of top-k, top-p, min-p and the draw keeps
// or ends a prefix of the ranking.  So all of them ask one question: which is
// the first rank at which a running count or a running mass reaches a target?
//
// Mass.  w = exp((l - max) / T) in fixed point, `bits` binary places (45 for a
// vocabulary up to 2^18), so that sums are exact, do not depend on their
// order, and a target is met at the same token on every run.  exp is computed
// in fp64 (Tang's table method: 2^(j/32) times a polynomial on |r| <= 1/64),
// since a draw among 2^18 tokens is decided by differences far below fp32.
//
// Two ways.  A cluster of CTAs takes a row.  One pass over memory gives the
// maximum, sums of fp32 exponentials (behind logp, and the total mass to a
// known error) and the largest logit of every segment of 512.
//  * List.  Nearly always the kept ranks are few.  The segments' maxima say
//    below which value enough ranks, or enough mass, must lie; only segments
//    that reach it are read again, and the candidates are sorted by the
//    cluster's first CTA and summed exactly.  The result stands if the
//    total's error leaves no doubt about it.
//  * Search.  Otherwise (a flat row, many equal logits, a doubt) one pass
//    counts the live logits in 2,048 bins of equal width below the maximum and
//    sums their weights by bin, exactly (three 32-bit digits of 15 bits each
//    by shared-memory atomics: 0.16 cycles a logit and SM for one or two of
//    them, 0.7 to 2 for one 64-bit atomic).  The bin in which the target is
//    reached is collected and sorted; one that holds more logits than the
//    list takes is binned again, over its values or, where those are all
//    equal, over its indices.  A step that does not halve it is followed by a
//    bisection, so the search ends for every input.
// Measured: one row of 73,440 fp32 logits 10.6 us by list and 59 by search; 256
// rows of 262,144 bf16 46 us greedy with logp (20 us of DRAM; 12 instructions a
// logit), 62 us with top-k 50, 262 us with top-p 0.95 where a fifth of the rows
// is flat, 652 us where all are, but for some likely tokens, 752 without those.
// Many rows run as two launches: the list with few CTAs a row (its fixed
// costs, mostly waits, are paid by fewer CTAs), and the search with more of
// them (eight, fewer where many rows may be left) for the rows that are left,
// so that one flat row does not hold up the batch.
#pragma once

#include <cooperative_groups.h>

#include "row_ops.cuh"

namespace cce {

constexpr int SA_THREADS = 512;
constexpr int SA_WARPS = SA_THREADS / 32;
constexpr int SA_BINS = 2048;
constexpr int SA_CAP = 2048;  // candidates of one list
constexpr int SA_MAX_CLUSTER = 8;
constexpr int SA_SEG = 512;        // logits that a warp reads at once: one segment
constexpr int SA_MAX_SEGS = 1024;  // segments (or groups of them) of one CTA
constexpr int SA_OPEN = 128;       // segments that the list opens if their mass is not enough
constexpr int SA_COUNT_SLICE = 16384; // logits of a CTA up to which the list counts them all
constexpr int SA_RING = 64 * 1024; // copies in flight during the first pass
constexpr int SA_FLUSH = 65536;    // logits that 15-bit digits can be summed over in 32 bits
constexpr int SA_UNDECIDED = -2;   // token of a row that the first launch leaves to the second,
constexpr int SA_CLAIMED = -3;     // and of one that a cluster of the second works on
enum : int { SA_BOTH = 0, SA_LIST_ONLY = 1, SA_SEARCH_ONLY = 2 };  // what a launch does
static_assert(SA_CAP == 4 * SA_THREADS && SA_BINS == 4 * SA_THREADS, "four entries per thread");

// Relative error of the pass's sums of exponentials: 2^-22 of ex2.approx (once
// a logit and once in each of two joins, of warps and of CTAs), the roundings
// of the arguments and of c (3 2^-24 ln 2 times the exponent, at most 50 where
// it counts) and fp32 sums of 8 terms.  Together below 8e-6, however often a
// larger maximum turns up: those factors are fp64.
constexpr double SA_SUM_ERROR = 0x1p-16;

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int B, V;
  int slice;    // logits per CTA, a multiple of SA_SEG
  int seg_mul;  // segments that share an entry of segs[]
  int bits;     // binary places of a weight
  const float* temperature;  // the next four may be null: 1, off, off, off
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* logp;  // may be null
};

using u64 = unsigned long long;

__device__ __forceinline__ uint32_t value_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 ranks with +0
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ u64 rank_of(float l, int idx) {
  return (u64(value_key(l)) << 32) | (0xFFFFFFFFu - uint32_t(idx));
}
__device__ __forceinline__ float rank_value(u64 c) { return key_value(uint32_t(c >> 32)); }
__device__ __forceinline__ int rank_index(u64 c) { return int(0xFFFFFFFFu - uint32_t(c)); }

// What the CTAs of a cluster tell one another after a pass.
struct SaPart {
  u64 hi, lo;  // largest and smallest rank
  u64 mass;
};
// The same after the first pass: the largest rank and the sums of
// exp(l - m) and exp((l - m) / T) over the logits below its value m.
struct SaFirst {
  u64 hi;
  double tail, z;
  float least;  // of the segments' maxima
  int n;        // instances of m, which the sums leave out
};

struct SaShared {
  union {
    uint8_t ring[SA_RING];  // first pass: each thread's own copies
    uint16_t opened[SA_RING / 2];  // list: segments to read again
    struct {
      uint32_t tot[SA_BINS];  // search: the cluster's counts and masses
      u64 mass[SA_BINS];
      uint32_t hist[SA_BINS];  // and this CTA's: counts, digits of the masses
      uint32_t dig[3][SA_BINS];
    };
  };
  uint32_t open[SA_BINS];  // first CTA: counts of the segments' maxima
  u64 list[SA_CAP];
  uint32_t segs[SA_MAX_SEGS];  // value keys of the segments' largest logits, 0: none
  double pow2[32];             // 2^(j/32)
  SaPart parts[2][SA_MAX_CLUSTER];
  SaPart warp_part[SA_WARPS];
  SaFirst firsts[SA_MAX_CLUSTER];
  SaFirst warp_first[SA_WARPS];
  u64 warp_sum[2][SA_WARPS];
  u64 res_rank, res_cum, end;
  u64 base;      // the measure above the bin
  uint32_t n_in; // logits in it
  int bin;
  int n_list, n_opened;
  int done;  // the list gave the answer
  int row;   // the search's, and what claim_row's threads tell one another
  int found[SA_WARPS], claimed;
};

template <typename T>
struct SaRaw {  // eight logits
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void raw_values(const SaRaw<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t u[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w,
                           r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
  } else {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

// 2^(j/32), rounded to nearest.
__device__ const double SA_POW2[32] = {
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0};

template <typename T>
class Sampler {
 public:
  // all_run: every CTA of the cluster is known to run already; otherwise the
  // kernel has arrived on the cluster's barrier and the first pass waits.
  __device__ Sampler(const SampleArgs& a, SaShared& s, int row, bool all_run)
      : a_(a), s_(s), cl_(cooperative_groups::this_cluster()), all_run_(all_run) {
    C_ = int(cl_.num_blocks());
    me_ = int(cl_.block_rank());
    row_ = row;
    g_ = static_cast<const T*>(a.logits) + int64_t(row_) * a.ld;
    off_ = int((reinterpret_cast<uintptr_t>(g_) & 15) / sizeof(T));
    s0_ = int(min(int64_t(a.V) + off_, int64_t(me_) * a.slice));
    s1_ = int(min(int64_t(a.V) + off_, int64_t(s0_) + a.slice));
  }

  template <int MODE>
  __device__ void run();

 private:
  const SampleArgs& a_;
  SaShared& s_;
  cooperative_groups::cluster_group cl_;
  // Positions count from the 16-byte boundary at or before the row's first
  // logit, off_ logits ahead of it, so that pieces of eight are whole 16-byte
  // loads wherever the row begins.  The slice is [s0_, s1_).
  int C_, me_, row_, off_, s0_, s1_;
  const bool all_run_;
  const T* g_;
  int turn_ = 0;      // which half of `parts` the next exchange uses
  float max_ = 0.f;
  double c_ = 0.0;    // log2(e) / T
  float bin_scale_ = 0.f;
  bool level0_ = false;  // tot and mass hold the bins below the row's maximum

  // ------------------------------------------------------------- passes --
  __device__ SaRaw<T> fetch(int c) const {
    if (c < off_ || c + 8 > s1_) return fetch_ragged(g_, c - off_, s1_ - off_);
    SaRaw<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
      r.v[i] = __ldg(reinterpret_cast<const uint4*>(g_ - off_ + c) + i);
    return r;
  }
  // From index c on, -inf outside [0, end).
  __device__ static __noinline__ SaRaw<T> fetch_ragged(const T* g, int c, int end) {
    auto in = [&](int i) { return i >= 0 && i < end; };
    SaRaw<T> r;
    uint32_t w[sizeof(T) * 2];
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * 2); ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = in(c + i) ? __float_as_uint(g[c + i]) : 0xFF800000u;
      } else {
        const uint32_t lo = in(c + 2 * i) ? __bfloat16_as_ushort(g[c + 2 * i]) : 0xFF80u;
        const uint32_t hi = in(c + 2 * i + 1) ? __bfloat16_as_ushort(g[c + 2 * i + 1]) : 0xFF80u;
        w[i] = lo | (hi << 16);
      }
    }
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
      r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    return r;
  }
  __device__ int n_segs() const { return (s1_ - s0_ + SA_SEG - 1) / SA_SEG; }
  // Calls f(values, first index) on every piece of eight logits in the
  // segments [from, to) whose largest logit's key passes want().  One piece is
  // loaded ahead; not unrolled (the callers' code for eight logits is long,
  // and four copies of it did not fit the instruction cache: 16 % of the
  // search's warp cycles).
  template <typename W, typename F>
  __device__ void pass(int from, int to, W want, F f) const {
    const int lane8 = int(threadIdx.x & 31) * 8;
    auto skip = [&](int i) {  // the first wanted segment from i on
      for (; i < to; i += SA_WARPS) {
        const uint32_t key = s_.segs[a_.seg_mul == 1 ? i : i / a_.seg_mul];
        if (key != 0 && want(key)) break;
      }
      return i;
    };
    int i = skip(from + int(threadIdx.x >> 5)), k = 0;
    if (i >= to) return;
    int c = s0_ + i * SA_SEG + lane8;
    SaRaw<T> r = fetch(c);
#pragma unroll 1
    while (i < to) {
      if (++k == NB) {
        k = 0;
        i = skip(i + SA_WARPS);
      }
      const int next = s0_ + i * SA_SEG + k * 256 + lane8;
      SaRaw<T> ahead = r;
      if (i < to) ahead = fetch(next);
      float v[8];
      raw_values<T>(r, v);
      f(v, c - off_);
      c = next;
      r = ahead;
    }
  }
  template <typename F>
  __device__ void pass(F f) const {
    pass(0, n_segs(), [](uint32_t) { return true; }, f);
  }
  // The logits of a lane's piece that hit() takes, as bits (c: the first one's
  // index).
  template <typename H>
  __device__ uint32_t hits(const float (&v)[8], int c, H hit) const {
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mask |= uint32_t(v[j] > -INFINITY && hit(v[j], c + j)) << j;
    return mask;
  }
  // Calls f with the rank of each of them.
  template <typename F>
  __device__ static void each(uint32_t mask, const float (&v)[8], int c, F f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (mask >> j & 1) f(rank_of(v[j], c + j));
  }

  __device__ float below(float l) const { return l == max_ ? 0.f : max_ - l; }
  __device__ int bin_of(float l) const { return bin_below(max_, l, bin_scale_); }

  // 2^(x + places), |x| up to 900: with k = round(32 x), r = x - k/32,
  // 2^x = 2^(k div 32) 2^((k mod 32)/32) 2^r, and 2^r by its series to r^5
  // (the next term is below 2.3e-15).
  __device__ double exp2_fp64(double x, int places = 0) const {
    constexpr double MAGIC = 6755399441055744.0;  // 1.5 * 2^52
    const double kd = fma(x, 32.0, MAGIC);
    const int k = __double2loint(kd);
    const double r = fma(kd - MAGIC, -1.0 / 32.0, x);
    constexpr double L = 0.693147180559945309417;  // ln 2
    double p = fma(r, L * L * L * L * L / 120.0, L * L * L * L / 24.0);
    p = fma(r, p, L * L * L / 6.0);
    p = fma(r, p, L * L / 2.0);
    p = fma(r, p, L);
    const double t = s_.pow2[k & 31];
    const double ts = __hiloint2double(__double2hiint(t) + ((k >> 5) + places) * (1 << 20),
                                       __double2loint(t));
    return fma(ts, r * p, ts);
  }
  // round(2^bits * 2^x) for x <= 0.  The addition leaves the integer in the low
  // bits of the sum.
  __device__ u64 weight_log2(double x) const {
    if (!(x > -50.0)) return 0;
    const double w = exp2_fp64(x, a_.bits) + 4503599627370496.0;  // + 2^52
    return u64(__double_as_longlong(w)) & 0x000FFFFFFFFFFFFFull;
  }
  // l - max, exact (infinities are equal).
  __device__ double diff(float l) const { return l == max_ ? 0.0 : double(l) - double(max_); }
  __device__ u64 weight(float l) const {
    if (l == max_) return u64(1) << a_.bits;
    return weight_log2(diff(l) * c_);
  }

  // ------------------------------------------------- block and cluster --
  // A barrier of the cluster (of the block where that is all of it).
  __device__ void meet() {
    if (C_ == 1) __syncthreads();
    else cl_.sync();
  }
  __device__ static SaPart nothing() { return SaPart{0, ~u64(0), 0}; }
  __device__ static SaPart merge_lanes(SaPart p, int o) {
    p.hi = max(p.hi, __shfl_xor_sync(0xffffffffu, p.hi, o));
    p.lo = min(p.lo, __shfl_xor_sync(0xffffffffu, p.lo, o));
    p.mass += __shfl_xor_sync(0xffffffffu, p.mass, o);
    return p;
  }
  // The threads' parts of all CTAs, merged; every thread of the cluster gets
  // the result.  Also a barrier of the cluster.
  __device__ SaPart exchange(SaPart p) {
    const int lane = threadIdx.x & 31;
    for (int o = 16; o > 0; o >>= 1) p = merge_lanes(p, o);
    if (lane == 0) s_.warp_part[threadIdx.x >> 5] = p;
    __syncthreads();
    if (threadIdx.x < 32) {
      p = s_.warp_part[lane & (SA_WARPS - 1)];
      for (int o = SA_WARPS / 2; o > 0; o >>= 1) p = merge_lanes(p, o);
      if (lane < C_) *cl_.map_shared_rank(&s_.parts[turn_][me_], lane) = p;
    }
    meet();
    p = s_.parts[turn_][lane & (C_ - 1)];
    for (int o = C_ / 2; o > 0; o >>= 1) p = merge_lanes(p, o);
    turn_ ^= 1;
    return p;
  }
  // Inclusive prefix sum of x over the threads of the block.
  __device__ u64 scan(u64 x, u64* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    for (int i = 0; i < warp; ++i) x += sums[i];
    return x;
  }
  // Counts (and, by_mass, weights) of the logits by bin, of the whole cluster:
  // bin(value, index) < 0 leaves a logit out, as it does all of a segment
  // whose maximum's key want() refuses.  Ends with a barrier of the cluster.
  template <typename W, typename F>
  __device__ void bin_up(bool by_mass, W want, F bin) {
    auto clear = [&](bool counts) {
      for (int i = threadIdx.x; i < SA_BINS; i += SA_THREADS) {
        if (counts) s_.hist[i] = 0;
        if (by_mass) s_.dig[0][i] = s_.dig[1][i] = s_.dig[2][i] = 0;
      }
    };
    auto digits = [&](int r, int b) -> u64 {
      const uint32_t(*d)[SA_BINS] = cl_.map_shared_rank(s_.dig, r);
      return u64(d[0][b]) + (u64(d[1][b]) << 15) + (u64(d[2][b]) << 30);
    };
    clear(true);
    const int n = SA_BINS / C_, b0 = me_ * n;  // the bins that this CTA adds up
    u64 sum[SA_BINS / SA_THREADS] = {};
    const int end = a_.slice / SA_SEG;  // the same number of rounds in every CTA
    for (int from = 0; from < end; from += SA_FLUSH / SA_SEG) {
      __syncthreads();
      pass(from, min(n_segs(), from + SA_FLUSH / SA_SEG), want, [&](const float (&v)[8], int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!(v[j] > -INFINITY)) continue;
          const int b = bin(v[j], c + j);
          if (b < 0) continue;
          atomicAdd(&s_.hist[b], 1u);
          if (!by_mass) continue;
          const u64 w = weight(v[j]);
          if (w == 0) continue;
          atomicAdd(&s_.dig[0][b], uint32_t(w) & 0x7FFFu);
          atomicAdd(&s_.dig[1][b], uint32_t(w >> 15) & 0x7FFFu);
          atomicAdd(&s_.dig[2][b], uint32_t(w >> 30));
        }
      });
      if (!by_mass) continue;
      meet();
      for (int k = 0, i = threadIdx.x; i < n; ++k, i += SA_THREADS) {
        u64 x = 0;
        for (int r = 0; r < C_; ++r) x += digits(r, b0 + i);
#pragma unroll
        for (int q = 0; q < SA_BINS / SA_THREADS; ++q)
          if (q == k) sum[q] += x;
      }
      if (from + SA_FLUSH / SA_SEG < end) {
        meet();
        clear(false);
      }
    }
    if (!by_mass) meet();
    for (int k = 0, i = threadIdx.x; i < n; ++k, i += SA_THREADS) {
      uint32_t x = 0;
      u64 y = 0;
      for (int r = 0; r < C_; ++r) x += *cl_.map_shared_rank(&s_.hist[b0 + i], r);
#pragma unroll
      for (int q = 0; q < SA_BINS / SA_THREADS; ++q)
        if (q == k) y = sum[q];
      for (int r = 0; r < C_; ++r) {
        *cl_.map_shared_rank(&s_.tot[b0 + i], r) = x;
        *cl_.map_shared_rank(&s_.mass[b0 + i], r) = y;
      }
    }
    meet();
  }

  __device__ void bin_level0() {
    bin_up(true, [](uint32_t) { return true; }, [&](float l, int) { return bin_of(l); });
    level0_ = true;
  }

  // The bin in which the running count or mass reaches the target (the last
  // one if none does): bin, base (above it), n_in.
  __device__ void locate(bool by_mass, u64 target) {
    u64 x[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = threadIdx.x * 4 + i;
      x[i] = sum += by_mass ? s_.mass[b] : s_.tot[b];
    }
    __syncthreads();
    const u64 before = scan(sum, s_.warp_sum[0]) - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = threadIdx.x * 4 + i;
      const u64 prev = before + (i ? x[i - 1] : 0);
      if ((before + x[i] >= target || b == SA_BINS - 1) && (prev < target || b == 0)) {
        s_.bin = b;
        s_.base = prev;
        s_.n_in = s_.tot[b];
      }
    }
    __syncthreads();
  }

  // A warp's candidates go to the first CTA's list, with one addition to its
  // length (with one for each candidate, 215 flat rows of 145,242 bf16 logits,
  // whose bins hold many equal ones, took 636 us instead of 346).
  __device__ void append(uint32_t mask, const float (&v)[8], int c) {
    if (__ballot_sync(0xffffffffu, mask != 0) == 0) return;
    const int lane = threadIdx.x & 31, n = __popc(mask);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    int at = 0;
    if (lane == 31) at = atomicAdd(cl_.map_shared_rank(&s_.n_list, 0), upto);
    at = __shfl_sync(0xffffffffu, at, 31) + upto - n;
    u64* list = cl_.map_shared_rank(s_.list, 0);
    each(mask, v, c, [&](u64 r) {
      if (at < SA_CAP) list[at] = r;
      ++at;
    });
  }
  // First CTA: sorts the list from the highest rank down; its length.  Thread
  // t gets the ranks 4t to 4t + 3.
  __device__ int sort_list(u64 (&r)[4]) {
    const int n = min(s_.n_list, SA_CAP), e0 = threadIdx.x * 4;
    if (n <= SA_THREADS) {
      // Few: an element's place is the number of those above it.  The threads
      // are spread over elements and parts of the list (a network over 128 took
      // 7,000 cycles, over 2,048 29,000).
      int np = 32;
      while (np < n) np *= 2;
      const int parts = SA_THREADS / np, e = threadIdx.x & (np - 1), part = threadIdx.x / np;
      for (int i = threadIdx.x; i < np; i += SA_THREADS) {
        s_.open[i] = 0;
        if (i >= n) s_.list[i] = 0;
      }
      __syncthreads();
      if (threadIdx.x == 0) s_.n_list = 0;  // for the next list
      const u64 x = s_.list[e];
      const int len = (n + parts - 1) / parts, to = min(n, (part + 1) * len);
      int above = 0;
#pragma unroll 4
      for (int j = part * len; j < to; ++j) above += s_.list[j] > x;
      if (e < n) atomicAdd(&s_.open[e], uint32_t(above));
      __syncthreads();
      if (part == 0 && e < n) s_.list[SA_CAP / 2 + s_.open[e]] = x;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = e0 + i < n ? s_.list[SA_CAP / 2 + e0 + i] : 0;
        if (e0 + i < n) s_.list[e0 + i] = r[i];
      }
      __syncthreads();
      return n;
    }
    // A bitonic network: strides below 4 stay in a thread, those below 128 in a
    // warp (shuffles), the others go through the list's memory.
    int len = 128;
    while (len < n) len *= 2;
    const bool in = e0 < len;  // the same for a whole warp
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = e0 + i < n ? s_.list[e0 + i] : 0;
    __syncthreads();
    if (threadIdx.x == 0) s_.n_list = 0;
    auto order = [](u64& x, u64& y, bool down) {
      const u64 a = x, b = y;
      const bool swap = (a < b) == down;
      x = swap ? b : a;
      y = swap ? a : b;
    };
    for (int k = 2; k <= len; k *= 2) {
      const bool down = (e0 & k) == 0;
      for (int j = k / 2; j >= 128; j /= 2) {
        if (in) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s_.list[e0 + i] = r[i];
        }
        __syncthreads();
        if (in) {
          const bool most = down == ((e0 & j) == 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const u64 o = s_.list[(e0 ^ j) + i];
            r[i] = (o > r[i]) == most ? o : r[i];
          }
        }
        __syncthreads();
      }
      if (!in) continue;
#pragma unroll
      for (int j = 64; j >= 4; j /= 2) {
        if (j >= k) continue;
        const bool most = down == ((e0 & j) == 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u64 o = __shfl_xor_sync(0xffffffffu, r[i], j / 4);
          r[i] = (o > r[i]) == most ? o : r[i];
        }
      }
      if (k > 2) {
        order(r[0], r[2], down);
        order(r[1], r[3], down);
      }
      order(r[0], r[1], down);
      order(r[2], r[3], ((e0 + 2) & k) == 0);
    }
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s_.list[e0 + i] = r[i];
    }
    __syncthreads();
    return n;
  }
  // First CTA: the masses up to and including each of this thread's sorted
  // candidates, above `base`.  Returns the mass before the first.
  __device__ u64 running_mass(int n, u64 base, const u64 (&r)[4], u64 (&cum)[4]) {
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum += int(threadIdx.x) * 4 + i < n ? weight(rank_value(r[i])) : 0;
      cum[i] = sum;
    }
    const u64 before = base + scan(sum, s_.warp_sum[0]) - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) cum[i] += before;
    return before;
  }
  // First CTA: the first rank whose running mass reaches the target (the last
  // one if none does), and that mass; both into res_*.
  __device__ void pick(int n, u64 before, const u64 (&r)[4], const u64 (&cum)[4], u64 target) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = threadIdx.x * 4 + i;
      const u64 prev = i ? cum[i - 1] : before;
      if (k < n && (cum[i] >= target || k == n - 1) && (prev < target || k == 0)) {
        s_.res_rank = r[i];
        s_.res_cum = cum[i];
      }
    }
    __syncthreads();
  }
  // The first CTA's result to all; a barrier of the cluster.
  __device__ void share_result() {
    __syncthreads();
    if (me_ == 0 && int(threadIdx.x) < C_ && threadIdx.x > 0) {
      *cl_.map_shared_rank(&s_.res_rank, threadIdx.x) = s_.res_rank;
      *cl_.map_shared_rank(&s_.res_cum, threadIdx.x) = s_.res_cum;
    }
    meet();
  }

  // Bins of equal width below the value vt, the last one open.
  __device__ static int bin_below(float vt, float l, float scale) {
    return l == vt ? 0 : int(fminf((vt - l) * scale, float(SA_BINS - 1)));
  }
  __device__ static float scale_for(float span) {
    const float s = span > 0.f ? float(SA_BINS - 1) / span : 1.f;
    return s < 1e30f ? s : 1e30f;
  }

  // A ring of copies (cp.async), each thread's own, so that the loads of the
  // next DEPTH segments are under way while one is worked on.  A segment is
  // NB pieces of 256: eight logits a lane.
  static constexpr int NB = SA_SEG / 256;
  static constexpr int DEPTH = SA_RING / (SA_THREADS * 8 * int(sizeof(T)) * NB);
  static_assert(DEPTH >= 2 && (DEPTH & (DEPTH - 1)) == 0, "a power of two");
  __device__ uint4* slot(int p) const {
    return reinterpret_cast<uint4*>(s_.ring) + threadIdx.x +
           (p & (DEPTH - 1)) * (NB * int(sizeof(T) / 2) * SA_THREADS);
  }
  // The warp's p-th segment of the slice, on its way.
  __device__ void copy_in(int p) const {
    constexpr int PL = sizeof(T) / 2, STEP = SA_WARPS * SA_SEG;
    const int c = s0_ + int(threadIdx.x >> 5) * SA_SEG + p * STEP, lane8 = int(threadIdx.x & 31) * 8;
    if (c >= off_ && c + SA_SEG <= s1_) {
      const uint32_t to = smem_u32(slot(p));
      const uint4* from = reinterpret_cast<const uint4*>(g_ - off_ + c + lane8);
#pragma unroll
      for (int i = 0; i < NB * PL; ++i)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(
                         to + i * SA_THREADS * 16),
                     "l"(from + (i / PL) * 32 * PL + i % PL)
                     : "memory");
    } else if (c < s1_) {
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const SaRaw<T> r = fetch(c + k * 256 + lane8);
#pragma unroll
        for (int i = 0; i < PL; ++i) slot(p)[(k * PL + i) * SA_THREADS] = r.v[i];
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  template <bool TAIL, bool Z>
  __device__ SaFirst first_pass(float cz);
  // 2^(c m - h): what a weight of 1 is in sums that are relative to h, or with
  // sign -1 its inverse.  The difference is h's rounding error, exact in fp32
  // and as large as half a step of h: 0.5 where |h| is 2^23.  A logit below m
  // is at least that far below, so where the difference passes a few hundred
  // (or h is infinite) the sums are zero, and the bound keeps zero zero.
  __device__ double unround(float m, float c, float h, float sign = 1.f) const {
    return exp2_fp64(double(sign * fminf(fmaxf(fmaf(m, c, -h), -500.f), 500.f)));
  }
  // What sums relative to h are multiplied by to be relative to a larger
  // maximum's `next`.  c m leaves fp32 only where the next smaller logit is
  // 2^104 / c below m, so those sums are nothing beside the new maximum.  In
  // fp64, since a rising row does this for each of a warp's segments (256 of
  // ex2.approx's errors of 2^-22 would be four times SA_SUM_ERROR).  Nothing
  // too where the maxima are a factor of 2^900 apart, so that unround()'s bound,
// which is for sums of zero, never meets another.
  __device__ double rescale(float h, float next) const {
    const double x = double(h) - double(next);  // NaN, if both are infinite
    return x > -900.0 && fabsf(h) < INFINITY ? exp2_fp64(x) : 0.0;
  }
  struct Settings {
    float temp, tp;
    int k;
    bool use_p, use_m;
    double u, thr;  // min_p as a bound on l - max
  };
  __device__ bool above_min(float l, const Settings& o) const {
    return diff(l) >= o.thr;
  }
  __device__ static u64 nucleus(float tp, double z) {  // ceil(tp z), one at least
    return u64(fmax(1.0, ceil(double(tp) * z)));
  }
  // What is known of the mass of all live logits.
  struct Total {
    bool exact;
    u64 mass;       // if exact
    double lo, hi;  // if not
  };
  // Both set res_rank to the chosen rank; by_list returns false if it cannot
  // be sure of it.
  __device__ bool by_list(const Settings& o, const SaFirst& f);
  // From the list, which holds a prefix of the ranks (all: every one), if that
  // is sure to hold what stays; a barrier of the cluster on both sides.
  __device__ bool finish(const Settings& o, const Total& z, bool all);
  __device__ void by_search(const Settings& o, const SaFirst& f);
  // The rank at which the running count (by_mass: mass) reaches the target
  // (at least 1, at most the total): res_rank, and by mass res_cum.
  // Not inlined (three calls): works on a copy, so that the members stay in
  // registers.
  __device__ void find(bool by_mass, u64 target) {
    const int was = find_apart(*this, by_mass, target);
    turn_ = was & 1;
    level0_ = was >> 1;
  }
  __device__ static __noinline__ int find_apart(Sampler me, bool by_mass, u64 target) {
    me.search(by_mass, target);
    return me.turn_ | (me.level0_ ? 2 : 0);
  }
  __device__ void search(bool by_mass, u64 target);
  // Mass of the logits for which keep(value, index) holds.
  template <typename F>
  __device__ u64 mass_of(F keep) {
    SaPart p = nothing();
    pass([&](const float (&v)[8], int c) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (v[j] > -INFINITY && keep(v[j], c + j)) p.mass += weight(v[j]);
    });
    return exchange(p).mass;
  }
  __device__ static u64 part_of(double f, double z) {  // floor(f z), f in [0, 1)
    return u64(floor(f * z));
  }
};

template <typename T>
__device__ void Sampler<T>::search(bool by_mass, u64 target) {
  u64 top = ~u64(0), bottom = 0, base = 0;  // the ranks searched; the measure above them
  float vt = max_, scale = bin_scale_;      // their bins: by value,
  int shift = -1;                           // or by index (one value)
  bool fits = false;
  if (!level0_) bin_level0();
  // Every step leaves at most half of the ranks, so 64 steps are enough.
  for (int step = 0; step < 64; ++step) {
    const u64 top0 = top, bottom0 = bottom;
    auto bin = [&](float l, int i) {
      if (step == 0) return bin_of(l);
      const u64 r = rank_of(l, i);
      if (r > top0 || r < bottom0) return -1;
      return shift >= 0 ? int((top0 - r) >> shift) : bin_below(vt, l, scale);
    };
    if (step > 0)  // the first bins are there already
      bin_up(by_mass, [&](uint32_t key) { return key >= uint32_t(bottom0 >> 32); }, bin);
    locate(by_mass, target - base);
    base += s_.base;
    fits = s_.n_in <= SA_CAP;
    const int here = s_.bin;
    SaPart p = nothing();
    pass(
        0, n_segs(),
        [&](uint32_t key) {
          return step == 0 ? bin_of(key_value(key)) <= here : key >= uint32_t(bottom0 >> 32);
        },
        [&](const float (&v)[8], int c) {
          const uint32_t mask = hits(v, c, [&](float l, int i) { return bin(l, i) == here; });
          if (fits)
            append(mask, v, c);
          else
            each(mask, v, c, [&](u64 r) {
              p.hi = max(p.hi, r);
              p.lo = min(p.lo, r);
            });
        });
    if (fits) break;
    p = exchange(p);
    top = p.hi;
    bottom = p.lo;
    if (top - bottom > (top0 - bottom0) / 2) {
      const u64 mid = bottom + (top - bottom) / 2;
      p = nothing();
      pass([&](const float (&v)[8], int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!(v[j] > -INFINITY)) continue;
          const u64 r = rank_of(v[j], c + j);
          if (r > mid && r <= top) p.mass += by_mass ? weight(v[j]) : 1;
        }
      });
      p = exchange(p);
      if (base + p.mass >= target) {
        bottom = mid + 1;
      } else {
        base += p.mass;
        top = mid;
      }
    }
    vt = rank_value(top);
    if ((top ^ bottom) >> 32) {
      shift = -1;
      scale = scale_for(vt - rank_value(bottom));
    } else {
      shift = max(0, 64 - __clzll((top - bottom) | 1) - 11);
    }
    level0_ = false;
  }
  meet();
  if (me_ == 0) {
    u64 r[4];
    const int n = sort_list(r);
    if (by_mass) {
      u64 cum[4];
      const u64 before = running_mass(n, base, r, cum);
      pick(n, before, r, cum, target);
    } else if (threadIdx.x == 0 && n > 0) {
      s_.res_rank = s_.list[min(max(int(target - base), 1), n) - 1];
    }
  }
  share_result();
}

// Largest of the lanes' values; NaN drops out.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The logits come in once.  Every warp keeps its own running maximum m, and
// its sums are relative to that until the end.  An exponential is one FMA and
// one ex2: 2^(c l - h) with h = c m rounded; the sums are put right by
// 2^(h - c m) at the end (the difference is the same for all terms).
template <typename T>
template <bool TAIL, bool Z>
__device__ SaFirst Sampler<T>::first_pass(float cz) {
  constexpr int STEP = SA_WARPS * SA_SEG;
  constexpr float CT = 1.44269504f;  // log2(e)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY, ht = 0.f, hz = 0.f, least = INFINITY;
  int mi = 0x7FFFFFFF, ne = 0;
  double tail = 0.0, z = 0.0;
  constexpr int PL = sizeof(T) / 2;
  const int cw = s0_ + warp * SA_SEG;  // where the warp's first segment begins
  const int np = cw < s1_ ? (s1_ - cw + STEP - 1) / STEP : 0;
  __syncthreads();  // what run() laid out in shared memory
  for (int p = 0; p < np; ++p) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    float v[NB][8], vm = -INFINITY;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      SaRaw<T> r;
#pragma unroll
      for (int i = 0; i < PL; ++i) r.v[i] = slot(p)[(k * PL + i) * SA_THREADS];
      raw_values<T>(r, v[k]);
    }
    copy_in(p + DEPTH);
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) vm = fmaxf(vm, v[k][j]);  // NaN drops out
    const float bm = warp_max(vm);
    if (bm == -INFINITY) continue;  // nothing live
    if (lane == 0) {
      const int seg = warp + p * SA_WARPS;
      if (a_.seg_mul == 1) s_.segs[seg] = value_key(bm);
      else atomicMax(&s_.segs[seg / a_.seg_mul], value_key(bm));
    }
    least = fminf(least, bm);
    if (bm > m) {
      // the sums so far, and the instances of the old maximum, in the new scale
      const float nt = bm * CT, nz = bm * cz;
      if (m > -INFINITY) {
        if (TAIL) tail = (tail + double(ne) * unround(m, CT, ht)) * rescale(ht, nt);
        if (Z) z = (z + double(ne) * unround(m, cz, hz)) * rescale(hz, nz);
      }
      m = bm;
      ht = nt;
      hz = nz;
      ne = 0;
      mi = 0x7FFFFFFF;
    }
    float st[NB] = {}, sz[NB] = {};
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (TAIL) st[k] += ex2_approx(fmaf(v[k][j], CT, -ht));
        if (Z) sz[k] += ex2_approx(fmaf(v[k][j], cz, -hz));
      }
    float sum_t = st[0], sum_z = sz[0];
#pragma unroll
    for (int k = 1; k < NB; ++k) {
      sum_t += st[k];
      sum_z += sz[k];
    }
    // the maximum itself, NaN, infinities, a maximum whose h is infinite
    if (vm == m || !(sum_t < INFINITY) || !(sum_z < INFINITY)) {
      sum_t = sum_z = 0.f;
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float l = v[k][j];
          if (l == m) {
            ++ne;
            mi = min(mi, cw + p * STEP + k * 256 + lane * 8 + j - off_);
          } else if (l - m > -INFINITY) {
            // nothing beside a maximum whose h is not finite (rescale())
            if (fabsf(ht) < INFINITY) sum_t += ex2_approx(fmaf(l, CT, -ht));
            if (fabsf(hz) < INFINITY) sum_z += ex2_approx(fmaf(l, cz, -hz));
          }
        }
    }
    if (TAIL) tail += double(sum_t);
    if (Z) z += double(sum_z);
  }
  if (TAIL) tail *= unround(m, CT, ht, -1.f);
  if (Z) z *= unround(m, cz, hz, -1.f);
  // threads -> CTA
  SaFirst f;
  f.hi = mi != 0x7FFFFFFF ? rank_of(m, mi) : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    f.hi = max(f.hi, __shfl_xor_sync(0xffffffffu, f.hi, o));
    tail += __shfl_xor_sync(0xffffffffu, tail, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    ne += __shfl_xor_sync(0xffffffffu, ne, o);
  }
  f.tail = tail;
  f.z = z;
  f.n = ne;
  f.least = least;
  if (lane == 0) s_.warp_first[warp] = f;
  __syncthreads();
  // The first store to the others' shared memory is below.
  if (!all_run_) cluster_wait_started();
  // The parts of n members, one in each of n lanes, relative to their common
  // maximum.
  auto join = [&](SaFirst p, int n) {
    u64 hi = p.hi;
    float lo = p.least;
    for (int o = n / 2; o > 0; o >>= 1) {
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (p.hi == 0) {
      p.tail = p.z = 0.0;
      p.n = 0;
    } else if (p.hi >> 32 != hi >> 32) {
      const float d = rank_value(p.hi) - rank_value(hi);
      p.tail = (p.tail + p.n) * ex2_approx(d * 1.44269504f);
      p.z = (p.z + p.n) * ex2_approx(d == -INFINITY ? d : d * cz);
      p.n = 0;
    }
    for (int o = n / 2; o > 0; o >>= 1) {
      p.tail += __shfl_xor_sync(0xffffffffu, p.tail, o);
      p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
      p.n += __shfl_xor_sync(0xffffffffu, p.n, o);
    }
    p.hi = hi;
    p.least = lo;
    return p;
  };
  if (warp == 0) {
    f = join(s_.warp_first[lane & (SA_WARPS - 1)], SA_WARPS);
    if (lane < C_) *cl_.map_shared_rank(&s_.firsts[me_], lane) = f;
  }
  meet();
  return join(s_.firsts[lane & (C_ - 1)], C_);
}

template <typename T>
__device__ bool Sampler<T>::by_list(const Settings& o, const SaFirst& f) {
  // Bins between the maximum and the least of the segments' maxima, which
  // falls short of the last bin; that one takes what is below.
  float scale = scale_for(below(f.least)) * 0.996f;
  int last;  // candidates: the logits in bins up to this one
  bool all = false;
  if (o.use_m && !o.use_p && o.k == 0) {
    last = int(fmin(floor(-o.thr * (1.0 + 0x1p-20) * double(scale)) + 1.0, double(SA_BINS)));
  } else {
    // top-k: the bin of the k-th rank; else the bin down to which there is the
    // mass that is asked for.  From the maxima alone if those are enough (of
    // each segment that reaches a bin one logit is known to be there).  If not,
    // from the counts of all logits where a CTA has few of them (4,096 logits,
    // top-k 50: 30 us without), else the SA_OPEN largest segments are opened.
    const double part = (o.use_p ? double(fmaxf(o.tp, 0.f)) : o.u) * (1.0 + SA_SUM_ERROR);
    const u64 mass = u64(part * (double(f.n) + f.z) * 0x1p20) + 2;
    // The bin in which the count or the mass reaches `want`, or -1; n_in: the
    // count up to it.
    auto reach = [&](uint4 n4, bool count, u64 want) {
      const uint32_t n[4] = {n4.x, n4.y, n4.z, n4.w};
      u64 m[4], sum = 0, cnt = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // a weight at the bin's far end, rounded down; the last bin has no end
        const int b = threadIdx.x * 4 + i;
        const float x = float(b + 1) / scale * float(-c_);
        const u64 w = b < SA_BINS - 1 ? u64(ex2_approx(x) * 0x1p20f * 0.99f) : 0;
        cnt += n[i];
        m[i] = sum += count ? u64(n[i]) : n[i] * w;
      }
      if (threadIdx.x == 0) s_.bin = -1;
      __syncthreads();
      const u64 before = scan(sum, s_.warp_sum[0]) - sum;
      u64 upto = scan(cnt, s_.warp_sum[1]) - cnt;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        upto += n[i];
        if (before + m[i] >= want && before + (i ? m[i - 1] : 0) < want) {
          s_.bin = threadIdx.x * 4 + i;
          s_.n_in = uint32_t(upto);
        }
      }
      __syncthreads();
      const int b = s_.bin;
      __syncthreads();
      return b;
    };
    if (o.k > SA_CAP / 2 && a_.V > SA_CAP) return false;
    const int n_maxima = (n_segs() + a_.seg_mul - 1) / a_.seg_mul;
    uint32_t* open = cl_.map_shared_rank(s_.open, 0);
    for (int i = threadIdx.x; i < n_maxima; i += SA_THREADS)
      if (s_.segs[i] != 0) atomicAdd(&open[bin_below(max_, key_value(s_.segs[i]), scale)], 1u);
    meet();
    const uint4 maxima = reinterpret_cast<const uint4*>(open)[threadIdx.x];
    last = reach(maxima, o.k > 0, o.k > 0 ? u64(o.k) : mass);
    if (last < 0 && a_.slice <= SA_COUNT_SLICE) {
      // twice as far down as the least of the maxima
      scale *= 0.5f;
      bin_up(false, [](uint32_t) { return true; },
             [&](float l, int) { return bin_below(max_, l, scale); });
      last = reach(reinterpret_cast<const uint4*>(s_.tot)[threadIdx.x], o.k > 0,
                   o.k > 0 ? u64(o.k) : mass);
      if (last < 0 && a_.V <= SA_CAP) {
        last = SA_BINS;
        all = true;
      } else if (last < 0 || s_.n_in > SA_CAP) {
        return false;
      }
    } else if (last < 0) {
      last = o.k > 0 ? -1 : reach(maxima, true, SA_OPEN);
      if (last < 0) last = bin_below(max_, f.least, scale);
    }
    __syncthreads();
  }
  // the segments that reach that far, then their logits
  for (int i = threadIdx.x; i < n_segs(); i += SA_THREADS) {
    const uint32_t key = s_.segs[i / a_.seg_mul];
    if (key != 0 && bin_below(max_, key_value(key), scale) <= last)
      s_.opened[atomicAdd(&s_.n_opened, 1)] = uint16_t(i);
  }
  __syncthreads();
  constexpr int UN = 4;
  const int n_opened = s_.n_opened;
  for (int i0 = threadIdx.x >> 5; i0 < n_opened * NB; i0 += SA_WARPS * UN) {
    SaRaw<T> r[UN];
    int c[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int i = i0 + k * SA_WARPS;
      // a piece of 256 of each
      c[k] = i < n_opened * NB ? s0_ + int(s_.opened[i / NB]) * SA_SEG + i % NB * 256 +
                                     int(threadIdx.x & 31) * 8
                               : s1_;
      if (c[k] < s1_) r[k] = fetch(c[k]);
    }
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      float v[8] = {};
      uint32_t mask = 0;
      if (c[k] < s1_) {
        raw_values<T>(r[k], v);
        mask = hits(v, c[k] - off_, [&](float l, int) { return bin_below(max_, l, scale) <= last; });
      }
      append(mask, v, c[k] - off_);
    }
  }
  const double unit = double(u64(1) << a_.bits);
  Total z;
  z.exact = all;
  z.mass = 0;
  z.lo = (double(f.n) + f.z * (1.0 - SA_SUM_ERROR)) * unit - double(a_.V);
  z.hi = (double(f.n) + f.z * (1.0 + SA_SUM_ERROR)) * unit + double(a_.V);
  return finish(o, z, all);
}

template <typename T>
__device__ bool Sampler<T>::finish(const Settings& o, const Total& z, bool all) {
  meet();
  if (me_ == 0) {
    bool ok = s_.n_list <= SA_CAP;
    if (ok) {
      u64 r[4], cum[4];
      const int n = sort_list(r);
      const u64 before = running_mass(n, 0, r, cum);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = threadIdx.x * 4 + i;
        if (q == n - 1) s_.end = cum[i];
        if (o.k > 0 && q == min(o.k, n) - 1) s_.res_cum = cum[i];
      }
      __syncthreads();
      const u64 end = s_.end;
      // mass of the kept ranks: exact, or between two bounds
      u64 keep = all ? end : z.mass;
      bool exact = z.exact;
      if (o.k > 0) {
        ok = all || n >= o.k;
        keep = s_.res_cum;
        exact = true;
      }
      // the rank that both ends of the interval lead to
      auto settle = [&](u64 a, u64 b) {
        pick(n, before, r, cum, a);
        const u64 first = s_.res_rank;
        if (b != a) pick(n, before, r, cum, b);
        return b <= end && s_.res_rank == first;
      };
      if (ok && o.use_p) {
        ok = exact ? settle(min(nucleus(o.tp, double(keep)), keep), min(nucleus(o.tp, double(keep)), keep))
                   : settle(nucleus(o.tp, z.lo), nucleus(o.tp, z.hi));
        keep = exact ? min(keep, s_.res_cum) : s_.res_cum;
        exact = true;
      }
      if (ok && o.use_m) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the last rank that min_p leaves
          const int q = threadIdx.x * 4 + i;
          const bool in = q < n && above_min(rank_value(r[i]), o);
          if (in && !(q + 1 < n && above_min(rank_value(s_.list[q + 1]), o))) s_.res_cum = cum[i];
        }
        __syncthreads();
        keep = exact ? min(keep, s_.res_cum) : s_.res_cum;
        exact = true;
      }
      if (ok)
        ok = exact ? settle(part_of(o.u, double(keep)) + 1, part_of(o.u, double(keep)) + 1)
                   : settle(part_of(o.u, z.lo) + 1, part_of(o.u, z.hi) + 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) s_.n_list = 0;  // it may have run over
    if (int(threadIdx.x) < C_) *cl_.map_shared_rank(&s_.done, threadIdx.x) = ok;
  }
  meet();
  return s_.done;
}

template <typename T>
__device__ void Sampler<T>::by_search(const Settings& o, const SaFirst& f) {
  // Whether all ranks down to `last`, in bins of this scale, fit a list, and
  // settle the rest.
  auto settled = [&](const Settings& p, int last, float scale, u64 keep) {
    u64 n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (int(threadIdx.x) * 4 + i <= last) n += s_.tot[threadIdx.x * 4 + i];
    __syncthreads();
    n = scan(n, s_.warp_sum[0]);
    if (threadIdx.x == SA_THREADS - 1) s_.base = n;
    __syncthreads();
    if (s_.base > SA_CAP) return false;
    pass(
        0, n_segs(), [&](uint32_t key) { return bin_below(max_, key_value(key), scale) <= last; },
        [&](const float (&v)[8], int c) {
          append(hits(v, c, [&](float l, int) { return bin_below(max_, l, scale) <= last; }), v, c);
        });
    return finish(p, Total{true, keep, 0.0, 0.0}, false);
  };
  if (o.k > 0 && o.k <= SA_CAP) {
    // Counts alone, down to twice as far as the least of the segments' maxima.
    const float scale = scale_for(2.f * below(f.least));
    bin_up(false, [](uint32_t) { return true; },
           [&](float l, int) { return bin_below(max_, l, scale); });
    locate(false, u64(o.k));
    const int last = s_.bin;
    if (s_.base + s_.n_in >= u64(o.k) && settled(o, last, scale, 0)) return;
    meet();  // the counts have been read
  }
  // Bins over 24 T: what lies below has less than 4e-11 of the largest weight
  // each, and falls into the last bin.
  bin_scale_ = scale_for(24.f * o.temp);
  bin_level0();
  u64 live = 0, keep = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    live += s_.tot[threadIdx.x * 4 + i];
    keep += s_.mass[threadIdx.x * 4 + i];
  }
  live = scan(live, s_.warp_sum[0]);
  keep = scan(keep, s_.warp_sum[1]);
  if (threadIdx.x == SA_THREADS - 1) {
    s_.base = live;
    s_.end = keep;
  }
  __syncthreads();
  live = s_.base;
  keep = s_.end;
  Settings p = o;
  if (u64(o.k) >= live) p.k = 0;
  if (p.k > 0) {
    find(false, u64(p.k));
    const u64 cut = s_.res_rank;
    keep = mass_of([&](float l, int i) { return rank_of(l, i) >= cut; });
  } else {
    // the bin that the first filter, or the draw, ends in
    if (p.use_p) locate(true, min(nucleus(p.tp, double(keep)), keep));
    else if (!p.use_m) locate(true, part_of(p.u, double(keep)) + 1);
    const int last = p.use_p || !p.use_m
                         ? s_.bin
                         : int(fmin(floor(-p.thr * (1.0 + 0x1p-20) * double(bin_scale_)) + 1.0,
                                    double(SA_BINS - 1)));
    if (settled(p, last, bin_scale_, keep)) return;
  }
  if (o.use_p) {
    find(true, min(nucleus(o.tp, double(keep)), keep));
    keep = min(keep, s_.res_cum);
  }
  if (o.use_m) keep = min(keep, mass_of([&](float l, int) { return above_min(l, o); }));
  find(true, part_of(o.u, double(keep)) + 1);
}

template <typename T>
template <int MODE>
__device__ void Sampler<T>::run() {
  for (int p = 0; p < DEPTH; ++p) copy_in(p);  // before anything is waited for
  Settings o;
  o.temp = a_.temperature == nullptr ? 1.f : a_.temperature[row_];
  o.k = a_.top_k == nullptr ? 0 : a_.top_k[row_];
  o.tp = a_.top_p == nullptr ? 1.f : a_.top_p[row_];
  const float mp = a_.min_p == nullptr ? 0.f : a_.min_p[row_];
  const float u = a_.u[row_];
  for (int i = threadIdx.x; i < SA_BINS; i += SA_THREADS) s_.open[i] = 0;
  for (int i = threadIdx.x; i < SA_MAX_SEGS; i += SA_THREADS) s_.segs[i] = 0;
  if (threadIdx.x == 0) s_.n_list = s_.n_opened = 0;
  if (threadIdx.x < 32) s_.pow2[threadIdx.x] = SA_POW2[threadIdx.x];
  o.k = o.k < 0 || o.k >= a_.V ? 0 : o.k;
  o.u = double(fminf(fmaxf(u, 0.f), 1.f - 0x1p-24f));
  o.use_p = o.tp < 1.f;
  o.use_m = mp > 0.f;
  o.thr = o.use_m && mp < 1.f ? double(o.temp) * log(double(mp)) : 0.0;
  // (a min_p above 1 leaves no weight: the first rank, equal ones apart)
  const bool greedy = !(o.temp > 0.f) || o.k == 1 || mp > 1.f;
  const bool need_z =
      MODE != SA_SEARCH_ONLY && !greedy && o.k == 0 && (o.use_p || !o.use_m);
  c_ = 1.4426950408889634074 / double(o.temp);
  const bool same = o.temp == 1.f;  // one sum serves both

  const bool tail = a_.logp != nullptr || (need_z && same);
  SaFirst f = need_z && !same ? (tail ? first_pass<true, true>(float(c_))
                                      : first_pass<false, true>(float(c_)))
                              : (tail ? first_pass<true, false>(0.f) : first_pass<false, false>(0.f));
  if (same) f.z = f.tail;
  // a temperature so small that 1 / T is beyond fp32: the mass is not known
  if (need_z && !(float(c_) < INFINITY)) f.z = INFINITY;
  const bool lead = me_ == 0 && threadIdx.x == 0;
  if (f.hi == 0) {
    if (lead) {
      a_.token[row_] = -1;
      if (a_.logp != nullptr) a_.logp[row_] = 0.f;
    }
    return;
  }
  max_ = rank_value(f.hi);
  u64 token = f.hi;
  if (!greedy) {
    const bool done = MODE != SA_SEARCH_ONLY && by_list(o, f);
    if (!done) {
      if (MODE == SA_LIST_ONLY) {
        if (lead) a_.token[row_] = SA_UNDECIDED;
        return;
      }
      by_search(o, f);
    }
    token = s_.res_rank;
  }
  if (lead) {
    a_.token[row_] = rank_index(token);
    if (a_.logp != nullptr)
      a_.logp[row_] =
          float(diff(rank_value(token)) - log1p(f.tail + double(f.n - 1)));
  }
}

// The next row, from `start` round the batch, that the list left undecided and
// no cluster has claimed yet, now claimed; -1: none.  For a whole CTA.  A row
// that was seen taken never comes back, so each CTA goes over the batch once,
// 2,048 rows a step.  2^20 rows of 8 logits, none of them left: 16.0 ms in all,
// 27.1 with one warp that went over 32 rows a step, again for each claim; 256
// rows, none left: 2 us less.
__device__ inline int claim_row(const SampleArgs& a, SaShared& s, int start, int& seen) {
  constexpr int EACH = 4, NONE = 0x7FFFFFFF;
  const int lane = threadIdx.x & 31;
  while (seen < a.B) {
    int at = NONE;
    uint32_t t[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int k = seen + j * SA_THREADS + int(threadIdx.x);
      t[j] = 0;
      if (k < a.B)
        t[j] = ld_relaxed_gpu(
            reinterpret_cast<const uint32_t*>(a.token + (start + k < a.B ? start + k : start + k - a.B)));
    }
#pragma unroll
    for (int j = EACH - 1; j >= 0; --j)
      if (t[j] == uint32_t(SA_UNDECIDED)) at = seen + j * SA_THREADS + int(threadIdx.x);
    at = __reduce_min_sync(0xffffffffu, at);
    __syncthreads();  // the last step's answers have been read
    if (lane == 0) s.found[threadIdx.x >> 5] = at;
    __syncthreads();
    at = __reduce_min_sync(0xffffffffu, s.found[lane & (SA_WARPS - 1)]);
    if (at == NONE) {
      seen += EACH * SA_THREADS;
      continue;
    }
    seen = at;
    const int row = start + at < a.B ? start + at : start + at - a.B;
    if (threadIdx.x == 0) s.claimed = atomicCAS(a.token + row, SA_UNDECIDED, SA_CLAIMED) == SA_UNDECIDED;
    __syncthreads();
    if (s.claimed) return row;
  }
  return -1;
}

// 128 registers a thread where the search runs: with 64 (two CTAs on an SM) it
// spilled more, and one row took 17 us instead of 13 by list and 51 instead of
// 35 by search.  What spills now (bytes stored a thread, fp32 and bf16): 152 and
// 116 in the search, 32 and 44 where one launch does both, and 218 and 192 in
// the list's own launch, whose 64 registers are worth it for many rows
// (launch_sample_rows).  One cluster a row; the search's clusters take rows that
// are left, each when it is done with its last (the rows cost very different
// times).
template <typename T, int MODE>
__global__ void __launch_bounds__(SA_THREADS, MODE == SA_LIST_ONLY ? 2 : 1)
    sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t sa_smem[];
  SaShared& s = *reinterpret_cast<SaShared*>(sa_smem);
  const int n = int(cluster_count_x()), id = int(cluster_id_x());
  auto cluster = cooperative_groups::this_cluster();
  // No CTA touches another's shared memory before all of them run.  Arrived
  // here, waited for only where the first such store is made, so that the wait
  // lies behind the row's first copies.
  const bool alone = cluster.num_blocks() == 1;
  if (!alone) cluster_arrive_started();
  if (MODE != SA_SEARCH_ONLY) {
    Sampler<T>(a, s, id, alone).template run<MODE>();
    return;
  }
  if (!alone) cluster_wait_started();
  const int start = int(int64_t(a.B) * id / n);
  int seen = 0;  // rows from start on that are known to be taken
  for (;;) {
    if (cluster.block_rank() == 0) {
      const int row = claim_row(a, s, start, seen);
      if (threadIdx.x < cluster.num_blocks()) *cluster.map_shared_rank(&s.row, threadIdx.x) = row;
    }
    cluster.sync();
    const int row = s.row;
    if (row < 0) return;
    Sampler<T>(a, s, row, true).template run<MODE>();
    cluster.sync();  // the row's shared memory is done with
  }
}

}  // namespace cce
