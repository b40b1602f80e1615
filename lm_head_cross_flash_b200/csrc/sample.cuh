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
// Search.  A cluster of CTAs holds the row in shared memory, so the logits are
// read from memory once.  One pass counts the live logits in 2,048 bins of
// equal width below the maximum.  The counts, with the largest and smallest
// weight that a bin can hold, bracket the bin in which the target is reached;
// the few candidates of the bracket are collected, sorted by the cluster's
// first CTA, and summed exactly.  A bracket that holds more candidates than
// the list takes (a flat row, or many equal logits) is searched again with
// 2,048 bins of its own, over its values or, where those are all equal, over
// its indices, until it fits; a step that does not halve it is followed by a
// bisection, so the search ends for every input.
#pragma once

#include <cooperative_groups.h>

#include "row_ops.cuh"

namespace cce {

constexpr int SA_THREADS = 512;
constexpr int SA_WARPS = SA_THREADS / 32;
constexpr int SA_BINS = 2048;
constexpr int SA_CAP = 2048;  // candidates of one list
constexpr int SA_MAX_CLUSTER = 8;
static_assert(SA_CAP == 4 * SA_THREADS && SA_BINS == 4 * SA_THREADS, "four entries per thread");

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V;
  int slice;     // logits per CTA, a multiple of 8
  int resident;  // the slice is kept in shared memory
  int vec;       // rows start on 16-byte boundaries
  int bits;      // binary places of a weight
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
  double tail;  // sum of exp(l - max) without the maximum itself
  float least;
  int n;
};

struct SaShared {
  uint32_t tot[SA_BINS];   // level-0 counts of the cluster
  uint32_t hist[SA_BINS];  // this CTA's counts
  union {
    u64 list[SA_CAP];
    uint32_t tot2[SA_BINS];  // counts of a finer search
  };
  double pow2[32];  // 2^(j/32)
  SaPart parts[2][SA_MAX_CLUSTER];
  SaPart warp_part[SA_WARPS];
  u64 warp_sum[3][SA_WARPS];
  u64 res_rank, res_cum;
  int lo_bin, hi_bin, last_bin;
  uint32_t n_above, n_in;
  int n_list;
  int counts[SA_MAX_CLUSTER];
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

template <typename T>
class Sampler {
 public:
  __device__ Sampler(const SampleArgs& a, SaShared& s, uint4* store)
      : a_(a), s_(s), store_(store), cl_(cooperative_groups::this_cluster()) {
    C_ = int(cl_.num_blocks());
    me_ = int(cl_.block_rank());
    row_ = int(blockIdx.x) / C_;
    g_ = static_cast<const T*>(a.logits) + int64_t(row_) * a.ld;
    s0_ = int(min(int64_t(a.V), int64_t(me_) * a.slice));
    s1_ = int(min(int64_t(a.V), int64_t(s0_) + a.slice));
    if (threadIdx.x < 32) s_.pow2[threadIdx.x] = exp2(double(threadIdx.x) / 32.0);
  }

  __device__ void run();

 private:
  const SampleArgs& a_;
  SaShared& s_;
  uint4* store_;
  cooperative_groups::cluster_group cl_;
  int C_, me_, row_, s0_, s1_;
  const T* g_;
  int turn_ = 0;      // which half of `parts` the next exchange uses
  float max_ = 0.f;
  double c_ = 0.0;    // log2(e) / T
  float bin_scale_ = 0.f;

  // ------------------------------------------------------------- passes --
  __device__ SaRaw<T> fetch(int c) const {
    SaRaw<T> r;
    if (a_.vec && c + 8 <= s1_) {
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i)
        r.v[i] = __ldg(reinterpret_cast<const uint4*>(g_ + c) + i);
    } else {  // -inf behind the end
      uint32_t w[sizeof(T) * 2];
#pragma unroll
      for (int i = 0; i < int(sizeof(T) * 2); ++i) {
        if constexpr (sizeof(T) == 4) {
          w[i] = c + i < s1_ ? __float_as_uint(g_[c + i]) : 0xFF800000u;
        } else {
          const uint32_t lo = c + 2 * i < s1_ ? __bfloat16_as_ushort(g_[c + 2 * i]) : 0xFF80u;
          const uint32_t hi = c + 2 * i + 1 < s1_ ? __bfloat16_as_ushort(g_[c + 2 * i + 1]) : 0xFF80u;
          w[i] = lo | (hi << 16);
        }
      }
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i)
        r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    return r;
  }
  // Calls f(values, first index) on every piece of eight logits of the slice.
  template <typename F>
  __device__ void pass(F f) const {
    const int plane = a_.slice / 8;
    for (int c = s0_ + int(threadIdx.x) * 8; c < s1_; c += SA_THREADS * 8) {
      SaRaw<T> r;
      if (a_.resident) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) r.v[i] = store_[i * plane + (c - s0_) / 8];
      } else {
        r = fetch(c);
      }
      float v[8];
      raw_values<T>(r, v);
      f(v, c);
    }
  }

  __device__ float below(float l) const { return l == max_ ? 0.f : max_ - l; }
  __device__ int bin_of(float l) const { return bin_below(max_, l, bin_scale_); }

  // round(2^bits * 2^x) for x <= 0: with k = round(32 x), r = x - k/32,
  // 2^x = 2^(k div 32) 2^((k mod 32)/32) 2^r, and 2^r by its series to r^5
  // (the next term is below 2.3e-15).  The last addition leaves the integer
  // in the low bits of the sum.
  __device__ u64 weight_log2(double x) const {
    if (!(x > -50.0)) return 0;
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
    const double ts = __hiloint2double(__double2hiint(t) + ((k >> 5) + a_.bits) * (1 << 20),
                                       __double2loint(t));
    const double w = fma(ts, r * p, ts) + 4503599627370496.0;  // + 2^52
    return u64(__double_as_longlong(w)) & 0x000FFFFFFFFFFFFFull;
  }
  __device__ u64 weight(float l) const {
    if (l == max_) return u64(1) << a_.bits;
    return weight_log2((double(l) - double(max_)) * c_);
  }

  // ------------------------------------------------- block and cluster --
  __device__ static SaPart merge(const SaPart& x, const SaPart& y) {
    SaPart r;
    r.hi = max(x.hi, y.hi);
    r.lo = min(x.lo, y.lo);
    r.mass = x.mass + y.mass;
    r.tail = x.tail + y.tail;
    r.least = fminf(x.least, y.least);
    r.n = x.n + y.n;
    return r;
  }
  __device__ static SaPart nothing() {
    SaPart p;
    p.hi = 0;
    p.lo = ~u64(0);
    p.mass = 0;
    p.tail = 0.0;
    p.least = INFINITY;
    p.n = 0;
    return p;
  }
  // The threads' parts of all CTAs, merged in a fixed order; every thread of
  // the cluster gets the result.  Also a barrier of the cluster.
  __device__ SaPart exchange(SaPart p) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      SaPart q;
      q.hi = __shfl_xor_sync(0xffffffffu, p.hi, o);
      q.lo = __shfl_xor_sync(0xffffffffu, p.lo, o);
      q.mass = __shfl_xor_sync(0xffffffffu, p.mass, o);
      q.tail = __shfl_xor_sync(0xffffffffu, p.tail, o);
      q.least = __shfl_xor_sync(0xffffffffu, p.least, o);
      q.n = __shfl_xor_sync(0xffffffffu, p.n, o);
      p = merge(p, q);
    }
    if ((threadIdx.x & 31) == 0) s_.warp_part[threadIdx.x >> 5] = p;
    __syncthreads();
    if (int(threadIdx.x) < C_) {
      p = s_.warp_part[0];
      for (int i = 1; i < SA_WARPS; ++i) p = merge(p, s_.warp_part[i]);
      *cl_.map_shared_rank(&s_.parts[turn_][me_], threadIdx.x) = p;
    }
    cl_.sync();
    p = s_.parts[turn_][0];
    for (int i = 1; i < C_; ++i) p = merge(p, s_.parts[turn_][i]);
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
  __device__ void clear_hist() {
    for (int i = threadIdx.x; i < SA_BINS; i += SA_THREADS) s_.hist[i] = 0;
    __syncthreads();
  }
  // The CTAs' counts added into `tot` of every CTA; barriers on both sides.
  __device__ void total_hist(uint32_t* tot) {
    cl_.sync();
    const int n = SA_BINS / C_;
    for (int i = threadIdx.x; i < n; i += SA_THREADS) {
      const int b = me_ * n + i;
      uint32_t x = 0;
      for (int r = 0; r < C_; ++r) x += *cl_.map_shared_rank(&s_.hist[b], r);
      for (int r = 0; r < C_; ++r) *cl_.map_shared_rank(&tot[b], r) = x;
    }
    cl_.sync();
  }

  // Bins [lo_bin, hi_bin] that hold the rank at which the target is reached,
  // and the counts above and inside, from the bins' counts.  edge(b, up): the
  // largest / smallest weight that bin b can hold (by mass only).
  template <typename E>
  __device__ void bracket(const uint32_t* tot, bool by_mass, u64 target, E edge) {
    const int b0 = threadIdx.x * 4;
    u64 n[4], up[4], dn[4], sn = 0, su = 0, sd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 k = tot[b0 + i];
      n[i] = sn += k;
      up[i] = su += by_mass && k ? k * edge(b0 + i, true) : k;
      dn[i] = sd += by_mass && k ? k * edge(b0 + i, false) : k;
    }
    if (threadIdx.x == 0) {
      s_.lo_bin = s_.hi_bin = s_.last_bin = -1;
      s_.n_above = s_.n_in = 0;
    }
    __syncthreads();
    const u64 en = scan(sn, s_.warp_sum[0]) - sn;
    const u64 eu = scan(su, s_.warp_sum[1]) - su;
    const u64 ed = scan(sd, s_.warp_sum[2]) - sd;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 u0 = i ? up[i - 1] : 0, d0 = i ? dn[i - 1] : 0;
      // exactly one bin reaches the target first, if any does
      if (eu + up[i] >= target && eu + u0 < target) s_.lo_bin = b0 + i;
      if (ed + dn[i] >= target && ed + d0 < target) s_.hi_bin = b0 + i;
      if (up[i] > u0) atomicMax(&s_.last_bin, b0 + i);
    }
    __syncthreads();
    // the last bin that can hold any of the measure bounds both
    const int last = max(s_.last_bin, 0);
    const int lo = s_.lo_bin < 0 ? last : s_.lo_bin, hi = s_.hi_bin < 0 ? last : s_.hi_bin;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (b0 + i == lo - 1) s_.n_above = uint32_t(en + n[i]);
      if (b0 + i == hi) s_.n_in = uint32_t(en + n[i]);  // up to here, for now
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      s_.n_in -= s_.n_above;
      s_.lo_bin = lo;
      s_.hi_bin = hi;
    }
    __syncthreads();
  }

  // This CTA's candidates go to its list; the caller's pass appends them.
  __device__ void append(u64 r) {
    const int i = atomicAdd(&s_.n_list, 1);
    if (i < SA_CAP) s_.list[i] = r;
  }
  // All lists into the first CTA's, sorted there from the highest rank down.
  // Returns the number of candidates (first CTA only).  Begins with a barrier
  // of the cluster.
  __device__ int gather_sorted() {
    cl_.sync();
    if (me_ != 0) return 0;
    if (int(threadIdx.x) < C_)
      s_.counts[threadIdx.x] = min(*cl_.map_shared_rank(&s_.n_list, threadIdx.x), SA_CAP);
    __syncthreads();
    int n = s_.counts[0];
    for (int r = 1; r < C_; ++r) {
      const u64* from = cl_.map_shared_rank(s_.list, r);
      const int k = min(s_.counts[r], SA_CAP - n);
      for (int i = threadIdx.x; i < k; i += SA_THREADS) s_.list[n + i] = from[i];
      n += k;
    }
    int len = 2;
    while (len < n) len *= 2;
    for (int i = n + threadIdx.x; i < len; i += SA_THREADS) s_.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= len; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int t = threadIdx.x; t < len / 2; t += SA_THREADS) {
          const int i = 2 * t - (t & (j - 1)), o = i + j;
          const u64 x = s_.list[i], y = s_.list[o];
          if ((x < y) == ((i & k) == 0)) {
            s_.list[i] = y;
            s_.list[o] = x;
          }
        }
        __syncthreads();
      }
    return n;
  }
  // First CTA: the four sorted candidates of this thread with the masses up
  // to and including each, above `base`.  Returns the mass before the first.
  __device__ u64 running_mass(int n, u64 base, u64 (&r)[4], u64 (&cum)[4]) {
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = threadIdx.x * 4 + i;
      r[i] = k < n ? s_.list[k] : 0;
      sum += k < n ? weight(rank_value(r[i])) : 0;
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
    cl_.sync();
  }

  // Bins of equal width below the value vt: a logit l falls into bin
  // min(2047, (vt - l) scale), so bin b holds vt - l in [b, b + 1) / scale,
  // give or take the two roundings (below 2^-22 relative).  The largest or
  // smallest weight that it can hold; nothing is known of the last bin's end.
  __device__ u64 edge(int b, bool up, float vt, float scale) const {
    if (!up && b == SA_BINS - 1) return 0;
    const double d = up ? double(b) / double(scale) * (1.0 - 0x1p-20)
                        : double(b + 1) / double(scale) * (1.0 + 0x1p-20);
    const double off = vt == max_ ? 0.0 : double(vt) - double(max_);
    return weight_log2((off - d) * c_);
  }
  __device__ static int bin_below(float vt, float l, float scale) {
    return l == vt ? 0 : int(fminf((vt - l) * scale, float(SA_BINS - 1)));
  }
  __device__ static float scale_for(float span) {
    const float s = span > 0.f ? float(SA_BINS - 1) / span : 1.f;
    return s < 1e30f ? s : 1e30f;
  }

  // The rank at which the running count (by_mass: mass) reaches the target
  // (at least 1, at most the total): res_rank, and by mass res_cum.
  __device__ void find(bool by_mass, u64 target);
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
  __device__ static u64 part_of(double f, u64 z) {  // floor(f z), f in [0, 1)
    const double x = floor(f * double(z));
    return u64(x);
  }
};

template <typename T>
__device__ void Sampler<T>::find(bool by_mass, u64 target) {
  u64 top = ~u64(0), bottom = 0, base = 0;  // the bracket's ranks; the measure above it
  float vt = max_, scale = bin_scale_;      // its bins: by value,
  int shift = -1;                           // or by index (one value)
  const uint32_t* tot = s_.tot;
  // Every step leaves at most half of the ranks, so 64 steps are enough.
  for (int step = 0; step < 64; ++step) {
    const u64 top0 = top, bottom0 = bottom;
    auto bin = [&](u64 r, float l) {
      return shift >= 0 ? int((top0 - r) >> shift) : bin_below(vt, l, scale);
    };
    bracket(tot, by_mass, target - base, [&](int b, bool up) -> u64 {
      return shift >= 0 ? weight(vt) : edge(b, up, vt, scale);
    });
    const bool whole = base == 0 && s_.n_above + s_.n_in <= SA_CAP;  // no pass for the mass above
    const int lo = whole ? 0 : s_.lo_bin, hi = s_.hi_bin;
    const uint32_t n_above = whole ? 0 : s_.n_above;
    const bool fits = whole || s_.n_in <= SA_CAP;
    __syncthreads();
    if (threadIdx.x == 0) s_.n_list = 0;
    cl_.sync();  // the list's memory has been read
    SaPart p = nothing();
    pass([&](const float (&v)[8], int c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(v[j] > -INFINITY)) continue;
        const u64 r = rank_of(v[j], c + j);
        if (r > top0 || r < bottom0) continue;
        const int b = bin(r, v[j]);
        if (b < lo) {
          if (by_mass) p.mass += weight(v[j]);
        } else if (b <= hi) {
          p.hi = max(p.hi, r);
          p.lo = min(p.lo, r);
          if (fits) append(r);
        }
      }
    });
    p = exchange(p);
    base += by_mass ? p.mass : n_above;
    if (fits || p.hi == 0) break;
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
    const u64 top1 = top, bottom1 = bottom;
    clear_hist();
    pass([&](const float (&v)[8], int c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(v[j] > -INFINITY)) continue;
        const u64 r = rank_of(v[j], c + j);
        if (r <= top1 && r >= bottom1)
          atomicAdd(&s_.hist[shift >= 0 ? int((top1 - r) >> shift) : bin_below(vt, v[j], scale)], 1u);
      }
    });
    total_hist(s_.tot2);
    tot = s_.tot2;
  }
  const int n = gather_sorted();
  if (me_ == 0) {
    if (by_mass) {
      u64 r[4], cum[4];
      const u64 before = running_mass(n, base, r, cum);
      pick(n, before, r, cum, target);
    } else if (threadIdx.x == 0 && n > 0) {
      s_.res_rank = s_.list[min(max(int(target - base), 1), n) - 1];
    }
  }
  share_result();
}

template <typename T>
__device__ void Sampler<T>::run() {
  const int plane = a_.slice / 8;
  // Pass 1: the logits come in (and stay, if they fit); maximum, least live
  // value, number of live ones.
  float m = -INFINITY, least = INFINITY;
  int mi = 0, n_live = 0;
  constexpr int UN = 4;  // pieces in flight
  for (int c0 = s0_ + int(threadIdx.x) * 8; c0 < s1_; c0 += SA_THREADS * 8 * UN) {
    SaRaw<T> r[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (c0 + k * SA_THREADS * 8 < s1_) r[k] = fetch(c0 + k * SA_THREADS * 8);
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int c = c0 + k * SA_THREADS * 8;
      if (c >= s1_) continue;
      if (a_.resident) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) store_[i * plane + (c - s0_) / 8] = r[k].v[i];
      }
      float v[8];
      raw_values<T>(r[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (v[j] > -INFINITY) {
          ++n_live;
          least = fminf(least, v[j]);
          if (v[j] > m) {
            m = v[j];
            mi = c + j;
          }
        }
      }
    }
  }
  SaPart p = nothing();
  p.n = n_live;
  p.least = least;
  if (n_live > 0) p.hi = rank_of(m, mi);
  p = exchange(p);
  const bool lead = me_ == 0 && threadIdx.x == 0;
  if (p.n == 0) {
    if (lead) {
      a_.token[row_] = -1;
      if (a_.logp != nullptr) a_.logp[row_] = 0.f;
    }
    return;
  }
  const u64 best = p.hi;
  const int live = p.n;
  max_ = rank_value(best);

  const float temp = a_.temperature == nullptr ? 1.f : a_.temperature[row_];
  const int k = a_.top_k == nullptr ? 0 : a_.top_k[row_];
  const float tp = a_.top_p == nullptr ? 1.f : a_.top_p[row_];
  const float mp = a_.min_p == nullptr ? 0.f : a_.min_p[row_];
  const float u = fminf(fmaxf(a_.u[row_], 0.f), 1.f - 0x1p-24f);
  const bool greedy = !(temp > 0.f) || k == 1 || live == 1;
  const bool use_k = k > 0 && k < live, use_p = tp < 1.f, use_m = mp > 0.f;
  const bool need_z = !greedy && !use_k && (use_p || !use_m);
  c_ = 1.4426950408889634074 / double(temp);
  // Bins over 40 T: a weight changes by 2 % across one, and those past the
  // end (the last bin) are below half a unit, exactly 0.
  bin_scale_ = scale_for(fminf(below(p.least), 40.f * temp));

  // Pass 2: counts by bin, the sum behind logp, the total mass.
  p = nothing();
  if (!greedy) clear_hist();
  if (!greedy || a_.logp != nullptr) {
    const int skip = rank_index(best);
    pass([&](const float (&v)[8], int c) {
      float tail = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(v[j] > -INFINITY)) continue;
        if (c + j != skip) tail += ex2_approx(-below(v[j]) * 1.44269504f);
        if (!greedy) atomicAdd(&s_.hist[bin_of(v[j])], 1u);
        if (need_z) p.mass += weight(v[j]);
      }
      p.tail += double(tail);
    });
    p = exchange(p);
  }
  const u64 z = p.mass;
  const double lse = log1p(p.tail);  // log sum exp(l - max)
  u64 token = best;
  if (!greedy) {
    total_hist(s_.tot);
    const double thr = use_m && mp < 1.f ? double(temp) * log(double(mp)) : 0.0;
    auto above_min = [&](float l) { return -(l == max_ ? 0.0 : double(max_) - double(l)) >= thr; };
    // Which ranks can the first filter (or the draw itself) reach?
    const bool by_mass = !use_k;
    u64 target;
    if (use_k) target = u64(k);
    else if (use_p) target = max(u64(1), min(z, u64(ceil(double(tp) * double(z)))));
    else target = part_of(double(u), z) + 1;
    bool in_list;
    int last_bin;
    if (!use_k && !use_p && use_m) {
      last_bin = int(min(floor(-thr * (1.0 + 0x1p-20) * double(bin_scale_)) + 1.0,
                         double(SA_BINS - 1)));
      u64 n = 0;
      for (int i = 0; i < 4; ++i)
        if (int(threadIdx.x) * 4 + i <= last_bin) n += s_.tot[threadIdx.x * 4 + i];
      n = scan(n, s_.warp_sum[0]);
      if (threadIdx.x == SA_THREADS - 1) s_.n_in = uint32_t(n);
      __syncthreads();
      in_list = s_.n_in <= SA_CAP;
    } else {
      bracket(s_.tot, by_mass, target, [&](int b, bool up) { return edge(b, up, max_, bin_scale_); });
      last_bin = s_.hi_bin;
      in_list = s_.n_above + s_.n_in <= SA_CAP;
    }
    if (in_list) {
      // Everything that can be kept fits the list: the first CTA finishes.
      if (threadIdx.x == 0) s_.n_list = 0;
      __syncthreads();
      pass([&](const float (&v)[8], int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v[j] > -INFINITY && bin_of(v[j]) <= last_bin) append(rank_of(v[j], c + j));
      });
      const int n = gather_sorted();
      if (me_ == 0) {
        u64 r[4], cum[4];
        const u64 before = running_mass(n, 0, r, cum);
        u64 keep = z;  // mass of the kept ranks
        if (use_k) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (int(threadIdx.x) * 4 + i == min(k, n) - 1) s_.res_cum = cum[i];
          __syncthreads();
          keep = s_.res_cum;
        }
        if (use_p) {
          const u64 t = max(u64(1), min(keep, u64(ceil(double(tp) * double(keep)))));
          pick(n, before, r, cum, t);
          keep = min(keep, s_.res_cum);
        }
        if (use_m) {
          __syncthreads();
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // the last rank above the threshold
            const int q = threadIdx.x * 4 + i;
            const bool in = q < n && above_min(rank_value(r[i]));
            const bool next = q + 1 < n && above_min(rank_value(s_.list[q + 1]));
            if (in && !next) s_.res_cum = cum[i];
          }
          __syncthreads();
          keep = use_k || use_p ? min(keep, s_.res_cum) : s_.res_cum;
        }
        pick(n, before, r, cum, part_of(double(u), keep) + 1);
        token = s_.res_rank;
      }
    } else {
      u64 keep = z;
      if (use_k) {
        find(false, u64(k));
        const u64 cut = s_.res_rank;
        keep = mass_of([&](float l, int i) { return rank_of(l, i) >= cut; });
      }
      if (use_p) {
        find(true, max(u64(1), min(keep, u64(ceil(double(tp) * double(keep))))));
        keep = min(keep, s_.res_cum);
      }
      if (use_m) {
        const u64 w = mass_of([&](float l, int) { return above_min(l); });
        keep = use_k || use_p ? min(keep, w) : w;
      }
      find(true, part_of(double(u), keep) + 1);
      token = s_.res_rank;
    }
  }
  if (lead) {
    a_.token[row_] = rank_index(token);
    if (a_.logp != nullptr) a_.logp[row_] = float(-double(below(rank_value(token))) - lse);
  }
  cl_.sync();  // shared memory stays until every CTA has read it
}

template <typename T>
__global__ void __launch_bounds__(SA_THREADS) sample_kernel(SampleArgs a) {
  extern __shared__ uint4 sa_store[];
  __shared__ SaShared s;
  Sampler<T> sampler(a, s, sa_store);
  __syncthreads();
  sampler.run();
}

}  // namespace cce
