// row_ops.cuh — the bandwidth-bound operators around the head: 8-bit
// quantisation (rows in groups of 128, weights in 128x128 blocks) and the
// final norm, forward with an 8-bit checkpoint of its input and backward from
// that checkpoint.
//
// Format.  A group holds e4m3 codes q and one fp32 scale s; its values are
// q * s.  With m = max(|x|) over the group, at least 2^-90 so that nothing
// below leaves the fp32 range,
//   s = m * (1 / 448),  q = e4m3(x * (448 * (1 / m))),
// the quotients and the products rounded in fp32, the code rounded to nearest
// even and saturated.  e4m3 keeps the relative error of every element above
// m * 2^-15 within 2^-4, where an 8-bit integer would lose the small elements
// of a group that holds an outlier.  A NaN stays a NaN; a group that holds an
// infinity restores as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "ptx.cuh"

namespace cce {

constexpr int QGROUP = 128;
constexpr float E4M3_MAX = 448.f;
constexpr float E4M3_INV = 1.f / 448.f;
constexpr float QAMAX_MIN = 8.077935669463161e-28f;  // 2^-90

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else return __float2bfloat16_rn(x);
}

// Eight consecutive elements of a row as fp32, from column c < n on; columns
// at or past n give 0.  VEC: every row starts on a 16-byte boundary (8 for
// codes) and n is a multiple of 8.  It is a template parameter so that a
// thread's loads carry no branches and are all in flight together (the 128 x
// 128 quantiser of a [73440, 1536] bf16 head: 64 us; 166 us with a test at run
// time).
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* __restrict__ p, int c, int n, float (&v)[8]) {
  if constexpr (VEC) {
    if constexpr (std::is_same_v<T, float>) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + c));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p + c + 4));
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p + c));
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? to_f32(p[c + i]) : 0.f;
  }
}

// The same eight elements as they lie in memory, for loads that run ahead.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* __restrict__ p, int c, int n) {
  Raw8<T> r;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
      r.v[i] = __ldg(reinterpret_cast<const uint4*>(p + c) + i);
  } else {
    uint32_t w[2 * sizeof(T)] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(p[c + i]);
        else w[i / 2] |= uint32_t(__bfloat16_as_ushort(p[c + i])) << (16 * (i & 1));
      }
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
      r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void open8(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) {
    const uint32_t u[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[4 * i + j] = __uint_as_float(u[j]);
      } else {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    }
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, int c, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    if constexpr (std::is_same_v<T, float>) {
      *reinterpret_cast<float4*>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p + c) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) p[c + i] = from_f32<T>(v[i]);
  }
}

// Eight e4m3 codes of v * inv.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(v[2 * i], inv), __fmul_rn(v[2 * i + 1], inv)), __NV_SATFINITE,
        __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* __restrict__ p, int c, int n, uint2 q) {
  if constexpr (VEC) {
    *reinterpret_cast<uint2*>(p + c) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) p[c + i] = uint8_t((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

// Eight codes; columns at or past n give 0.
template <bool VEC>
__device__ __forceinline__ uint2 load_codes8(const uint8_t* __restrict__ p, int c, int n) {
  if constexpr (VEC) return __ldg(reinterpret_cast<const uint2*>(p + c));
  uint2 q = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) {
      const uint32_t b = p[c + i];
      if (i < 4) q.x |= b << (8 * i);
      else q.y |= b << (8 * (i - 4));
    }
  return q;
}

// Their values, unscaled.
__device__ __forceinline__ void code_values8(uint2 q, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = ((i < 2 ? q.x : q.y) >> (16 * (i & 1))) & 0xFFFFu;
    const __half2_raw hr =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    const float2 f = __half22float2(__half2(hr));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
// Maximum over the 16 lanes that hold one group.
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return fmaxf(m, QAMAX_MIN);
}

// A strided matrix of 8-bit codes with its scales.
struct QMat {
  uint8_t* q;
  int64_t ldq;  // bytes
  float* s;
  int64_t lds;  // elements
};

__device__ __forceinline__ float code_factor(float m) {
  return __fmul_rn(E4M3_MAX, __frcp_rn(m));
}

// Codes and scale of the group that the 16 lanes of this half warp hold.
template <bool VEC>
__device__ __forceinline__ void quant_group(const QMat& o, int64_t row, int c, int n,
                                            const float (&v)[8]) {
  const float m = group_max(amax8(v));
  if (c < n) {
    store_codes8<VEC>(o.q + row * o.ldq, c, n, codes8(v, code_factor(m)));
    if ((c & (QGROUP - 1)) == 0) o.s[row * o.lds + c / QGROUP] = __fmul_rn(m, E4M3_INV);
  }
}

// ------------------------------------------------------------ quant rows --
// A half warp takes one group: 16 lanes x 8 elements, UN groups under way at
// once.  Reads each element once; bound by bandwidth.
template <bool VEC, typename T, int UN>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, int64_t ldx,
                                                         int64_t M, int D, int G, QMat o) {
  const int64_t n = M * G;
  const int lane8 = (threadIdx.x & 15) * 8;
  // whole warps stay together: group_max shuffles over the full warp
  for (int64_t u0 = int64_t(blockIdx.x) * (16 * UN) + (threadIdx.x >> 5) * 2; u0 < n;
       u0 += int64_t(gridDim.x) * (16 * UN)) {
    Raw8<T> r[UN];
    int64_t row[UN];
    int c[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int64_t u = u0 + 16 * k + ((threadIdx.x >> 4) & 1);
      row[k] = u / G;
      c[k] = u < n ? int(u - row[k] * G) * QGROUP + lane8 : D;
      r[k] = Raw8<T>();
      if (c[k] < D) r[k] = raw8<VEC>(x + row[k] * ldx, c[k], D);
    }
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      float v[8];
      open8<T>(r[k], v);
      quant_group<VEC>(o, row[k], c[k], D, v);
    }
  }
}

// ---------------------------------------------------------- quant blocks --
// One CTA per 128x128 block: 256 threads hold 8 rows x 8 elements each (the
// block is read once and stays in registers).  [73440, 1536] bf16: 64 us, 5.3
// TB/s.
template <bool VEC, typename T>
__global__ void __launch_bounds__(256) quant_blocks_kernel(const T* __restrict__ x, int64_t ldx,
                                                           int64_t N, int K, QMat o) {
  const int g = blockIdx.x;
  const int64_t r0 = int64_t(blockIdx.y) * QGROUP;
  const int c = g * QGROUP + (threadIdx.x & 15) * 8;
  const int64_t row0 = r0 + (threadIdx.x >> 4);
  float v[8][8] = {};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i;
    if (row < N && c < K) load8<VEC>(x + row * ldx, c, K, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  __shared__ float sm[8];
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, sm[i]);
  m = fmaxf(m, QAMAX_MIN);
  const float inv = code_factor(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i;
    if (row < N && c < K) store_codes8<VEC>(o.q + row * o.ldq, c, K, codes8(v[i], inv));
  }
  if (threadIdx.x == 0) o.s[blockIdx.y * o.lds + g] = __fmul_rn(m, E4M3_INV);
}

// ------------------------------------------------------------------ norm --
// Sum over the TPR threads of one row; every thread of the block calls it.
// Two buffers taken in turn, so one barrier a sum is enough.
template <int TPR, int WARPS>
__device__ __forceinline__ float team_sum(float s, float (&sm)[2][WARPS], int turn) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, w0 = warp & ~(TPR / 32 - 1);
    if ((threadIdx.x & 31) == 0) sm[turn & 1][warp] = s;
    __syncthreads();
    s = sm[turn & 1][w0 + (threadIdx.x & (TPR / 32 - 1))];
#pragma unroll
    for (int off = TPR / 64; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  }
  return s;
}

struct NormFwdArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  int w_bf16;
  int64_t M;
  int D;
  float inv_d, eps;
  void* h;       // null: not wanted
  int64_t ldh;
  QMat h8, x8;   // q null: not wanted
  float* rstd;   // null: not wanted
};

template <bool VEC>
__device__ __forceinline__ void load_w8(const void* w, int bf16, int c, int n, float (&v)[8]) {
  if (bf16) load8<VEC>(static_cast<const __nv_bfloat16*>(w), c, n, v);
  else load8<VEC>(static_cast<const float*>(w), c, n, v);
}

constexpr int norm_block(int tpr) { return tpr > 256 ? tpr : 256; }
// Blocks that share an SM where a thread has one piece of the row: 1,024
// threads of 64 registers, or 768 of 80 where the block's teams also meet.
constexpr int norm_per_sm(int tpr, int r) {
  return r > 1 ? 1 : tpr < 256 ? 3 : 1024 / norm_block(tpr);
}

// h = x * rstd * w with rstd = 1 / sqrt(mean(x^2) + eps), all in fp32.  TPR
// threads hold a row in registers (R pieces of 8 elements each), so x is read
// once; the codes of x and of h come from the same registers.  A block takes
// row after row, the next one on its way while the current one is summed.
// [8192, 2048] bf16 to H and checkpoint 19 us (4.4 TB/s), [32768, 4096] 135 us
// (5.0 TB/s); bound by its instructions, 213 a warp and 256 elements (with
// IEEE quotients in every thread and the weights read again for each row, 273
// and 162 us).
template <bool VEC, typename T, typename TH, int TPR, int R>
__global__ void __launch_bounds__(norm_block(TPR), norm_per_sm(TPR, R))
    norm_fwd_kernel(const __grid_constant__ NormFwdArgs a) {
  constexpr int RPB = norm_block(TPR) / TPR;
  __shared__ float sm[2][norm_block(TPR) / 32];
  const int t = threadIdx.x % TPR;
  // One piece a thread: the weights stay in registers too.
  constexpr bool KEEP = R == 1;
  float w[R][8];
  if constexpr (KEEP) {
    if (t * 8 < a.D) load_w8<VEC>(a.w, a.w_bf16, t * 8, a.D, w[0]);
  }
  Raw8<T> x[R];
  const int64_t step = int64_t(gridDim.x) * RPB;
  int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
  const T* src = static_cast<const T*>(a.x) + row * a.ldx;  // of the next fetch
  auto fetch = [&](bool live) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + t) * 8;
      x[i] = Raw8<T>();
      if (live && c < a.D) x[i] = raw8<VEC>(src, c, a.D);
    }
    src += step * a.ldx;
  };
  fetch(row < a.M);
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < a.M; row0 += step, row += step, ++turn) {
    const bool live = row < a.M;
    float v[R][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      open8<T>(x[i], v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    fetch(row + step < a.M);
    ss = team_sum<TPR>(ss, sm, turn);
    const float rstd = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + t) * 8;
      const int cl = live ? c : a.D;  // nothing is stored behind the last row
      if (a.x8.q != nullptr) quant_group<VEC>(a.x8, row, cl, a.D, v[i]);
      if (a.h == nullptr && a.h8.q == nullptr) continue;
      float h[8] = {};
      if (cl < a.D) {
        if constexpr (!KEEP) load_w8<VEC>(a.w, a.w_bf16, c, a.D, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = v[i][j] * rstd * w[i][j];
        if (a.h != nullptr) store8<VEC>(static_cast<TH*>(a.h) + row * a.ldh, c, a.D, h);
      }
      if (a.h8.q != nullptr) quant_group<VEC>(a.h8, row, cl, a.D, h);
    }
  }
}

struct NormBwdArgs {
  QMat x8;
  const float* rstd;
  const void* w;
  int w_bf16;
  const void* dh;
  int64_t lddh;
  int64_t M;
  int D;
  float inv_d;
  void* dx;
  int64_t lddx;
  float* dw_part;  // [gridDim.x, D] or null
};

// With n = q * s * rstd (the normalised row restored from the checkpoint) and
// g = dh * w:
//   dx = rstd * (g - n * mean(g * n)),   dw = sum over the rows of dh * n.
// A row stays in registers between its sum and its output, so each input is
// read once.  Every thread keeps the dw terms of its own columns in registers
// over all of its rows; the blocks' parts are added in a fixed order by
// norm_dw_kernel, so dw does not depend on timing.
// The next row's loads are issued before the current row's sum.  [32768, 4096]
// with fp32 dH 157 us (6.0 TB/s, 92 % of the measured copy rate); 244 us while
// its registers let one block of 512 threads onto an SM instead of two.  Rows
// wider than 8,192 take four pieces a thread, whose weights, dw terms and next
// row do not fit 128 registers: 304 to 856 bytes of spills a thread, [4096,
// 16384] 232 us (2.0 TB/s; [4096, 8192] 45 us, 5.3 TB/s), 350 where rows are not
// aligned.
template <bool VEC, typename TX, typename TH, int TPR, int R>
__global__ void __launch_bounds__(norm_block(TPR), norm_per_sm(TPR, R))
    norm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
  constexpr int RPB = norm_block(TPR) / TPR;
  __shared__ float sm[2][norm_block(TPR) / 32];
  __shared__ float sw[RPB > 1 ? (RPB - 1) * TPR * R * 8 : 1];
  const int t = threadIdx.x % TPR;
  float w[R][8], dw[R][8] = {};
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = (i * TPR + t) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = 0.f;
    if (c < a.D) load_w8<VEC>(a.w, a.w_bf16, c, a.D, w[i]);
  }
  // one row as it comes from memory
  uint2 q[R];
  Raw8<TH> dh[R];
  float sc[R], rstd;
  auto fetch = [&](int64_t row) {
    const bool live = row < a.M;
    rstd = live ? __ldg(a.rstd + row) : 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + t) * 8;
      q[i] = make_uint2(0, 0);
      sc[i] = 0.f;
      dh[i] = Raw8<TH>();
      if (live && c < a.D) {
        q[i] = load_codes8<VEC>(a.x8.q + row * a.x8.ldq, c, a.D);
        dh[i] = raw8<VEC>(static_cast<const TH*>(a.dh) + row * a.lddh, c, a.D);
        sc[i] = __ldg(a.x8.s + row * a.x8.lds + c / QGROUP);
      }
    }
  };
  const int64_t step = int64_t(gridDim.x) * RPB;
  int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
  fetch(row);
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < a.M; row0 += step, row += step, ++turn) {
    float n[R][8], h[R][8];
    const float r = rstd;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float k = sc[i] * r;
      float g[8];
      code_values8(q[i], n[i]);
      open8<TH>(dh[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[i][j] *= k;
        dw[i][j] = fmaf(g[j], n[i][j], dw[i][j]);
        h[i][j] = g[j] * w[i][j];
        dot = fmaf(h[i][j], n[i][j], dot);
      }
    }
    fetch(row + step);
    dot = team_sum<TPR>(dot, sm, turn) * a.inv_d;
    if (row < a.M) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int c = (i * TPR + t) * 8;
        if (c < a.D) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = r * fmaf(-n[i][j], dot, h[i][j]);
          store8<VEC>(static_cast<TX*>(a.dx) + row * a.lddx, c, a.D, h[i]);
        }
      }
    }
  }
  if (a.dw_part == nullptr) return;
  if constexpr (RPB > 1) {
    const int team = threadIdx.x / TPR;
    if (team > 0) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sw[(((team - 1) * R + i) * 8 + j) * TPR + t] = dw[i][j];
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int k = 0; k < RPB - 1; ++k)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] += sw[((k * R + i) * 8 + j) * TPR + t];
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = (i * TPR + t) * 8;
    if (c < a.D) store8<VEC>(a.dw_part + size_t(blockIdx.x) * a.D, c, a.D, dw[i]);
  }
}

// dw[d] = sum over p of part[p, d]: 32 columns a block, 32 slices of the parts
// a column, each in order, then the slices in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int P, int D,
                                                       float* __restrict__ dw) {
  __shared__ float sm[32][33];
  const int d = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float s = 0.f;
  if (d < D) {
    int p = k;
    for (; p + 96 < P; p += 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldg(part + size_t(p + 32 * i) * D + d);
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; p < P; p += 32) s += __ldg(part + size_t(p) * D + d);
  }
  sm[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k == 0 && d < D) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sm[i][threadIdx.x];
    dw[d] = s;
  }
}

}  // namespace cce
