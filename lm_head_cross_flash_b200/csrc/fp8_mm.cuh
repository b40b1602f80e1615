// fp8_mm.cuh — the product of 8-bit rows and an 8-bit head,
//   C[m,n] = sum_g sa[m,g] sb[n/128,g] sum_{k in group g} a[m,k] b[n,k],
// on the 8-bit tensor-core path (tcgen05.mma.kind::f8f6f4, e4m3 operands,
// fp32 accumulation).
//
// The scales differ from one group of 128 to the next, so a group's partial
// sum (4 MMAs of K = 32) is taken out of tensor memory and added, times its
// scales, to fp32 sums in registers.  That costs one tensor-memory read and
// one FMA per partial; both run beside the next group's MMAs.
//
// fp8_rows_kernel: any number of rows; 256 x 256 tiles of C by CTA pairs, row
//   tiles fastest, so the CTAs in flight share the same rows of b.
// fp8_few_kernel: up to 128 rows (decoding).  The roles of the operands are
//   exchanged: 128 rows of b are the MMA's M side and the few rows of a its N
//   side, so a pass over b costs no idle tensor rows; the CTAs of a cluster
//   split the groups where the head has too few rows to fill the SMs.
#pragma once

#include "row_ops.cuh"

namespace cce {

// kind::f8f6f4, e4m3 x e4m3, fp32 accumulator, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void umma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 16 consecutive fp32 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// tcgen05.wait::ld that names the registers it waits for.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

struct Fp8Args {
  int M, N;
  int G;  // groups of K
  const float* sa;  // [M, G]
  const float* sb;  // [ceil(N/128), G]
  void* c;
  int64_t ldc;
  int c_bf16;
  int vec;         // rows of c start on 16-byte boundaries
  int n_rt, n_ct;  // row and column tiles
  int group_rt;    // row tiles per raster group
  uint64_t wait_ns;
  uint32_t* status;
};

// Barriers and flags at the end of shared memory.
template <int NST, int NBUF>
struct Fp8Sync {
  uint64_t full[NST], empty[NST];
  uint64_t acc_full[NBUF], acc_empty[NBUF];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

// Every copy that was issued lands before the CTA may exit.
template <int NST>
__device__ __forceinline__ void drain_copies(uint64_t* full, uint32_t mask, uint32_t phases) {
  for (int s = 0; s < NST; ++s)
    if (mask & (1u << s)) wait_bounded(&full[s], (phases >> s) & 1u, 1000000000ull, nullptr);
}

// ----------------------------------------------------------- many rows --
// A pair of CTAs makes a 256 x 256 tile with tcgen05.mma.cta_group::2: each
// CTA loads its 128 rows of a and half of the 256 rows of b, so a group costs
// it 32 KB of shared-memory writes and as much of reads (48 KB each for 128 x
// 256 tiles of single CTAs, whose 768 cycles of shared memory stood against
// 512 of MMAs).  Both copies complete on the leader's barrier, only the leader
// issues MMAs; no copy is multicast.
//
// Warps 0 and 1 copy and issue; warps 4 to 11 drain, one row and 128 columns
// (one 128-block of b, so one scale) a thread.  128 sums and two buffers of 32
// partials need more registers than an even share, so the first warpgroup
// hands its own over (setmaxnreg: 128 * 56 + 256 * 224 = 384 * 168).
//
// What bounds it (2048 x 18944 x 4096, codes and scales constant): 135 us in
// all, 105 with the partials left alone, 105 with the MMAs left out, so each
// side is near the other's time and the hand-over between them is what is
// left.  With real codes and scales 177 us in a long run, at 1.47 GHz under the
// power cap.  2048 x 128256 x 4096: 1013 us cold, 1190 in a long run.  Measured
// against this form when it took 1013: fma.rn.f32 instead of f32x2 1255 us,
// tiles of 256 x 128 with four accumulators 1343, halves of 128 columns with
// accumulators of their own 1148, sixteen draining warps 1614 (the instructions
// that are not FMAs add up).
constexpr int F8_BM = 128, F8_BN = 256, F8_BK = 128;
constexpr int F8_STAGES = 5;
constexpr int F8_STAGE = (F8_BM + F8_BN / 2) * F8_BK;
constexpr int F8_THREADS = 384;
constexpr int F8_REGS = 168, F8_REGS_ISSUE = 56, F8_REGS_DRAIN = 224;
static_assert(128 * F8_REGS_ISSUE + 256 * F8_REGS_DRAIN <= F8_THREADS * F8_REGS, "registers");
constexpr int F8_OUT = 8 * 32 * 128;  // a 32 x 128-byte block for each draining warp
using F8Sync = Fp8Sync<F8_STAGES, 2>;
constexpr int F8_SMEM = F8_STAGES * F8_STAGE + F8_OUT + sizeof(F8Sync) + 1024;

__device__ __forceinline__ void umma_e4m3_ss2(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the pair leader's barrier without a fence of cluster scope: what
// is handed over is tensor memory whose reads have completed
// (tcgen05.wait::ld), no memory.  With .release.cluster the draining warps
// spent a third of their time in that fence (2048 x 128256 x 4096: 1890 us).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Two FMAs at once: c += (lo, hi) * s2.
__device__ __forceinline__ void fma2(uint64_t& c, uint32_t lo, uint32_t hi, uint64_t s2) {
  asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tfma.rn.f32x2 %0, x, %3, %0;\n\t}"
      : "+l"(c)
      : "r"(lo), "r"(hi), "l"(s2));
}
__device__ __forceinline__ float2 unpack2(uint64_t c) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(c));
  return f;
}

// 32 rows x (128 / sizeof(T)) columns of a warp go out through shared memory:
// each lane writes its row (16-byte pieces, swizzled by row), then the warp
// writes rows of C in whole 128-byte lines.
template <typename T>
__device__ __forceinline__ void store_block(const Fp8Args& a, uint8_t* sm, int row0, int col0,
                                            const uint4 (&piece)[8]) {
  const int lane = threadIdx.x & 31;
  constexpr int NC = 128 / sizeof(T);
  T* const c = static_cast<T*>(a.c);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(sm + lane * 128 + ((i ^ (lane & 7)) << 4)) = piece[i];
  __syncwarp();
  if (a.vec && col0 + NC <= a.N) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3), k = lane & 7;
      const uint4 v = *reinterpret_cast<const uint4*>(sm + r * 128 + ((k ^ (r & 7)) << 4));
      if (row0 + r < a.M)
        *reinterpret_cast<uint4*>(c + (row0 + r) * a.ldc + col0 + k * (16 / sizeof(T))) = v;
    }
  } else {
    const int rows = min(32, a.M - row0);
#pragma unroll
    for (int h = 0; h < NC / 32; ++h) {
      const int j = h * 32 + lane, at = j * int(sizeof(T));
      T* const p = c + row0 * a.ldc + col0 + j;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8) {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = *reinterpret_cast<const T*>(sm + (r0 + i) * 128 + (((at >> 4) ^ i) << 4) + (at & 15));
        T* q = p + r0 * a.ldc;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += a.ldc)
          if (r0 + i < rows && col0 + j < a.N) *q = v[i];
      }
    }
  }
  __syncwarp();
}

__global__ void __launch_bounds__(F8_THREADS, 1)
    fp8_rows_kernel(const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Fp8Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const out = base + F8_STAGES * F8_STAGE;
  F8Sync* sy = reinterpret_cast<F8Sync*>(out + F8_OUT);
  volatile int* abort_flag = &sy->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_ctarank());
  const int ntiles = a.n_rt * a.n_ct;
  const int tile0 = int(cluster_id_x()), tstep = int(cluster_count_x());

  if (threadIdx.x == 0) {
    for (int s = 0; s < F8_STAGES; ++s) {
      mbar_init(&sy->full[s], 1);
      mbar_init(&sy->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sy->acc_full[b], 1);
      mbar_init(&sy->acc_empty[b], 16);  // the draining warps of both CTAs
    }
    mbar_init(&sy->drain, 1);
    sy->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc2(&sy->tmem, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised
  tc_fence_after();
  const uint32_t tmem = sy->tmem;

  // Row tiles fastest inside a group of row tiles that stays in L2.
  auto tile_at = [&](int t, int& rt, int& ct) {
    const int per_group = a.group_rt * a.n_ct;
    const int grp = t / per_group, r = t - grp * per_group;
    const int g0 = grp * a.group_rt, gn = min(a.group_rt, a.n_rt - g0);
    rt = g0 + r % gn;
    ct = r / gn;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8_REGS_ISSUE));
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0, mask = 0, phases = 0;
      bool ok = true;
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_normal();
      for (int t = tile0; t < ntiles && ok; t += tstep) {
        int rt, ct;
        tile_at(t, rt, ct);
        for (int g = 0; g < a.G; ++g) {
          if (!wait_bounded(&sy->empty[stage], phase ^ 1u, a.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* s = base + stage * F8_STAGE;
          const uint32_t bar = mapa_shared(smem_u32(&sy->full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&sy->full[stage], 2 * F8_STAGE);
          tma_load_2d_pair(s, &tmA, bar, g * F8_BK, (rt * 2 + rank) * F8_BM, keep);
          tma_load_2d_pair(s + F8_BM * F8_BK, &tmB, bar, g * F8_BK,
                           ct * F8_BN + rank * (F8_BN / 2), once);
          mask |= 1u << stage;
          phases = (phases & ~(1u << stage)) | (phase << stage);
          if (++stage == F8_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        set_status(a.status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      // the leader's barriers count the other CTA's copies too
      if (rank == 0) drain_copies<F8_STAGES>(sy->full, mask, phases);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_e4m3(2 * F8_BM, F8_BN);
      int stage = 0;
      uint32_t phase = 0, acc = 0;
      bool ok = true;
      for (int t = tile0; t < ntiles && ok; t += tstep) {
        for (int g = 0; g < a.G; ++g, ++acc) {
          const int b = acc & 1;
          // the accumulator comes back last: everything else is done by then
          if (!wait_bounded(&sy->full[stage], phase, a.wait_ns, abort_flag) ||
              !wait_bounded(&sy->acc_empty[b], ((acc >> 1) & 1) ^ 1u, a.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = smem_u32(base + stage * F8_STAGE), sB = sA + F8_BM * F8_BK;
#pragma unroll
          for (int j = 0; j < F8_BK / 32; ++j)
            umma_e4m3_ss2(tmem + b * F8_BN, sdesc_sw128(sA + j * 32, 16, 1024),
                          sdesc_sw128(sB + j * 32, 16, 1024), idesc, j != 0);
          umma_commit2_mc(&sy->acc_full[b], 0x3);
          umma_commit2_mc(&sy->empty[stage], 0x3);
          if (++stage == F8_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        set_status(a.status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      // the MMAs of this thread complete before tensor memory is released
      umma_commit2_mc(&sy->drain, 0x1);
      wait_bounded(&sy->drain, 0, 1000000000ull, nullptr);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F8_REGS_DRAIN));
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
    uint8_t* const sm = out + (warp - 4) * 4096;
    const uint32_t empty0 = mapa_shared(smem_u32(&sy->acc_empty[0]), 0);
    const uint32_t empty1 = mapa_shared(smem_u32(&sy->acc_empty[1]), 0);
    uint32_t acc = 0;
    for (int t = tile0; t < ntiles; t += tstep) {
      int rt, ct;
      tile_at(t, rt, ct);
      const int row0 = (rt * 2 + rank) * F8_BM + quad * 32, col = ct * F8_BN + half * 128;
      const float* psa = a.sa + static_cast<size_t>(min(row0 + lane, a.M - 1)) * a.G;
      const float* psb = a.sb + static_cast<size_t>(min(col, a.N - 1) / QGROUP) * a.G;
      uint64_t c[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) c[j] = 0;
      float sa = __ldg(psa), sb = __ldg(psb);
      bool ok = true;
      for (int g = 0; g < a.G; ++g, ++acc) {
        const int b = acc & 1;
        const float s = sa * sb;
        uint64_t s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
        const int gn = min(g + 1, a.G - 1);
        sa = __ldg(psa + gn);
        sb = __ldg(psb + gn);
        if (!wait_bounded(&sy->acc_full[b], (acc >> 1) & 1, a.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(taddr + b * F8_BN, r[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tmem_ld_wait(r[i & 1]);
          if (i < 3) {
            tmem_ld32(taddr + b * F8_BN + (i + 1) * 32, r[(i + 1) & 1]);
          } else {
            tc_fence_before();  // all of the partial sums are in registers
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(b ? empty1 : empty0);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(c[i * 16 + j], r[i & 1][2 * j], r[i & 1][2 * j + 1], s2);
        }
      }
      if (!ok) {
        if (lane == 0) {
          set_status(a.status, ST_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      if (row0 >= a.M || col >= a.N) continue;
      if (a.c_bf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 piece[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = unpack2(c[h * 32 + i * 4 + j]);
              const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
              w[j] = *reinterpret_cast<const uint32_t*>(&p);
            }
            piece[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          store_block<__nv_bfloat16>(a, sm, row0, col + h * 64, piece);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint4 piece[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = unpack2(c[h * 16 + i * 2]), e = unpack2(c[h * 16 + i * 2 + 1]);
            piece[i] = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y),
                                  __float_as_uint(e.x), __float_as_uint(e.y));
          }
          store_block<float>(a, sm, row0, col + h * 32, piece);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // a CTA stays until both are done with each other's barriers and memory
  cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

// ------------------------------------------------------------- few rows --
// NP: rows of a, padded (16, 32, 64, 128).  A stage holds 128 rows of b and
// the NP rows of a for one group; four accumulators of NP columns.  N = 128256,
// K = 4096: 87.5 us with one row (6.0 TB/s, 91 % of the measured copy rate),
// 114 to 125 us with 64, 160 with 128; N = 73440, K = 1536 to fp32: 24 us with 16
// rows, 29 us with 61, 42 with 128.  The form for 128 rows spills 64 bytes a
// thread (64 sums and as many partials in 168 registers), the others none.
// More stages (8 to 12 instead of 6 to 8) changed nothing.
constexpr int FF_MAX_SCALES = 8192;  // NP * groups per CTA, kept in shared memory
template <int NP>
struct FfCfg {
  static constexpr int STAGE = (128 + NP) * 128;
  static constexpr int SCALES = FF_MAX_SCALES * 4;
  static constexpr int NST = (NP <= 64 ? 160 : 176) * 1024 / STAGE;
  static constexpr int NBUF = 4;
  static constexpr int COLS = NBUF * NP < 32 ? 32 : NBUF * NP;
  static constexpr int HALVES = NP >= 64 ? 2 : 1;  // warps that share a lane quarter
  static constexpr int NC = NP / HALVES;           // columns per thread
  static constexpr int THREADS = 64 + HALVES * 128;
  using Sync = Fp8Sync<NST, NBUF>;
  static constexpr int SMEM = NST * STAGE + SCALES + int(sizeof(Sync)) + 1024;
  static_assert(NST * STAGE >= 128 * NP * 4, "the stages hold a tile's sums");
};

// One tile of 128 rows of b per cluster and round; CTA `rank` of the cluster
// takes the groups [rank*G/S, (rank+1)*G/S).  With S > 1 every cluster has one
// tile, and the CTAs' sums meet in shared memory: each CTA adds one share of
// the columns over all of them, in the order of the ranks.
template <int NP>
__global__ void __launch_bounds__(FfCfg<NP>::THREADS, 1)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmA,
                   const __grid_constant__ CUtensorMap tmB, Fp8Args a, int S) {
  using C = FfCfg<NP>;
  constexpr int NST = C::NST, NBUF = C::NBUF, NC = C::NC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(base + NST * C::STAGE);  // [groups, NP]
  typename C::Sync* sy = reinterpret_cast<typename C::Sync*>(base + NST * C::STAGE + C::SCALES);
  volatile int* abort_flag = &sy->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = S > 1 ? int(cluster_ctarank()) : 0;
  const int tile0 = S > 1 ? int(blockIdx.x) / S : int(blockIdx.x);
  const int tstep = S > 1 ? a.n_ct : int(gridDim.x);
  const int g0 = rank * a.G / S, ng = (rank + 1) * a.G / S - g0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sy->full[s], 1);
      mbar_init(&sy->empty[s], 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&sy->acc_full[b], 1);
      mbar_init(&sy->acc_empty[b], C::HALVES * 4);
    }
    mbar_init(&sy->drain, 1);
    sy->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sy->tmem, C::COLS);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < ng * NP; i += C::THREADS) {
    const int m = i / ng, g = i - m * ng;
    scales[g * NP + m] = m < a.M ? __ldg(a.sa + static_cast<size_t>(m) * a.G + g0 + g) : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy->tmem;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, mask = 0, phases = 0;
      bool ok = true;
      const uint64_t keep = l2_policy_evict_last(), stream = l2_policy_evict_first();
      for (int t = tile0; t < a.n_ct && ok; t += tstep) {
        for (int g = 0; g < ng; ++g) {
          if (!wait_bounded(&sy->empty[stage], phase ^ 1u, a.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* s = base + stage * C::STAGE;
          mbar_arrive_expect_tx(&sy->full[stage], C::STAGE);
          tma_load_2d_hint(s, &tmB, &sy->full[stage], (g0 + g) * 128, t * 128, stream);
          tma_load_2d_hint(s + 128 * 128, &tmA, &sy->full[stage], (g0 + g) * 128, 0, keep);
          mask |= 1u << stage;
          phases = (phases & ~(1u << stage)) | (phase << stage);
          if (++stage == NST) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        set_status(a.status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      drain_copies<NST>(sy->full, mask, phases);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(128, NP);
      int stage = 0;
      uint32_t phase = 0, acc = 0;
      bool ok = true;
      for (int t = tile0; t < a.n_ct && ok; t += tstep) {
        for (int g = 0; g < ng; ++g, ++acc) {
          const int b = acc % NBUF;
          if (!wait_bounded(&sy->acc_empty[b], ((acc / NBUF) & 1) ^ 1u, a.wait_ns, abort_flag) ||
              !wait_bounded(&sy->full[stage], phase, a.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sB = smem_u32(base + stage * C::STAGE), sA = sB + 128 * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_e4m3_ss(tmem + b * NP, sdesc_sw128(sB + j * 32, 16, 1024),
                         sdesc_sw128(sA + j * 32, 16, 1024), idesc, j != 0);
          umma_commit(&sy->empty[stage]);
          umma_commit(&sy->acc_full[b]);
          if (++stage == NST) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        set_status(a.status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      umma_commit(&sy->drain);
      wait_bounded(&sy->drain, 0, 1000000000ull, nullptr);
    }
  } else {
    // One row of b (one column of C) and NC rows of C per thread.
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int vrow = quad * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * NC;
    uint32_t acc = 0;
    bool ok = true;
    for (int t = tile0; t < a.n_ct && ok; t += tstep) {
      const float* psb = a.sb + static_cast<size_t>(t) * a.G + g0;
      float c[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) c[j] = 0.f;
      float nb = ng > 0 ? __ldg(psb) : 0.f;
      for (int g = 0; g < ng; ++g, ++acc) {
        const int b = acc % NBUF;
        const float sb = nb;
        nb = __ldg(psb + min(g + 1, ng - 1));
        if (!wait_bounded(&sy->acc_full[b], (acc / NBUF) & 1, a.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float4* sg = reinterpret_cast<const float4*>(scales + g * NP + half * NC);
        uint32_t r[NC / 16][16];
#pragma unroll
        for (int i = 0; i < NC / 16; ++i) tmem_ld16(taddr + b * NP + i * 16, r[i]);
#pragma unroll
        for (int i = 0; i < NC / 16; ++i) {
          tmem_ld_wait16(r[i]);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 s = sg[i * 4 + j / 4];
            c[i * 16 + j] = fmaf(__uint_as_float(r[i][j]), s.x * sb, c[i * 16 + j]);
            c[i * 16 + j + 1] = fmaf(__uint_as_float(r[i][j + 1]), s.y * sb, c[i * 16 + j + 1]);
            c[i * 16 + j + 2] = fmaf(__uint_as_float(r[i][j + 2]), s.z * sb, c[i * 16 + j + 2]);
            c[i * 16 + j + 3] = fmaf(__uint_as_float(r[i][j + 3]), s.w * sb, c[i * 16 + j + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sy->acc_empty[b]);
      }
      if (!ok) {
        if (lane == 0) {
          set_status(a.status, ST_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      if (S == 1) {
        const int n = t * 128 + vrow, m0 = half * NC;
        if (n < a.N) {
          if (a.c_bf16) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.c) + m0 * a.ldc + n;
#pragma unroll
            for (int j = 0; j < NC; ++j, out += a.ldc)
              if (m0 + j < a.M) *out = __float2bfloat16_rn(c[j]);
          } else {
            float* out = static_cast<float*>(a.c) + m0 * a.ldc + n;
#pragma unroll
            for (int j = 0; j < NC; ++j, out += a.ldc)
              if (m0 + j < a.M) *out = c[j];
          }
        }
      } else {
        // the stages are free: all of this CTA's MMAs have been waited for
        float* part = reinterpret_cast<float*>(base);
#pragma unroll
        for (int j = 0; j < NC; ++j) part[(half * NC + j) * 128 + vrow] = c[j];
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (S > 1) {
    cluster_sync_all();
    const uint32_t part = smem_u32(base);
    const int m0 = rank * NP / S, m1 = (rank + 1) * NP / S;
    for (int i = threadIdx.x; i < (m1 - m0) * 128; i += C::THREADS) {
      const int m = m0 + (i >> 7), v = i & 127, n = tile0 * 128 + v;
      float s = 0.f;
      for (int r = 0; r < S; ++r) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(x)
                     : "r"(mapa_shared(part + (m * 128 + v) * 4, r))
                     : "memory");
        s += x;
      }
      if (m < a.M && n < a.N) {
        if (a.c_bf16)
          static_cast<__nv_bfloat16*>(a.c)[m * a.ldc + n] = __float2bfloat16_rn(s);
        else
          static_cast<float*>(a.c)[m * a.ldc + n] = s;
      }
    }
    cluster_sync_all();  // the sums stay until every CTA has read them
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

}  // namespace cce
