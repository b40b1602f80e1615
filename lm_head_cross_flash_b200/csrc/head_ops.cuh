// head_ops.cuh — host side of the operators around the head (the last part of
// include/cce.h): argument checks and launches.  Included once, by cce.cu,
// behind the helpers it shares with the head's own entry points.
#pragma once

#include "fp8_mm.cuh"
#include "kept.cuh"
#include "row_ops.cuh"
#include "sample.cuh"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxQuantD = int64_t(1) << 16;
// A row lives in the registers of at most 512 threads, 4 pieces of 8 each.
constexpr int64_t kMaxNormD = 512 * 4 * 8;

bool dtype_ok(cce_dtype t) { return t == CCE_F32 || t == CCE_BF16; }
int64_t dtype_bytes(cce_dtype t) { return t == CCE_F32 ? 4 : 2; }
bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Rows of `ld` elements of `bytes` each that all start on a 16-byte boundary.
bool rows16(const void* p, int64_t ld, int64_t bytes) {
  return aligned_to(p, 16) && ld * bytes % 16 == 0;
}

cce_status check_matrix(const void* p, cce_dtype t, int64_t rows, int64_t cols, int64_t ld) {
  if (p == nullptr || !dtype_ok(t) || rows <= 0 || cols <= 0 || ld < cols)
    return CCE_ERR_INVALID_ARGUMENT;
  if (!aligned_to(p, uintptr_t(dtype_bytes(t)))) return CCE_ERR_INVALID_ARGUMENT;
  if (rows > kMaxRows || cols > kMaxRows || ld > (int64_t(1) << 32)) return CCE_ERR_UNSUPPORTED;
  return CCE_OK;
}

cce_status check_codes(const void* q, int64_t ldq, const float* s, int64_t cols) {
  if (q == nullptr || s == nullptr || ldq < cols || !aligned_to(s, 4))
    return CCE_ERR_INVALID_ARGUMENT;
  return ldq > (int64_t(1) << 32) ? CCE_ERR_UNSUPPORTED : CCE_OK;
}

bool codes8(const void* q, int64_t ldq) { return aligned_to(q, 8) && ldq % 8 == 0; }
QMat qmat(const void* q, int64_t ldq, const float* s, int64_t cols) {
  QMat m;
  m.q = static_cast<uint8_t*>(const_cast<void*>(q));
  m.ldq = ldq;
  m.s = const_cast<float*>(s);
  m.lds = ceil_div(cols, QGROUP);
  return m;
}

// Calls f with the types and the team shape (threads per row, pieces per
// thread) of a row of D elements.
template <typename T>
struct Tag { using type = T; };
template <int V>
using Int = std::integral_constant<int, V>;

template <typename F>
void with_type(cce_dtype t, F f) {
  if (t == CCE_F32) f(Tag<float>());
  else f(Tag<__nv_bfloat16>());
}
template <typename F>
void with_bool(bool b, F f) {
  if (b) f(std::true_type());
  else f(std::false_type());
}
// Unaligned rows (vec false) take one of three shapes only.
template <bool VEC, typename F>
void with_team(int64_t D, F f) {
  const int64_t n8 = ceil_div(D, 8);
  if (n8 <= 32) return f(Int<32>(), Int<1>());
  if constexpr (VEC) {
    if (n8 <= 64) return f(Int<64>(), Int<1>());
    if (n8 <= 128) return f(Int<128>(), Int<1>());
  }
  if (n8 <= 256) return f(Int<256>(), Int<1>());
  if constexpr (VEC) {
    if (n8 <= 512) return f(Int<512>(), Int<1>());
    if (n8 <= 1024) return f(Int<512>(), Int<2>());
  }
  f(Int<512>(), Int<4>());
}

// Blocks of the norm's kernels, for aligned rows or not: what runs at once.
template <bool VEC>
int norm_blocks(int64_t M, int64_t D) {
  int64_t rpb = 1, per_sm = 1;
  with_team<VEC>(D, [&](auto tpr, auto r) {
    rpb = norm_block(tpr()) / tpr();
    per_sm = norm_per_sm(tpr(), r());
  });
  return int(std::max<int64_t>(1, std::min<int64_t>(ceil_div(M, rpb), per_sm * sm_count_guess())));
}

// 8-bit matrix [rows, K] in boxes of one group by `box_rows` rows; bytes
// behind K are not read (zero fill).
bool make_fp8_map(CUtensorMap* m, const void* p, int64_t rows, int64_t K, int64_t ld,
                  uint32_t box_rows) {
  const uint64_t dims[2] = {uint64_t(K), uint64_t(rows)};
  const uint64_t strides[1] = {uint64_t(ld)};
  const uint32_t box[2] = {QGROUP, box_rows};
  return make_map_ex(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename K>
cce_status set_smem_once(K kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CCE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (!done[dev] && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bytes) != cudaSuccess)
    return CCE_ERR_CUDA;
  done[dev] = true;
  return CCE_OK;
}

// Few rows: CTAs per tile of 128 head rows, a power of two up to 8, as many
// as still run at once (a head of 4,096 rows has 32 tiles for 148 SMs).
int few_split(int64_t tiles, int64_t G, int sms) {
  int s = 1;
  while (s < 8 && 2 * s * tiles <= sms && 2 * s <= G) s *= 2;
  return s;
}

template <int NP>
cce_status launch_few(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t K, int S,
                      int sms, const Fp8Args& args, cudaStream_t st) {
  static bool done[64];
  using C = FfCfg<NP>;
  const cce_status s = set_smem_once(fp8_few_kernel<NP>, C::SMEM, done);
  if (s != CCE_OK) return s;
  CUtensorMap ma, mb;
  if (!make_fp8_map(&ma, A, args.M, K, lda, NP) || !make_fp8_map(&mb, B, args.N, K, ldb, 128))
    return CCE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S > 1 ? unsigned(args.n_ct * S) : unsigned(std::min(args.n_ct, sms)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(S);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fp8_few_kernel<NP>, ma, mb, args, S) == cudaSuccess
             ? launch_ok()
             : (cudaGetLastError(), CCE_ERR_CUDA);
}

// CTAs (a power of two up to 8) that share a row of logits: as many as run at
// once (two on an SM), down to 8,192 logits a CTA; and at most 2^21 logits.
int sample_cluster(int64_t B, int64_t V, int sms) {
  int c = 1;
  while (c < SA_MAX_CLUSTER && ((c * B <= sms && V > 8192 * c) || V > int64_t(c) << 21)) c *= 2;
  return c;
}

template <typename T, int MODE>
cce_status launch_sample(SampleArgs a, int64_t B, int c, cudaStream_t st) {
  static bool done[64];
  const cce_status s = set_smem_once(sample_kernel<T, MODE>, int(sizeof(SaShared)), done);
  if (s != CCE_OK) return s;
  a.slice = int(ceil_div(ceil_div(int64_t(a.V) + 7, c), SA_SEG)) * SA_SEG;  // + off_
  a.seg_mul = int(ceil_div(a.slice / SA_SEG, SA_MAX_SEGS));
  cudaLaunchConfig_t cfg = {};
  // the search: as many clusters as run at once (one CTA on an SM)
  const int64_t rows = MODE == SA_SEARCH_ONLY
                           ? std::min<int64_t>(B, std::max(1, sm_count_guess() / c)) : B;
  cfg.gridDim = dim3(unsigned(rows) * unsigned(c));
  cfg.blockDim = dim3(SA_THREADS);
  cfg.dynamicSmemBytes = sizeof(SaShared);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(c);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, MODE>, a) == cudaSuccess
             ? launch_ok()
             : (cudaGetLastError(), CCE_ERR_CUDA);
}

// One launch where a row gets nearly as many CTAs as it can use and there are
// few rounds of them (the list alone runs two CTAs on an SM: 4,000 rows of
// 1,000 logits 370 us, 500 in one launch), else two (256
// rows of 262,144 bf16 logits with top-k 50: 62 us with one CTA a row, 82 with
// two, 165 with eight).
template <typename T>
cce_status launch_sample_rows(const SampleArgs& a, int64_t B, cudaStream_t st) {
  const int c = sample_cluster(B, a.V, sm_count_guess());
  const int most = sample_cluster(1, a.V, sm_count_guess());
  if (2 * c >= most && c * B <= 2 * sm_count_guess())
    return launch_sample<T, SA_BOTH>(a, B, c, st);
  const cce_status s = launch_sample<T, SA_LIST_ONLY>(a, B, c, st);
  // Fewer CTAs a row where many rows may be left: 256 rows of 262,144 bf16
  // logits, all of them flat, take 657 us with 2 and 827 with 4; but 61 rows of
  // 128,256, few of them flat, 74 us with 8 and 102 with 2.
  int cs = most;
  while (cs > 1 && cs * B > 4 * sm_count_guess()) cs /= 2;
  return s != CCE_OK ? s : launch_sample<T, SA_SEARCH_ONLY>(a, B, cs, st);
}

}  // namespace

extern "C" {

cce_status cce_fp8_quant_rows(const void* X, cce_dtype x_dtype, int64_t M, int64_t D, int64_t ldx,
                              uint8_t* Q, int64_t ldq, float* S, cce_stream_t stream) {
  cce_status s = check_matrix(X, x_dtype, M, D, ldx);
  if (s == CCE_OK) s = check_codes(Q, ldq, S, D);
  if (s != CCE_OK) return s;
  if (D > kMaxQuantD) return CCE_ERR_UNSUPPORTED;
  const int G = int(ceil_div(D, QGROUP));
  const bool vec = D % 8 == 0 && rows16(X, ldx, dtype_bytes(x_dtype)) && codes8(Q, ldq);
  // Four groups of a half warp under way where every SM still gets four blocks
  // ([16384, 4096] bf16: 41 us, 47 with one; [250, 4096]: 2.9 us, 2.4 with one).
  const int sms = sm_count_guess();
  const bool many = M * G >= int64_t(4) * sms * 64;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(PK_QUANT, st);
  with_type(x_dtype, [&](auto t) {
    using T = typename decltype(t)::type;
    with_bool(vec, [&](auto v) {
      with_bool(many, [&](auto m) {
        constexpr int UN = decltype(m)::value ? 4 : 1;
        const int grid = int(std::min<int64_t>(ceil_div(M * G, 16 * UN), 16 * sms));
        quant_rows_kernel<decltype(v)::value, T, UN><<<grid, 256, 0, st>>>(
            static_cast<const T*>(X), ldx, M, int(D), G, qmat(Q, ldq, S, D));
      });
    });
  });
  return launch_ok();
}

cce_status cce_fp8_quant_blocks(const void* W, cce_dtype w_dtype, int64_t N, int64_t K,
                                int64_t ldw, uint8_t* Q, int64_t ldq, float* S,
                                cce_stream_t stream) {
  cce_status s = check_matrix(W, w_dtype, N, K, ldw);
  if (s == CCE_OK) s = check_codes(Q, ldq, S, K);
  if (s != CCE_OK) return s;
  if (K > kMaxQuantD || ceil_div(N, QGROUP) > 65535) return CCE_ERR_UNSUPPORTED;
  const dim3 grid(unsigned(ceil_div(K, QGROUP)), unsigned(ceil_div(N, QGROUP)));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(PK_QUANT, st);
  const bool vec = K % 8 == 0 && rows16(W, ldw, dtype_bytes(w_dtype)) && codes8(Q, ldq);
  with_type(w_dtype, [&](auto t) {
    using T = typename decltype(t)::type;
    with_bool(vec, [&](auto v) {
      quant_blocks_kernel<decltype(v)::value, T><<<grid, 256, 0, st>>>(
          static_cast<const T*>(W), ldw, N, int(K), qmat(Q, ldq, S, K));
    });
  });
  return launch_ok();
}

cce_status cce_norm_forward(const void* X, cce_dtype x_dtype, int64_t M, int64_t D, int64_t ldx,
                            const void* w, cce_dtype w_dtype, double eps, void* H,
                            cce_dtype h_dtype, int64_t ldh, uint8_t* H8, int64_t ldh8, float* Hs,
                            uint8_t* X8, int64_t ldx8, float* Xs, float* rstd,
                            cce_stream_t stream) {
  cce_status s = check_matrix(X, x_dtype, M, D, ldx);
  if (s == CCE_OK) s = check_matrix(w, w_dtype, 1, D, D);
  if (s == CCE_OK && H != nullptr) s = check_matrix(H, h_dtype, M, D, ldh);
  if (s == CCE_OK && (H8 != nullptr || Hs != nullptr)) s = check_codes(H8, ldh8, Hs, D);
  if (s == CCE_OK && (X8 != nullptr || Xs != nullptr)) s = check_codes(X8, ldx8, Xs, D);
  if (s != CCE_OK) return s;
  if (!(eps >= 0.0) || eps > 1e30 || (rstd != nullptr && !aligned_to(rstd, 4)) ||
      (H == nullptr && H8 == nullptr && X8 == nullptr && rstd == nullptr))
    return CCE_ERR_INVALID_ARGUMENT;
  if (D > kMaxNormD) return CCE_ERR_UNSUPPORTED;
  NormFwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = X;
  a.ldx = ldx;
  a.w = w;
  a.w_bf16 = w_dtype == CCE_BF16;
  a.M = M;
  a.D = int(D);
  a.inv_d = float(1.0 / double(D));
  a.eps = float(eps);
  a.h = H;
  a.ldh = ldh;
  const bool vec = D % 8 == 0 && rows16(X, ldx, dtype_bytes(x_dtype)) && aligned_to(w, 16) &&
                   (H == nullptr || rows16(H, ldh, dtype_bytes(h_dtype))) &&
                   (H8 == nullptr || codes8(H8, ldh8)) && (X8 == nullptr || codes8(X8, ldx8));
  if (H8 != nullptr) a.h8 = qmat(H8, ldh8, Hs, D);
  if (X8 != nullptr) a.x8 = qmat(X8, ldx8, Xs, D);
  a.rstd = rstd;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(PK_NORM, st);
  with_type(x_dtype, [&](auto tx) {
    with_type(H != nullptr ? h_dtype : CCE_BF16, [&](auto th) {
      with_bool(vec, [&](auto v) {
        with_team<decltype(v)::value>(D, [&](auto tpr, auto r) {
          constexpr int T = decltype(tpr)::value, B = norm_block(T);
          norm_fwd_kernel<decltype(v)::value, typename decltype(tx)::type,
                          typename decltype(th)::type, T, decltype(r)::value>
              <<<norm_blocks<decltype(v)::value>(M, D), B, 0, st>>>(a);
        });
      });
    });
  });
  return launch_ok();
}

size_t cce_norm_backward_workspace_bytes(int64_t M, int64_t D) {
  if (M <= 0 || D <= 0 || M > kMaxRows || D > kMaxNormD) return 0;
  // one part of dW for each block, of whichever form the rows' alignment asks for
  return kStatusBytes + size_t(std::max(norm_blocks<true>(M, D), norm_blocks<false>(M, D))) *
                            size_t(D) * 4;
}

cce_status cce_norm_backward(const uint8_t* X8, int64_t ldx8, const float* Xs, const float* rstd,
                             int64_t M, int64_t D, const void* w, cce_dtype w_dtype,
                             const void* dH, cce_dtype dh_dtype, int64_t lddh, void* dX,
                             cce_dtype dx_dtype, int64_t lddx, float* dW, void* ws,
                             size_t ws_bytes, cce_stream_t stream) {
  cce_status s = check_matrix(dH, dh_dtype, M, D, lddh);
  if (s == CCE_OK) s = check_matrix(dX, dx_dtype, M, D, lddx);
  if (s == CCE_OK) s = check_matrix(w, w_dtype, 1, D, D);
  if (s == CCE_OK) s = check_codes(X8, ldx8, Xs, D);
  if (s != CCE_OK) return s;
  if (rstd == nullptr || !aligned_to(rstd, 4)) return CCE_ERR_INVALID_ARGUMENT;
  if (D > kMaxNormD) return CCE_ERR_UNSUPPORTED;
  if (dW != nullptr) {
    if (ws == nullptr || !aligned16(ws) || !aligned_to(dW, 4)) return CCE_ERR_INVALID_ARGUMENT;
    if (ws_bytes < cce_norm_backward_workspace_bytes(M, D)) return CCE_ERR_WORKSPACE_TOO_SMALL;
  }
  NormBwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x8 = qmat(X8, ldx8, Xs, D);
  a.rstd = rstd;
  a.w = w;
  a.w_bf16 = w_dtype == CCE_BF16;
  a.dh = dH;
  a.lddh = lddh;
  a.M = M;
  a.D = int(D);
  a.inv_d = float(1.0 / double(D));
  a.dx = dX;
  a.lddx = lddx;
  const bool vec = D % 8 == 0 && rows16(dH, lddh, dtype_bytes(dh_dtype)) &&
                   rows16(dX, lddx, dtype_bytes(dx_dtype)) && aligned_to(w, 16) &&
                   codes8(X8, ldx8);
  if (dW != nullptr)
    a.dw_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  const int grid = vec ? norm_blocks<true>(M, D) : norm_blocks<false>(M, D);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(PK_NORM, st);
  with_type(dx_dtype, [&](auto tx) {
    with_type(dh_dtype, [&](auto th) {
      with_bool(vec, [&](auto v) {
        with_team<decltype(v)::value>(D, [&](auto tpr, auto r) {
          constexpr int T = decltype(tpr)::value;
          norm_bwd_kernel<decltype(v)::value, typename decltype(tx)::type,
                          typename decltype(th)::type, T, decltype(r)::value>
              <<<grid, norm_block(T), 0, st>>>(a);
        });
      });
    });
  });
  if (launch_ok() != CCE_OK) return CCE_ERR_CUDA;
  if (dW != nullptr)
    norm_dw_kernel<<<unsigned(ceil_div(D, 32)), 1024, 0, st>>>(a.dw_part, grid, int(D), dW);
  return launch_ok();
}

cce_status cce_fp8_matmul(const uint8_t* A, int64_t lda, const float* SA, const uint8_t* B,
                          int64_t ldb, const float* SB, int64_t M, int64_t N, int64_t K, void* C,
                          cce_dtype c_dtype, int64_t ldc, void* ws, size_t ws_bytes,
                          cce_stream_t stream) {
  cce_status s = check_matrix(C, c_dtype, M, N, ldc);
  if (s != CCE_OK) return s;
  if (K <= 0) return CCE_ERR_INVALID_ARGUMENT;
  if (M == 1) lda = int64_t(ceil_div(K, 16)) * 16;  // the stride of a single row says nothing
  if (N == 1) ldb = int64_t(ceil_div(K, 16)) * 16;
  s = check_codes(A, lda, SA, K);
  if (s == CCE_OK) s = check_codes(B, ldb, SB, K);
  if (s != CCE_OK) return s;
  if (!aligned16(A) || !aligned16(B) || lda % 16 != 0 || ldb % 16 != 0 || ws == nullptr ||
      !aligned16(ws))
    return CCE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < kStatusBytes) return CCE_ERR_WORKSPACE_TOO_SMALL;
  if (K > kMaxQuantD || ceil_div(M, 128) * ceil_div(N, 128) >= int64_t(1) << 31)
    return CCE_ERR_UNSUPPORTED;
  int sms = 0;
  s = device_info(&sms);
  if (s != CCE_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Fp8Args a;
  std::memset(&a, 0, sizeof(a));
  a.M = int(M);
  a.N = int(N);
  a.G = int(ceil_div(K, QGROUP));
  a.sa = SA;
  a.sb = SB;
  a.c = C;
  a.ldc = ldc;
  a.c_bf16 = c_dtype == CCE_BF16;
  a.vec = rows16(C, ldc, dtype_bytes(c_dtype));
  a.wait_ns = g_wait_ns.load();
  a.status = status_word(ws);
  ProfScope ps(PK_FP8, st);
  const int64_t np = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t tiles = ceil_div(N, 128);
  const int S = few_split(tiles, a.G, sms);
  if (M <= 128 && np * ceil_div(a.G, S) <= FF_MAX_SCALES) {
    a.n_ct = int(tiles);
    switch (np) {
      case 16: return launch_few<16>(A, lda, B, ldb, K, S, sms, a, st);
      case 32: return launch_few<32>(A, lda, B, ldb, K, S, sms, a, st);
      case 64: return launch_few<64>(A, lda, B, ldb, K, S, sms, a, st);
      default: return launch_few<128>(A, lda, B, ldb, K, S, sms, a, st);
    }
  }
  static bool done[64];
  s = set_smem_once(fp8_rows_kernel, F8_SMEM, done);
  if (s != CCE_OK) return s;
  // The kernel's register hand-over waits for ever if it was compiled to fewer
  // registers than it counts on; the build checks the same.
  static Kept kept_regs;
  int regs = 0;
  if (!kept_regs.get(
          [](int* n) {
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, fp8_rows_kernel) != cudaSuccess) {
              cudaGetLastError();
              return false;
            }
            *n = fa.numRegs;
            return true;
          },
          &regs))
    return CCE_ERR_CUDA;
  if (regs != F8_REGS) return CCE_ERR_UNSUPPORTED;
  a.n_rt = int(ceil_div(M, 2 * F8_BM));
  a.n_ct = int(ceil_div(N, F8_BN));
  // row tiles of one raster group: 48 MB of A, so that a group stays in L2
  // while the columns pass
  a.group_rt = int(std::max<int64_t>(
      1, std::min<int64_t>(a.n_rt, (int64_t(48) << 20) / (2 * F8_BM * K))));
  CUtensorMap ma, mb;
  if (!make_fp8_map(&ma, A, M, K, lda, F8_BM) || !make_fp8_map(&mb, B, N, K, ldb, F8_BN / 2))
    return CCE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * grid_for(int64_t(a.n_rt) * a.n_ct, sms / 2));
  cfg.blockDim = dim3(F8_THREADS);
  cfg.dynamicSmemBytes = F8_SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_rows_kernel, ma, mb, a) == cudaSuccess
             ? launch_ok()
             : (cudaGetLastError(), CCE_ERR_CUDA);
}

cce_status cce_sample_rows(const void* logits, cce_dtype dtype, int64_t B, int64_t V, int64_t ld,
                           const float* temperature, const int32_t* top_k, const float* top_p,
                           const float* min_p, const float* u, int32_t* tokens, float* logp,
                           cce_stream_t stream) {
  const cce_status s = check_matrix(logits, dtype, B, V, ld);
  if (s != CCE_OK) return s;
  if (u == nullptr || tokens == nullptr) return CCE_ERR_INVALID_ARGUMENT;
  for (const void* p : {static_cast<const void*>(temperature), static_cast<const void*>(top_k),
                        static_cast<const void*>(top_p), static_cast<const void*>(min_p),
                        static_cast<const void*>(u), static_cast<const void*>(tokens),
                        static_cast<const void*>(logp)})
    if (!aligned_to(p, 4)) return CCE_ERR_INVALID_ARGUMENT;
  if (V > (int64_t(1) << 24) || B > (int64_t(1) << 24)) return CCE_ERR_UNSUPPORTED;
  SampleArgs a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.ld = ld;
  a.B = int(B);
  a.V = int(V);
  int log2v = 0;
  while ((int64_t(1) << log2v) < V) ++log2v;
  a.bits = std::min(45, 63 - log2v);  // a row's mass stays below 2^63
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.token = tokens;
  a.logp = logp;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(PK_SAMPLE, st);
  return dtype == CCE_F32 ? launch_sample_rows<float>(a, B, st)
                          : launch_sample_rows<__nv_bfloat16>(a, B, st);
}

}  // extern "C"
