// Entry points of the 8-bit feed-forward operators declared in include/fp8q.h: per-row INT8
// quantization, INT8 products, and the gated projections with their backward pass.  Part of
// library.cu's translation unit (after fp8q.cu, whose host helpers it uses).
#include <algorithm>

#include "gated.cuh"
#include "int8.cuh"
#include "skinny.cuh"

namespace {

using fp8q::GatedArgs;
using fp8q::GatedBwdArgs;
using fp8q::Int8Args;
using fp8q::SkinnyArgs;

// CTAs of `kern` that fit the current device at once; sets its shared memory limit on first
// use.  0 on failure.
template <auto kern>
int resident_ctas(int threads, uint32_t smem) {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_acquire);
  if (n) return n;
  int sms = 0, per_sm = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
          cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess || per_sm <= 0) {
    (void)cudaGetLastError();   // handled here, not by the next launch check
    return 0;
  }
  n = sms * per_sm;
  cached[dev].store(n, std::memory_order_release);
  return n;
}

constexpr int64_t kMaxTiles = 0x7FFF0000;   // 32-bit tile indices, with room for a grid more

int launched() { return cudaGetLastError() == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA; }

template <typename... Params>
int launch_clusters(void (*kern)(Params...), int64_t grid, int cluster, int threads, uint32_t smem,
                    cudaStream_t stream, const Params&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return FP8Q_OK;
  (void)cudaGetLastError();   // reported here, not by the next launch check
  return FP8Q_ERR_CUDA;
}

constexpr int64_t kInt8MaxK = 131071;   // K 128^2 <= 2^31 - 1: the INT32 sums are exact

int check_int8(const int8_t* A, const float* sA, const int8_t* B, const float* sB, const void* C, int out_dtype,
               int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc) {
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (out_dtype != FP8Q_OUT_BF16 && out_dtype != FP8Q_OUT_FP32) return FP8Q_ERR_UNSUPPORTED;
  if (!A || !sA || !B || !sB || !C) return FP8Q_ERR_NULL;
  if (N == 0 || K == 0 || K > kInt8MaxK || M > 0x3FFFFFFF || N > 0x3FFFFFFF) return FP8Q_ERR_SHAPE;
  if (lda < K || ldb < K || ldc < N) return FP8Q_ERR_SHAPE;
  if (lda % 16 != 0 || ldb % 16 != 0 || !aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 4) || !aligned(sB, 4) ||
      !aligned(C, out_dtype == FP8Q_OUT_BF16 ? 2 : 4))
    return FP8Q_ERR_ALIGN;
  return FP8Q_OK;
}

// Tiling of the wide INT8 kernel: CTA pairs or single CTAs, and columns of B per tile, by the
// least time over all waves.  A tile's time per 128 K-elements, in ns, fitted to measurements
// with 4096 x 7168 x 7168: single CTAs 204 / 229 / 300 / 360 for widths 64, 128, 192 and 256 (up to
// 64 bytes a cycle from L2), pairs 207 / 221 / 264 / 330.
struct Int8Tiling {
  bool pair;
  int width;
};

Int8Tiling int8_tiling(int64_t M, int64_t rows, bool gated, int sms) {
  const int step = gated ? 64 : 32;
  Int8Tiling best{false, 256};
  int64_t best_cost = INT64_MAX;
  for (int pair = 0; pair < 2; ++pair) {
    const int64_t mt = pair ? (M + 255) / 256 : (M + 127) / 128;
    const int units = pair ? sms / 2 : sms;
    for (int w = 256; w >= step; w -= step) {
      const int64_t waves = (mt * ((rows + w - 1) / w) + units - 1) / units;
      const int64_t cost = waves * (pair ? std::max(20700, 11000 + 86 * w) : std::max(20400, 9500 + 105 * w));
      if (cost < best_cost) best = {pair != 0, w}, best_cost = cost;
    }
  }
  return best;
}

// Launch of the few-row kernel: `units` tiles of MP rows, K split over clusters of
// `split` CTAs.
template <int KIND, bool GATED, bool OUT_BF16, int MP>
int launch_skinny(const CUtensorMap& tmA, const CUtensorMap& tmW, const SkinnyArgs& a, int64_t units,
                  cudaStream_t stream) {
  using Cfg = fp8q::SkinnyCfg<KIND, MP>;
  static constexpr auto kern = fp8q::gemm_skinny_kernel<KIND, GATED, OUT_BF16, MP>;
  if (resident_ctas<kern>(Cfg::kThreads, Cfg::smem_bytes) <= 0) return FP8Q_ERR_CUDA;
  return launch_clusters(kern, units * a.split, a.split, Cfg::kThreads, Cfg::smem_bytes, stream, tmA, tmW, a);
}

// Rows of A per tile: the smallest that holds M, or the largest.
int skinny_rows(int64_t M, int most) {
  int mp = 16;
  while (mp < M && mp < most) mp *= 2;
  return mp;
}

// CTAs per cluster: as many as still fit two to an SM, at most four.  (16 x 7168 x 7168 INT8,
// 56 tiles: 22.0 / 15.2 / 14.9 / 14.1 us for 1 to 4; 16.3, 18.0 and 17.6 us for 5, 6 and 8:
// wider clusters leave SMs of a GPC without work.)
int skinny_split(int64_t units, int64_t G, int sms) {
  int s = fp8q::kMaxSplit;
  while (s > 1 && (units * s > 2 * sms || s > G)) s /= 2;
  return s;
}

int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_acquire);
  if (n) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cached[dev].store(n, std::memory_order_release);
  return n;
}

// Whether the few-row kernel takes the product: always up to 64 rows, and up to 512 while the wide
// kernel would leave most SMs idle (INT8: its 128 x 128 tiles half of them, and beyond 128 rows K
// has to be long enough to be split; FP8: its 128 x 256 tiles three quarters).
// us, few-row / wide:
//   INT8 N 7168 K 7168        128 rows 16.2 / 17.5, 192 19.6 / 16.8, 256 20.9 / 17.4
//   INT8 N 28672 K 2048       64 rows 17.0 / 16.6, 128 20.5 / 17.0
//   INT8 N 2048 K 1496        128 rows 6.7 / 7.1, 256 8.0 / 7.3;   N 512 K 7168, 512 rows 10.1 / 15.1
//   INT8 gated N 2048 K 7168  128 rows 12.4 / 15.7, 256 15.6 / 15.8, 384 17.7 / 16.7
//   FP8 gated N 2048 K 7168   64 rows 11.5 / 30.8, 256 22.2 / 31.4, 384 37.2 / 31.5
// and against the wide kernel for power-of-two scales:
//   N 2048 K 7168             64 rows 12.0 / 25.7, 256 22.1 / 26.2;   N 4096, 128 rows 22.4 / 26.9
//   N 1024 K 2048             64 rows 6.5 / 10.0, 256 9.0 / 10.3, 512 11.1 / 10.6
//   N 512 K 7168              256 rows 10.6 / 23.0, 512 15.0 / 24.6
bool few_rows(int64_t M, int64_t rows, int64_t G, int sms, bool fp8) {
  if (M <= 64) return true;
  if (M > 512) return false;
  const int64_t mt = (M + 127) / 128;
  if (fp8) return mt * ((rows + 255) / 256) * 4 <= sms;
  return mt * ((rows + 127) / 128) * 2 <= sms && (M <= 128 || G >= 32);
}

// Fills in the tiling of the few-row kernel; returns its tile count, or 0 on failure.
template <bool GATED>
int64_t plan_skinny(SkinnyArgs* a, int mp, int sms) {
  const int cols = GATED ? 64 : 128;
  const int64_t nt = (a->N + cols - 1) / cols, units = nt * ((a->M + mp - 1) / mp);
  if (units * fp8q::kMaxSplit > kMaxTiles) return 0;
  a->nt = static_cast<int>(nt);
  a->split = skinny_split(units, a->G, sms);
  return units;
}

template <bool GATED, bool OUT_BF16>
int run_int8_skinny(const int8_t* A, const float* sA, const int8_t* B, const float* sB, void* C, int64_t M, int64_t N,
                    int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int sms, cudaStream_t stream) {
  constexpr int KIND = fp8q::kSkinnyInt8;
  const int mp = skinny_rows(M, 128);
  SkinnyArgs a{};
  a.sA = sA; a.sB = sB; a.C = C; a.ldc = ldc; a.M = M; a.N = N; a.G = static_cast<int>((K + 127) / 128);
  const int64_t units = plan_skinny<GATED>(&a, mp, sms);
  if (units == 0) return FP8Q_ERR_SHAPE;
  constexpr int kVecBytes = OUT_BF16 ? 8 : 16;
  a.vec = (ldc * (OUT_BF16 ? 2 : 4)) % kVecBytes == 0 && aligned(C, kVecBytes);
  CUtensorMap tmA, tmW;
  int st = encode_operand(&tmA, A, K, M, lda, mp);
  if (st != FP8Q_OK || (st = encode_operand(&tmW, B, K, GATED ? 2 * N : N, ldb, GATED ? 64 : 128)) != FP8Q_OK) return st;
  switch (mp) {
    case 16: return launch_skinny<KIND, GATED, OUT_BF16, 16>(tmA, tmW, a, units, stream);
    case 32: return launch_skinny<KIND, GATED, OUT_BF16, 32>(tmA, tmW, a, units, stream);
    case 64: return launch_skinny<KIND, GATED, OUT_BF16, 64>(tmA, tmW, a, units, stream);
    default: return launch_skinny<KIND, GATED, OUT_BF16, 128>(tmA, tmW, a, units, stream);
  }
}

template <bool GATED, bool OUT_BF16, bool PAIR>
int launch_int8(const CUtensorMap& tmA, const CUtensorMap& tmB, Int8Args a, int sms, cudaStream_t stream) {
  using Cfg = fp8q::Int8Cfg<PAIR>;
  static constexpr auto kern = fp8q::gemm_int8_kernel<GATED, OUT_BF16, PAIR>;
  if (resident_ctas<kern>(Cfg::kThreads, Cfg::smem_bytes) <= 0) return FP8Q_ERR_CUDA;
  a.stages = Cfg::stages(a.width);
  const int64_t tiles = static_cast<int64_t>(a.mt) * a.nt;
  constexpr int cg = PAIR ? 2 : 1;
  const int64_t units = tiles < sms / cg ? tiles : sms / cg;
  return launch_clusters(kern, units * cg, cg, Cfg::kThreads, Cfg::smem_bytes, stream, tmA, tmB, a);
}

template <bool GATED, bool OUT_BF16>
int run_int8(const int8_t* A, const float* sA, const int8_t* B, const float* sB, void* C, int64_t M, int64_t N,
             int64_t K, int64_t lda, int64_t ldb, int64_t ldc, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return FP8Q_ERR_CUDA;
  const int64_t rows = GATED ? 2 * N : N;
  if (few_rows(M, rows, (K + 127) / 128, sms, false))
    return run_int8_skinny<GATED, OUT_BF16>(A, sA, B, sB, C, M, N, K, lda, ldb, ldc, sms, stream);
  const Int8Tiling t = int8_tiling(M, rows, GATED, sms);
  Int8Args a{};
  a.sA = sA; a.sB = sB; a.C = C; a.ldc = ldc; a.M = M; a.N = N;
  a.k_groups = static_cast<int>((K + 127) / 128);
  a.width = t.width;
  const int cols = GATED ? a.width / 2 : a.width, tile_m = t.pair ? 256 : 128;
  const int64_t mt = (M + tile_m - 1) / tile_m, nt = (N + cols - 1) / cols;
  if (mt * nt > kMaxTiles) return FP8Q_ERR_SHAPE;
  a.mt = static_cast<int>(mt);
  a.nt = static_cast<int>(nt);
  a.n_fastest = M > rows;
  a.vec = (ldc * (OUT_BF16 ? 2 : 4)) % 16 == 0 && aligned(C, 16);
  CUtensorMap tmA, tmB;
  int st = encode_operand(&tmA, A, K, M, lda, 128);
  // a box of B: the tile's rows of one CTA (gated: of one projection)
  if (st != FP8Q_OK || (st = encode_operand(&tmB, B, K, rows, ldb, GATED || t.pair ? a.width / 2 : a.width)) != FP8Q_OK)
    return st;
  return t.pair ? launch_int8<GATED, OUT_BF16, true>(tmA, tmB, a, sms, stream)
                : launch_int8<GATED, OUT_BF16, false>(tmA, tmB, a, sms, stream);
}

// Buffers of the gated layer, as byte offsets into what the forward pass keeps and into the
// scratch of either direction (each on 256 bytes).
struct GatedLayer {
  int64_t Tp;                                        // T rounded up to 128
  size_t gu, qw, sw, qxt, sxt, kept;                 // kept: g and u; W's codes and scales; X^T's
  size_t qx, sx, forward;                            // forward scratch: X's codes and scales
  size_t qd, sd, qdt, sdt, qwt, swt, ws, ws_bytes, backward;   // backward: D's, D^T's, W^T's; split-K
};

int gated_layer(GatedLayer* l, int64_t T, int64_t N, int64_t K, bool for_dx, bool for_dw, bool pow2) {
  if (T < 0 || N <= 0 || K <= 0 || N % 128 != 0 || K % 128 != 0) return FP8Q_ERR_SHAPE;
  if (T > 0x3FFFFFFF || N > 0x1FFFFFFF || K > 0x3FFFFFFF) return FP8Q_ERR_SHAPE;
  const int64_t R = 2 * N, Tp = (T + 127) / 128 * 128;
  l->Tp = Tp;
  size_t end = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = end;
    end += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return at;
  };
  l->gu = take(2 * T * R);
  l->qw = take(R * K);
  l->sw = take(R / 128 * (K / 128) * 4);
  l->qxt = take(for_dw ? K * Tp : 0);
  l->sxt = take(for_dw ? Tp / 128 * K * 4 : 0);
  l->kept = end;
  end = 0;
  l->qx = take(T * K);
  l->sx = take(K / 128 * T * 4);
  l->forward = end;
  end = 0;
  l->qd = take(T * R);
  l->sd = take(R / 128 * T * 4);
  l->qdt = take(R * Tp);
  l->sdt = take(Tp / 128 * R * 4);
  l->qwt = take(for_dx ? K * R : 0);
  l->swt = take(for_dx ? K / 128 * (R / 128) * 4 : 0);
  // The promoted products may split their last wave along K.  Below 2048 a split saves less than
  // its extra launch costs (a group of 128 takes 0.6 us, the launch 2.5 us).
  l->ws_bytes = 0;
  if (!pow2 && T > 0) {
    size_t dx = 0, dw = 0;
    int st = FP8Q_OK;
    if (for_dx && R >= 2048) st = fp8_gemm_workspace_size(T, K, R, &dx);
    if (st == FP8Q_OK && for_dw && Tp >= 2048) st = fp8_gemm_workspace_size(R, K, Tp, &dw);
    if (st != FP8Q_OK) return st;
    l->ws_bytes = std::max(dx, dw);
  }
  l->ws = take(static_cast<int64_t>(l->ws_bytes));
  l->backward = end;
  return FP8Q_OK;
}

// Tensor map of a bf16 matrix read in tiles of 128 rows x 64 columns, 128-byte swizzle.
bool encode_bf16_tiles(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int64_t ld) {
  auto enc = tensor_map_encoder();
  if (!enc || !bind_current_context()) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pow2: the scales are powers of two; others are reported.
int run_fp8_gated(bool pow2, const uint8_t* A, const float* sA, int64_t ld_sa, const uint8_t* W, const float* sW,
                  void* H, int64_t ldh, void* GU, int64_t ldgu, int64_t M, int64_t N, int64_t K, int64_t lda,
                  int64_t ldw, void* stream) {
  if (M == 0 && N >= 0 && K >= 0) return FP8Q_OK;
  if (N > 0x3FFFFFFF) return FP8Q_ERR_SHAPE;
  int st = check_dense_blockscaled(A, sA, ld_sa, W, sW, 0, FP8Q_BSCALE_BLOCK128x128, H, FP8Q_OUT_BF16, M, N, K, lda,
                                   ldw, ldh);
  if (st != FP8Q_OK) return st;
  if (GU != nullptr) {
    if (ldgu < 2 * N) return FP8Q_ERR_SHAPE;
    if (ldgu % 8 != 0 || !aligned(GU, 16)) return FP8Q_ERR_ALIGN;
  }
  const auto s = static_cast<cudaStream_t>(stream);
  const int sms = sm_count();
  if (sms <= 0) return FP8Q_ERR_CUDA;
  if (few_rows(M, 2 * N, K / 128, sms, true)) {
    constexpr int KIND = fp8q::kSkinnyFp8;
    const int mp = skinny_rows(M, 64);
    SkinnyArgs a{};
    a.sA = sA; a.ld_sa = ld_sa; a.sB = sW; a.C = H; a.ldc = ldh;
    a.gu = static_cast<__nv_bfloat16*>(GU); a.ld_gu = ldgu; a.M = M; a.N = N; a.G = static_cast<int>(K / 128);
    a.vec = 1;
    a.pow2 = pow2;
    const int64_t units = plan_skinny<true>(&a, mp, sms);
    if (units == 0) return FP8Q_ERR_SHAPE;
    CUtensorMap tmA, tmW;
    if ((st = encode_operand(&tmA, A, K, M, lda, mp)) != FP8Q_OK ||
        (st = encode_operand(&tmW, W, K, 2 * N, ldw, 64)) != FP8Q_OK)
      return st;
    switch (mp) {
      case 16: return launch_skinny<KIND, true, true, 16>(tmA, tmW, a, units, s);
      case 32: return launch_skinny<KIND, true, true, 32>(tmA, tmW, a, units, s);
      default: return launch_skinny<KIND, true, true, 64>(tmA, tmW, a, units, s);
    }
  }
  if (pow2) {
    using Cfg = fp8q::Ue8m0Cfg<false, true>;
    static constexpr auto kern = fp8q::gemm_fp8_ue8m0_kernel<false, true, false, true>;
    const int64_t tiles = ((M + Cfg::kTileM - 1) / Cfg::kTileM) * ((N + Cfg::kOutN - 1) / Cfg::kOutN);
    if (tiles > kMaxTiles) return FP8Q_ERR_SHAPE;
    CUtensorMap tmA, tmW;
    if ((st = encode_operand(&tmA, A, K, M, lda, Cfg::kTileM)) != FP8Q_OK ||
        (st = encode_operand(&tmW, W, K, 2 * N, ldw, Cfg::kOutN)) != FP8Q_OK)
      return st;
    GemmArgs a{};
    a.sA = sA; a.ld_sa = ld_sa; a.sB = sW; a.C = H; a.ldc = ldh;
    a.gu = static_cast<__nv_bfloat16*>(GU); a.ld_gu = ldgu;
    a.M = M; a.N = N; a.G = static_cast<int>(K / 128);
    a.n_fastest = M > 2 * N;
    const int units = resident_ctas<kern>(Cfg::kThreads, Cfg::smem_bytes);
    if (units <= 0) return FP8Q_ERR_CUDA;
    kern<<<static_cast<unsigned>(tiles < units ? tiles : units), Cfg::kThreads, Cfg::smem_bytes, s>>>(tmA, tmW, a);
    return launched();
  }
  using Cfg = fp8q::GatedCfg;
  GatedArgs a{};
  a.sA = sA; a.ld_sa = ld_sa; a.sW = sW;
  a.h = static_cast<__nv_bfloat16*>(H); a.ldh = ldh;
  a.gu = static_cast<__nv_bfloat16*>(GU); a.ld_gu = ldgu; a.M = M; a.N = N; a.G = static_cast<int>(K / 128);
  const int64_t mt = (M + Cfg::kTileM - 1) / Cfg::kTileM, nt = (N + Cfg::kTileN - 1) / Cfg::kTileN;
  if (mt * nt > kMaxTiles) return FP8Q_ERR_SHAPE;
  a.mt = static_cast<int>(mt);
  a.nt = static_cast<int>(nt);
  a.n_fastest = M > 2 * N;
  CUtensorMap tmA, tmW;
  if ((st = encode_operand(&tmA, A, K, M, lda, Cfg::kTileM)) != FP8Q_OK ||
      (st = encode_operand(&tmW, W, K, 2 * N, ldw, Cfg::kTileN)) != FP8Q_OK)
    return st;
  static constexpr auto plain = fp8q::gemm_fp8_gated_kernel<false>, keep = fp8q::gemm_fp8_gated_kernel<true>;
  const int units = GU != nullptr ? resident_ctas<keep>(Cfg::kThreads, Cfg::smem_bytes)
                                  : resident_ctas<plain>(Cfg::kThreads, Cfg::smem_bytes);
  if (units <= 0) return FP8Q_ERR_CUDA;
  const auto grid = static_cast<unsigned>(mt * nt < units ? mt * nt : units);
  if (GU != nullptr)
    keep<<<grid, Cfg::kThreads, Cfg::smem_bytes, s>>>(tmA, tmW, a);
  else
    plain<<<grid, Cfg::kThreads, Cfg::smem_bytes, s>>>(tmA, tmW, a);
  return launched();
}

}  // namespace

extern "C" {

int fp8q_quant_int8_rowwise(const void* x, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq, float* scales,
                            void* stream) {
  if (M < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x || !q || !scales) return FP8Q_ERR_NULL;
  if (ldx < K || ldq < K || M > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;
  if (!aligned(x, 2) || !aligned(scales, 4)) return FP8Q_ERR_ALIGN;
  const auto* xs = static_cast<const uint16_t*>(x);
  const auto st = static_cast<cudaStream_t>(stream);
  constexpr int T = fp8q::kInt8Threads, V = 8 * fp8q::kInt8Vecs;
  const auto m32 = static_cast<unsigned>(M);
  if (K % 8 != 0 || ldx % 8 != 0 || !aligned(x, 16) || ldq % 8 != 0 || !aligned(q, 8))
    fp8q::quant_int8_any_kernel<<<m32, T, 0, st>>>(xs, K, ldx, q, ldq, scales);
  else if (K <= 32 * V)
    fp8q::quant_int8_rows_kernel<32, true><<<m32 / 8 + (m32 % 8 != 0), T, 0, st>>>(xs, M, K, ldx, q, ldq, scales);
  else if (K <= T * V)
    fp8q::quant_int8_rows_kernel<T, true><<<m32, T, 0, st>>>(xs, M, K, ldx, q, ldq, scales);
  else
    fp8q::quant_int8_rows_kernel<T, false><<<m32, T, 0, st>>>(xs, M, K, ldx, q, ldq, scales);
  return launched();
}

int fp8q_gemm_int8(const int8_t* A, const float* sA, const int8_t* B, const float* sB, void* C, int out_dtype,
                   int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, void* stream) {
  if (M == 0 && N >= 0 && K >= 0) return FP8Q_OK;
  const int st = check_int8(A, sA, B, sB, C, out_dtype, M, N, K, lda, ldb, ldc);
  if (st != FP8Q_OK) return st;
  const auto s = static_cast<cudaStream_t>(stream);
  return out_dtype == FP8Q_OUT_BF16 ? run_int8<false, true>(A, sA, B, sB, C, M, N, K, lda, ldb, ldc, s)
                                    : run_int8<false, false>(A, sA, B, sB, C, M, N, K, lda, ldb, ldc, s);
}

int fp8q_gemm_int8_gated(const int8_t* A, const float* sA, const int8_t* W, const float* sW, void* H, int64_t M,
                         int64_t N, int64_t K, int64_t lda, int64_t ldw, int64_t ldh, void* stream) {
  if (M == 0 && N >= 0 && K >= 0) return FP8Q_OK;
  const int st = check_int8(A, sA, W, sW, H, FP8Q_OUT_BF16, M, N, K, lda, ldw, ldh);
  if (st != FP8Q_OK) return st;
  return run_int8<true, true>(A, sA, W, sW, H, M, N, K, lda, ldw, ldh, static_cast<cudaStream_t>(stream));
}

int fp8_gemm_blockscaled_gated(const uint8_t* A, const float* sA, int64_t ld_sa, const uint8_t* W, const float* sW,
                               void* H, int64_t ldh, void* GU, int64_t ldgu, int64_t M, int64_t N, int64_t K,
                               int64_t lda, int64_t ldw, void* stream) {
  return run_fp8_gated(false, A, sA, ld_sa, W, sW, H, ldh, GU, ldgu, M, N, K, lda, ldw, stream);
}

int fp8_gemm_gated_ue8m0(const uint8_t* A, const float* sA, int64_t ld_sa, const uint8_t* W, const float* sW, void* H,
                         int64_t ldh, void* GU, int64_t ldgu, int64_t M, int64_t N, int64_t K, int64_t lda,
                         int64_t ldw, void* stream) {
  return run_fp8_gated(true, A, sA, ld_sa, W, sW, H, ldh, GU, ldgu, M, N, K, lda, ldw, stream);
}

int fp8q_gated_backward_quant(const void* dH, int64_t lddh, const void* GU, int64_t ldgu, int64_t M, int64_t N,
                              uint8_t* q, int64_t ldq, float* s, int64_t ld_s, uint8_t* qt, int64_t ldqt, float* st,
                              int64_t ld_st, int pow2_scale, void* stream) {
  if (M < 0 || N < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || N == 0) return FP8Q_OK;
  if (!dH || !GU || !q || !s || !qt || !st) return FP8Q_ERR_NULL;
  if (N % 128 != 0 || N > 0x3FFFFFFF || M > 0x3FFFFFFF) return FP8Q_ERR_SHAPE;
  const int64_t mt = (M + 127) / 128;
  if (lddh < N || ldgu < 2 * N || ldq < 2 * N || ld_s < M || ldqt < 128 * mt || ld_st < 2 * N) return FP8Q_ERR_SHAPE;
  if (lddh % 8 != 0 || ldgu % 8 != 0 || ldq % 8 != 0 || ldqt % 16 != 0 || !aligned(dH, 16) || !aligned(GU, 16) ||
      !aligned(q, 8) || !aligned(qt, 16) || !aligned(s, 4) || !aligned(st, 4))
    return FP8Q_ERR_ALIGN;
  if (mt > 0x7FFFFFFF / (N / 128)) return FP8Q_ERR_SHAPE;     // one-dimensional grid
  CUtensorMap tmDh, tmGu;
  if (!encode_bf16_tiles(&tmDh, dH, M, N, lddh) || !encode_bf16_tiles(&tmGu, GU, M, 2 * N, ldgu)) return FP8Q_ERR_CUDA;
  GatedBwdArgs a{q, s, qt, st, ldq, ld_s, ldqt, ld_st, M, N};
  const auto grid = static_cast<unsigned>(mt * (N / 128));
  const auto stm = static_cast<cudaStream_t>(stream);
  static constexpr auto k1 = fp8q::gated_backward_quant_kernel<true>, k0 = fp8q::gated_backward_quant_kernel<false>;
  constexpr int T = fp8q::kGatedBwdThreads;
  if ((pow2_scale ? resident_ctas<k1>(T, fp8q::kGatedBwdSmem) : resident_ctas<k0>(T, fp8q::kGatedBwdSmem)) <= 0)
    return FP8Q_ERR_CUDA;
  if (pow2_scale)
    k1<<<grid, T, fp8q::kGatedBwdSmem, stm>>>(tmDh, tmGu, a);
  else
    k0<<<grid, T, fp8q::kGatedBwdSmem, stm>>>(tmDh, tmGu, a);
  return launched();
}

int fp8q_quant_act_dual_padded(const void* x, int64_t M, int64_t K, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                               int64_t ld_s, uint8_t* qt, int64_t ldqt, float* st, int64_t ld_st, int pow2_scale,
                               void* stream) {
  if (M < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x || !q || !s || !qt || !st) return FP8Q_ERR_NULL;
  if (K % 128 != 0 || M > 0x3FFFFFFF || K > 0x3FFFFFFF) return FP8Q_ERR_SHAPE;
  const int64_t mt = (M + 127) / 128;
  if (ldx < K || ldq < K || ld_s < M || ldqt < 128 * mt || ld_st < K) return FP8Q_ERR_SHAPE;
  if (ldx % 8 != 0 || ldq % 8 != 0 || ldqt % 16 != 0 || !aligned(x, 16) || !aligned(q, 8) || !aligned(qt, 16) ||
      !aligned(s, 4) || !aligned(st, 4))
    return FP8Q_ERR_ALIGN;
  if (mt > 0x7FFFFFFF / (K / 128)) return FP8Q_ERR_SHAPE;     // one-dimensional grid
  CUtensorMap tmx;
  if (!encode_bf16_tiles(&tmx, x, M, K, ldx)) return FP8Q_ERR_CUDA;
  const auto grid = static_cast<unsigned>(mt * (K / 128));
  const auto g32 = static_cast<uint32_t>(K / 128);
  const auto stm = static_cast<cudaStream_t>(stream);
  static constexpr auto k1 = fp8q::quant_act_dual_padded_kernel<true>, k0 = fp8q::quant_act_dual_padded_kernel<false>;
  if ((pow2_scale ? resident_ctas<k1>(256, fp8q::kDualSmem) : resident_ctas<k0>(256, fp8q::kDualSmem)) <= 0)
    return FP8Q_ERR_CUDA;
  if (pow2_scale)
    k1<<<grid, 256, fp8q::kDualSmem, stm>>>(tmx, M, q, ldq, s, ld_s, qt, ldqt, st, ld_st, g32);
  else
    k0<<<grid, 256, fp8q::kDualSmem, stm>>>(tmx, M, q, ldq, s, ld_s, qt, ldqt, st, ld_st, g32);
  return launched();
}

int fp8q_gated_linear_sizes(int64_t T, int64_t N, int64_t K, int for_dx, int for_dw, int pow2_scale,
                            size_t* bytes) {
  if (!bytes) return FP8Q_ERR_NULL;
  GatedLayer l{};
  const int st = gated_layer(&l, T, N, K, for_dx != 0, for_dw != 0, pow2_scale != 0);
  bytes[0] = l.kept;
  bytes[1] = l.forward;
  bytes[2] = l.backward;
  return st;
}

int fp8q_gated_linear_forward(const void* x, const void* w, int64_t T, int64_t N, int64_t K, int for_dw,
                              int pow2_scale, void* kept, void* scratch, void* H, void* stream) {
  GatedLayer l{};
  int st = gated_layer(&l, T, N, K, false, for_dw != 0, true);   // (no split-K on the way forward)
  if (st != FP8Q_OK) return st;
  if (!w || !kept || (T > 0 && (!x || !scratch || !H))) return FP8Q_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(kept, 16) || !aligned(scratch, 16) || !aligned(H, 16))
    return FP8Q_ERR_ALIGN;
  auto* k8 = static_cast<uint8_t*>(kept);
  auto* s8 = static_cast<uint8_t*>(scratch);
  auto f32 = [](uint8_t* p) { return reinterpret_cast<float*>(p); };
  const int64_t R = 2 * N;
  if ((st = fp8q_quant_weight_128x128(w, R, K, K, k8 + l.qw, K, f32(k8 + l.sw), pow2_scale, stream)) != FP8Q_OK || T == 0)
    return st;
  if (!for_dw)
    st = fp8q_quant_act_1x128(x, T, K, K, s8 + l.qx, K, f32(s8 + l.sx), T, pow2_scale, stream);
  else
    st = (l.Tp == T ? fp8q_quant_act_dual : fp8q_quant_act_dual_padded)(
        x, T, K, K, s8 + l.qx, K, f32(s8 + l.sx), T, k8 + l.qxt, l.Tp, f32(k8 + l.sxt), K, pow2_scale, stream);
  if (st != FP8Q_OK) return st;
  return (pow2_scale ? fp8_gemm_gated_ue8m0 : fp8_gemm_blockscaled_gated)(
      s8 + l.qx, f32(s8 + l.sx), T, k8 + l.qw, f32(k8 + l.sw), H, N, k8 + l.gu, R, T, N, K, K, K, stream);
}

int fp8q_gated_linear_backward(const void* dH, const void* kept, int64_t T, int64_t N, int64_t K, int for_dw,
                               int pow2_scale, void* scratch, void* dX, void* dW, void* stream) {
  GatedLayer l{};
  int st = gated_layer(&l, T, N, K, dX != nullptr, for_dw != 0, pow2_scale != 0);
  if (st != FP8Q_OK) return st;
  if (T == 0) return FP8Q_OK;
  if (!dH || !kept || !scratch || (dW && !for_dw)) return FP8Q_ERR_NULL;
  if (!aligned(dH, 16) || !aligned(kept, 16) || !aligned(scratch, 16) || !aligned(dX, 16) || !aligned(dW, 16))
    return FP8Q_ERR_ALIGN;
  const auto* k8 = static_cast<const uint8_t*>(kept);
  auto* s8 = static_cast<uint8_t*>(scratch);
  auto f32 = [](const uint8_t* p) { return reinterpret_cast<float*>(const_cast<uint8_t*>(p)); };
  const int64_t R = 2 * N, Tp = l.Tp;
  st = fp8q_gated_backward_quant(dH, N, k8 + l.gu, R, T, N, s8 + l.qd, R, f32(s8 + l.sd), T, s8 + l.qdt, Tp,
                                 f32(s8 + l.sdt), R, pow2_scale, stream);
  auto product = [&](const uint8_t* A, const float* sA, int64_t ld_sa, const uint8_t* B, const float* sB, int64_t ld_sb,
                     int mode, void* C, int64_t m, int64_t n, int64_t k) {
    if (pow2_scale)
      return fp8_gemm_blockscaled_ue8m0(A, sA, ld_sa, B, sB, ld_sb, mode, C, FP8Q_OUT_BF16, m, n, k, k, k, n, stream);
    const bool split = k >= 2048 && l.ws_bytes > 0;
    return fp8_gemm_blockscaled_ws(A, sA, ld_sa, B, sB, ld_sb, mode, C, FP8Q_OUT_BF16, m, n, k, k, k, n,
                                   split ? s8 + l.ws : nullptr, split ? l.ws_bytes : 0, stream);
  };
  if (st == FP8Q_OK && dX) {
    st = fp8q_transpose_blocks(k8 + l.qw, f32(k8 + l.sw), R, K, K, s8 + l.qwt, f32(s8 + l.swt), R, stream);
    if (st == FP8Q_OK)
      st = product(s8 + l.qd, f32(s8 + l.sd), T, s8 + l.qwt, f32(s8 + l.swt), 0, FP8Q_BSCALE_BLOCK128x128, dX, T, K, R);
  }
  if (st == FP8Q_OK && dW)
    st = product(s8 + l.qdt, f32(s8 + l.sdt), R, k8 + l.qxt, f32(k8 + l.sxt), K, FP8Q_BSCALE_ROW1x128, dW, R, K, Tp);
  return st;
}

}  // extern "C"
