// Per-row INT8 quantization and the INT8 product scaled per token and per channel
// (sm_100a: tcgen05.mma kind::i8, exact INT32 accumulation in TMEM).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "quant.cuh"
#include "gemm.cuh"
#include "silu.cuh"

namespace fp8q {

// ---------------------------------------------------------------- per-row quantization
//
//   a = max_k |x[m, k]|
//   a < 2^-100:      s = 1, q = 0          (counts as a zero row: a chosen threshold, above the 2^-121
//                                          below which 127 / a would leave FP32's range)
//   a Inf or NaN:    s = NaN, q = 0        (every product with the row is then NaN)
//   otherwise        s = RN_f32(a / 127), r = RN_f32(127 / a), q = round-half-even(x r)
//
// The product x r is rounded once: fma(x, r, 1.5 * 2^23) leaves round-half-even(x r) in the
// low bits of the sum, because the unit of the sum's binade is 1.  |x r| <= 127 (1 + 2^-24)
// rounds to 127 at most, so no clamp is needed.
//
// Bound by HBM: 2 bytes read and 1 written per element.  Measured: 53 us at 16384 x 7168, the
// copy rate; one row of 7168 takes 1.6 us.

struct Int8Scale {
  float s, r;
  uint32_t keep;          // mask of the packed codes: 0 for a row that is not finite
  // abs_bits: the largest |x| as a 16-bit bf16 pattern (patterns order like the values, Inf
  // and NaN above every finite one)
  __device__ __forceinline__ explicit Int8Scale(uint32_t abs_bits) {
    const float a = __uint_as_float(abs_bits << 16);
    s = 1.0f;
    r = 0.0f;
    keep = 0xFFFFFFFFu;
    if (abs_bits >= 0x7F80u) {
      s = __uint_as_float(0x7FC00000u);
      keep = 0;
    } else if (a >= 0x1p-100f) {
      s = __fdiv_rn(a, 127.0f);
      r = __fdiv_rn(127.0f, a);
    }
  }
  __device__ __forceinline__ uint32_t code(float x) const {    // the code in the low byte
    return __float_as_uint(__fmaf_rn(x, r, 12582912.0f));
  }
  __device__ __forceinline__ uint32_t pack(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) const {
    return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410) & keep;
  }
  __device__ __forceinline__ uint2 codes(const uint4& v) const {
    return make_uint2(pack(code(bf16lo(v.x)), code(bf16hi(v.x)), code(bf16lo(v.y)), code(bf16hi(v.y))),
                      pack(code(bf16lo(v.z)), code(bf16hi(v.z)), code(bf16lo(v.w)), code(bf16hi(v.w))));
  }
};

__device__ __forceinline__ uint32_t abs_max_u16x2(uint32_t m, const uint4& v) {
  m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
  return __vmaxu2(m, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

// The largest 16-bit half of m over the TPR threads of a row (a warp, or the whole block).
template <int TPR>
__device__ __forceinline__ uint32_t row_max_u16(uint32_t m) {
  m = m >> 16 > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu;
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if constexpr (TPR > 32) {
    __shared__ uint32_t red[TPR / 32];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) m = max(m, red[i]);
  }
  return m;
}

constexpr int kInt8Threads = 256;
constexpr int kInt8Vecs = 4;          // 8-element vectors a thread keeps in registers

// Rows that start on 16 bytes and hold whole 8-element vectors.  TPR threads per row: a
// warp for rows of at most 1024 elements (8 rows per block, no block barrier), otherwise
// the block.  RESIDENT: the row stays in registers between the maximum and the codes;
// longer rows are read again (from L2).
template <int TPR, bool RESIDENT>
__global__ void __launch_bounds__(kInt8Threads)
    quant_int8_rows_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t ldx,
                           int8_t* __restrict__ q, int64_t ldq, float* __restrict__ s) {
  constexpr int kRows = kInt8Threads / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (m >= M) return;                              // a whole warp (TPR = 32) or nothing
  const uint16_t* src = x + m * ldx;
  int8_t* dst = q + m * ldq;
  const int64_t nv = K / 8;
  uint4 v[kInt8Vecs];
  uint32_t mx = 0;
  if constexpr (RESIDENT) {
#pragma unroll
    for (int j = 0; j < kInt8Vecs; ++j) {
      const int64_t i = t + TPR * j;
      v[j] = i < nv ? ldg_stream(src + 8 * i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kInt8Vecs; ++j) mx = abs_max_u16x2(mx, v[j]);
  } else {
    for (int64_t i = t; i < nv; i += TPR) mx = abs_max_u16x2(mx, *reinterpret_cast<const uint4*>(src + 8 * i));
  }
  const Int8Scale sc(row_max_u16<TPR>(mx));
  if constexpr (RESIDENT) {
#pragma unroll
    for (int j = 0; j < kInt8Vecs; ++j) {
      const int64_t i = t + TPR * j;
      if (i < nv) stg_u2(dst + 8 * i, sc.codes(v[j]));
    }
  } else {
    for (int64_t i = t; i < nv; i += TPR) stg_u2(dst + 8 * i, sc.codes(*reinterpret_cast<const uint4*>(src + 8 * i)));
  }
  if (t == 0) s[m] = sc.s;
}

// Rows of any length and alignment, one block each.  The 16-byte vectors between a row's
// first and last 16-byte boundary are read whole (the elements before and after them one by
// one), and put into shared memory, from where each thread takes four elements at a time
// in the order of the codes.  Rows longer than the buffer are read element by element,
// twice.  Bound by the block per row, whatever its length, with its barrier and 33 KB of shared
// memory: 16384 rows of 100 elements 28 us (of 104, which take the kernel above: 5.0), of 1001 36 us (1000:
// 8.1), of 2047 43 us; 4096 rows of 7167 22 us (0.61 of HBM).
constexpr int kInt8Staged = 16384;    // elements

__global__ void __launch_bounds__(kInt8Threads)
    quant_int8_any_kernel(const uint16_t* __restrict__ x, int64_t K, int64_t ldx, int8_t* __restrict__ q,
                          int64_t ldq, float* __restrict__ s) {
  __shared__ __align__(16) uint16_t row[kInt8Staged + 8];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  const uint16_t* src = x + m * ldx;
  int8_t* dst = q + m * ldq;
  const bool staged = K <= kInt8Staged;
  uint32_t mx = 0;
  // element k sits at row[shift + k], so that a vector of the row lands on 16 bytes
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / 2);
  if (staged) {
    const int n = static_cast<int>(K);
    const int head = min(n, (8 - shift) & 7);
    const int nv = (n - head) / 8, tail = head + 8 * nv;
    for (int i = t; i < nv; i += kInt8Threads) {
      const uint4 v = ldg_stream(src + head + 8 * i);
      *reinterpret_cast<uint4*>(row + shift + head + 8 * i) = v;
      mx = abs_max_u16x2(mx, v);
    }
    const int k = t < head ? t : tail + (t - head);
    if (k < n && (t < head || k >= tail)) {
      const uint16_t e = src[k];
      row[shift + k] = e;
      mx = __vmaxu2(mx, static_cast<uint32_t>(e & 0x7FFFu));   // mx holds two 16-bit maxima
    }
  } else {
    for (int64_t k = t; k < K; k += kInt8Threads) mx = max(mx, static_cast<uint32_t>(src[k] & 0x7FFFu));
  }
  const Int8Scale sc(row_max_u16<kInt8Threads>(mx));   // its barrier also orders the row
  auto value = [&](int64_t k) {
    return __uint_as_float(static_cast<uint32_t>(staged ? row[shift + k] : src[k]) << 16);
  };
  const int64_t n4 = reinterpret_cast<uintptr_t>(dst) % 4 == 0 ? K / 4 : 0;
  for (int64_t i = t; i < n4; i += kInt8Threads) {
    const int64_t k = 4 * i;
    *reinterpret_cast<uint32_t*>(dst + k) =
        sc.pack(sc.code(value(k)), sc.code(value(k + 1)), sc.code(value(k + 2)), sc.code(value(k + 3)));
  }
  for (int64_t k = 4 * n4 + t; k < K; k += kInt8Threads) dst[k] = static_cast<int8_t>(sc.code(value(k)) & sc.keep);
  if (t == 0) s[m] = sc.s;
}

// ---------------------------------------------------------------- INT8 products
//
//   C[m, n] = (acc(m, n) sA[m]) sB[n],   acc(m, n) = sum_k qA[m, k] qB[n, k]   (INT32, exact)
//
// and, GATED, from a weight of 2N rows (the gate's N, then the up projection's N):
//
//   h[m, n] = silu(g) u,  g = C[m, n], u = C[m, N + n],  silu(g) = g / (1 + exp(-g)).
//
// acc is exact while K 128^2 <= 2^31 - 1 (the host refuses a longer K); it is rounded once
// to FP32, and so is each of the two products with the scales.  Unlike the block-scaled FP8
// products nothing has to be promoted along K: the whole sum stays in TMEM, and the epilogue
// of one tile runs under the products of the next (two accumulators).
//
// Tiles of 128 rows by `width` columns (a launch parameter, at most 256, chosen by the host
// so that the last wave is as full as it can be), persistent CTAs of 12 warps:
//   warp 0      TMA producer: A [128 x 128 B] and B [width x 128 B] per 128 K-elements into
//               a ring of as many stages as fit (4 at width 256, up to 8; 128-byte swizzle):
//               a narrow tile's products are over sooner, and its operands must be further
//               ahead.  K past the operand's end is filled with zeros.  GATED: width / 2 gate
//               rows, then width / 2 up rows.
//   warp 1      TMEM owner and MMA issuer: 4 x tcgen05.mma kind::i8 (M128, K32) per stage.
//   warps 2, 3  idle.
//   warps 4-11  epilogue: warp w reads TMEM lanes 32 (w % 4).. in chunks of 32 columns, the
//               chunks alternating between the two warpgroups.
//
// PAIR: two CTAs share a tile of 256 rows (cta_group::2).  Each loads and holds its 128 rows of
// A and half the tile's rows of B (GATED: one the gate's, the other the up projection's), and
// the first issues MMAs of M = 256 that leave each CTA its own rows' sums.  An SM takes in at
// most 64 bytes a cycle from L2; a 128 x 256 tile alone needs 48 KB per 512-cycle stage, half
// as much again, a paired one 32 KB.
//
// Measured: 4096 x 7168 x 7168 in 122-132 us on pairs (0.96-1.03 of twice the bf16 peak, 88 % of
// the tensor pipe's cycles) and 141 us on single CTAs; gated 4096 x 2048 x 7168 in 76-79 us on
// pairs.  With the MMAs issued from a lane's own registers, not uniform ones: 135, 144 and 80.
struct Int8Args {
  const float* sA;      // [M]
  const float* sB;      // [N], gated [2N]
  void* C;
  int64_t ldc, M, N;
  int k_groups;         // ceil(K / 128)
  int width;            // B rows per tile: a multiple of 32 (gated: of 64), at most 256
  int stages;           // Int8Cfg::stages(width)
  int mt, nt;           // tiles along M and N
  int n_fastest;
  int vec;              // C's rows start on 16 bytes
};

// Instruction descriptor, kind::i8: D = S32, A = B = S8, both K-major, dense, no saturation.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T, S8 x S8 -> S32.  CG = 2: a CTA pair, as in mma_f8.
template <int CG>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 x 32 words, row i in lane i's v[0 .. 31], transposed in place: afterwards lane i holds
// column i.  Five exchange stages; registers are indexed by constants only.
__device__ __forceinline__ void warp_transpose32(uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j & d) continue;
      const uint32_t send = up ? v[j] : v[j + d];
      const uint32_t recv = __shfl_xor_sync(0xFFFFFFFFu, send, d);
      if (up) v[j] = recv; else v[j + d] = recv;
    }
  }
}

// Writes a 32 x 32 chunk (row in lane, FP32 bits in v) at rows m0 .. m0 + 31, columns
// n0 .. n0 + 31 of C.  Whole chunks of rows that start on 16 bytes go out 64 bytes of a row at a
// time; any other chunk is transposed inside the warp, so that each store instruction
// writes up to 32 consecutive elements of one row.  Every condition on columns is
// warp-uniform.
template <bool OUT_BF16>
__device__ __forceinline__ void store_chunk32(uint32_t (&v)[32], void* C, int64_t ldc, int64_t m0, int64_t n0,
                                              int64_t M, int64_t N, bool vec) {
  const int lane = threadIdx.x & 31;
  if (vec && n0 + 32 <= N) {
    const bool row_ok = m0 + lane < M;
    if (OUT_BF16) {
      uint4 hv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[8 * j + 2 * t]),
                                                   __uint_as_float(v[8 * j + 2 * t + 1]));
          h[t] = *reinterpret_cast<uint32_t*>(&b);
        }
        hv[j] = make_uint4(h[0], h[1], h[2], h[3]);
      }
      store_rows_by_quads(hv, reinterpret_cast<uint8_t*>(reinterpret_cast<__nv_bfloat16*>(C) + (m0 + lane) * ldc + n0),
                          row_ok);
    } else {
      uint4 fv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) fv[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      store_rows_by_quads(fv, reinterpret_cast<uint8_t*>(reinterpret_cast<float*>(C) + (m0 + lane) * ldc + n0), row_ok);
    }
    return;
  }
  warp_transpose32(v, lane);
  if (n0 + lane >= N) return;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (m0 + i >= M) break;
    const int64_t at = (m0 + i) * ldc + n0 + lane;
    if (OUT_BF16) reinterpret_cast<__nv_bfloat16*>(C)[at] = __float2bfloat16_rn(__uint_as_float(v[i]));
    else reinterpret_cast<float*>(C)[at] = __uint_as_float(v[i]);
  }
}

template <bool PAIR>
struct Int8Cfg {
  static constexpr int kTileM = PAIR ? 256 : 128, kMaxWidth = 256, kMaxStages = 8;
  static constexpr int kThreads = 32 * (4 + 8);
  static constexpr uint32_t kABytes = 128 * kBK;
  static constexpr uint32_t kRingBytes = 4 * (kABytes + kMaxWidth * kBK);
  static constexpr uint32_t ring = 0;                                  // a stage: A, then B
  static constexpr uint32_t scales = ring + kRingBytes;                // float[2][kMaxWidth]
  static constexpr uint32_t bars = scales + 2 * kMaxWidth * 4;
  // full[8], empty[8], tfull[2], tempty[2], drain
  static constexpr uint32_t misc = align_up(bars + 8 * (2 * kMaxStages + 5), 16);
  static constexpr uint32_t smem_bytes = misc + 16 + 1024;
  static_assert(smem_bytes <= 232448, "fits the 227 KB opt-in shared memory");
  // of one CTA: its 128 rows of A and its share of B
  static constexpr __host__ __device__ uint32_t stage_bytes(int width) {
    return kABytes + (PAIR ? width / 2 : width) * kBK;
  }
  static constexpr int stages(int width) {
    const int n = kRingBytes / stage_bytes(width);
    return n < kMaxStages ? n : kMaxStages;
  }
};

template <bool GATED, bool OUT_BF16, bool PAIR>
__global__ void __launch_bounds__(Int8Cfg<PAIR>::kThreads, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const Int8Args p) {
  static_assert(OUT_BF16 || !GATED, "the gated product is bf16");
  using Cfg = Int8Cfg<PAIR>;
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int S = Cfg::kMaxStages;                       // barriers; the ring has p.stages
  extern __shared__ uint8_t smem_raw[];
  // (the pair's CTAs have the same layout: shared memory starts at the same offset in both)
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::bars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);
  float* scales = reinterpret_cast<float*>(smem + Cfg::scales);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;      // 0: the CTA that issues the MMAs
  const int unit0 = blockIdx.x / CG, units = gridDim.x / CG;
  const int G = p.k_groups;
  const int cols = GATED ? p.width / 2 : p.width;          // output columns per tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), CG * 32 * kEpiWarps);       // the pair's epilogues free rank 0's
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc<CG>(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish<CG>();
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();                                // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int tiles = p.mt * p.nt;
  const int n_tiles = unit0 < tiles ? (tiles - unit0 + units - 1) / units : 0;
  auto tile_at = [&](int i, int64_t& row0, int64_t& col0) {
    const int t = unit0 + i * units;
    const int fast = p.n_fastest ? p.nt : p.mt;
    const int q = t / fast, r = t - q * fast;
    row0 = static_cast<int64_t>(p.n_fastest ? q : r) * Cfg::kTileM + 128 * rank;
    col0 = static_cast<int64_t>(p.n_fastest ? r : q) * cols;
  };

  if (warp == 0) {
    // -------------------------------------------------------------- TMA producer
    const uint32_t stage = Cfg::stage_bytes(p.width);
    const bool leader = elect_one();
    uint32_t it = 0, phase = 1;                            // of the empty barriers
    int s = 0;
    bool ok = true;
    for (int i = 0; ok && i < n_tiles; ++i) {
      int64_t row0, col0;
      tile_at(i, row0, col0);
      const int32_t ya = static_cast<int32_t>(row0), yb = static_cast<int32_t>(col0);
      const int32_t yu = static_cast<int32_t>(GATED ? p.N + col0 : col0 + p.width / 2);   // the other half of B
      for (int g = 0; g < G; ++g, ++it) {
        if (!mbar_wait_warp(empty_bar(s), phase, kSiteProducer, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t a_addr = sbase + Cfg::ring + s * stage, b_addr = a_addr + Cfg::kABytes;
        const int32_t x = g * kBK;
        if (leader) {
          if constexpr (PAIR) {
            // both CTAs' bytes count on rank 0's barrier, whose phase its own arrival opens
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * stage);
            const uint32_t bar = map_shared_rank(full_bar(s), 0);
            tma_load_2d_pair(a_addr, &tmA, bar, x, ya);
            tma_load_2d_pair(b_addr, &tmB, bar, x, rank == 0 ? yb : yu);
          } else {
            mbar_arrive_expect_tx(full_bar(s), stage);
            tma_load_2d(a_addr, &tmA, full_bar(s), x, ya);
            tma_load_2d(b_addr, &tmB, full_bar(s), x, yb);
            if (GATED) tma_load_2d(b_addr + cols * kBK, &tmB, full_bar(s), x, yu);
          }
        }
        if (++s == p.stages) s = 0, phase ^= 1;
      }
    }
    // Every issued load lands before the CTA can exit: rank 0 sees its stages' bytes arrive, rank
    // 1 sees their products, which waited for them, complete (bounded; loads end on their
    // own).
    const uint32_t n = p.stages;
    for (uint32_t j = it > n ? it - n : 0; j < it; ++j)
      mbar_wait(rank == 0 ? full_bar(j % n) : empty_bar(j % n), (j / n) & 1u, kSiteDrain, nullptr);
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    // The whole warp walks the loop and one lane issues, so that descriptors and addresses live in
    // uniform registers: from a lane's own registers each MMA takes 64 cycles to issue and a
    // group 560 in all, more than its 512 cycles of products.
    if (rank == 0) {
      const uint32_t idesc = idesc_s8_s32(Cfg::kTileM, p.width);
      const uint32_t stage = Cfg::stage_bytes(p.width);
      const uint64_t a0 = smem_desc_k_sw128(sbase + Cfg::ring);
      const bool leader = elect_one();
      auto commit = [&](uint32_t bar) {
        if constexpr (PAIR) mma_commit_pair(bar, 3);
        else mma_commit<1>(bar);
      };
      uint32_t phase = 0;                                  // of the full barriers
      int s = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_tiles; ++i) {
        const uint32_t buf = i & 1;
        if (!mbar_wait_warp(tempty_bar(buf), ((i >> 1) & 1u) ^ 1u, kSiteMmaEmpty, abort_flag)) break;
        const uint32_t d = tmem_base + buf * Cfg::kMaxWidth;
        for (int g = 0; g < G; ++g) {
          if (!mbar_wait_warp(full_bar(s), phase, kSiteMmaFull, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = a0 + s * (stage >> 4), b = a + (Cfg::kABytes >> 4);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk) mma_i8<CG>(d, a + 2 * kk, b + 2 * kk, idesc, (g > 0 || kk > 0) ? 1u : 0u);
            commit(empty_bar(s));
          }
          if (++s == p.stages) s = 0, phase ^= 1;
        }
        if (ok && leader) commit(tfull_bar(buf));
      }
      if (leader) {
        mma_commit<CG>(drain_bar);
        mbar_wait(drain_bar, 0, kSiteDrain, nullptr);
      }
      __syncwarp();
    }
  } else if (warp >= kEpiWarp0) {
    // -------------------------------------------------------------- epilogue
    const int et = threadIdx.x - 32 * kEpiWarp0;           // 0 .. 255
    const int set = et >> 7;
    const int quad = warp & 3;
    bool ok = true;
    for (int i = 0; i < n_tiles; ++i) {
      int64_t row0, col0;
      tile_at(i, row0, col0);
      const uint32_t buf = i & 1;
      // the tile's column scales; the slot's previous readers passed the barrier of tile
      // i - 1 after their last read
      float* sb = scales + buf * Cfg::kMaxWidth;
      if (et < p.width) {
        const bool up = GATED && et >= cols;
        const int64_t n = col0 + (up ? et - cols : et);
        sb[et] = n < p.N ? __ldg(p.sB + (up ? p.N : 0) + n) : 0.0f;
      }
      const int64_t m0 = row0 + 32 * quad;
      const float sa = m0 + lane < p.M ? __ldg(p.sA + m0 + lane) : 0.0f;
      named_bar_sync(1, 32 * kEpiWarps);
      if (ok) ok = mbar_wait(tfull_bar(buf), (i >> 1) & 1u, kSiteEpilogue, abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);                    // TMEM loads are whole-warp
      if (ok) {
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * quad) << 16) + buf * Cfg::kMaxWidth;
#pragma unroll 1
        for (int c = 32 * set; c < cols; c += 64) {
          uint32_t r[32];
          tmem_ld_32cols(taddr + c, r);
          if constexpr (GATED) {
            uint32_t ru[32];
            tmem_ld_32cols(taddr + cols + c, ru);
            tmem_ld_wait_regs(r);
            tmem_ld_wait_regs(ru);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float g = (__int2float_rn(static_cast<int>(r[j])) * sa) * sb[c + j];
              const float u = (__int2float_rn(static_cast<int>(ru[j])) * sa) * sb[cols + c + j];
              r[j] = __float_as_uint(silu_mul(g, u));
            }
          } else {
            tmem_ld_wait_regs(r);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              r[j] = __float_as_uint((__int2float_rn(static_cast<int>(r[j])) * sa) * sb[c + j]);
          }
          if (m0 < p.M && col0 + c < p.N)
            store_chunk32<OUT_BF16>(r, p.C, p.ldc, m0, col0 + c, p.M, p.N, p.vec != 0);
        }
        tc_fence_before();                                 // accumulator free for tile i + 2
        if constexpr (PAIR) mbar_arrive_cluster(map_shared_rank(tempty_bar(buf), 0));
        else mbar_arrive(tempty_bar(buf));
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();                                // nothing reaches into the other CTA any more
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, kTmemCols);
  }
}

}  // namespace fp8q
