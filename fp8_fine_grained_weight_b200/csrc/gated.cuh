// The gated feed-forward projections in block-scaled FP8: both products, the activation and
// the product of the two in one kernel, and the backward pass's elementwise part fused with
// the quantization of its result (sm_100a: tcgen05 + TMEM + TMA).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "quant.cuh"
#include "gemm.cuh"
#include "int8.cuh"

namespace fp8q {

// ---------------------------------------------------------------- forward
//
//   g[m, n] = sum_G  P_G sA[m, G] sW[n / 128, G],        P_G over the gate's row n of W
//   u[m, n] = the same over row N + n of W
//   h[m, n] = silu(g) u,  silu(g) = g / (1 + exp(-g))
//
// W is [2N, K]: the gate's N rows, then the up projection's.  The promotion per 128 K-elements
// is that of the block-scaled GEMM: partial sums leave TMEM after each group, are multiplied
// by the group's scales and added in FP32 registers.  g and u stay in FP32 up to h; when the
// backward pass will need them (GU) they are also stored, rounded to bf16.
//
// A tile is 128 rows by 128 columns of h: 256 rows of W, the gate's 128 and the up projection's
// 128.  Two epilogue warpgroups each own 64 columns of h: a thread holds both factors of its 64
// outputs, so nothing is exchanged.
//
//   warp 0      TMA producer: A [128 x 128 B], W [128 x 128 B] twice, 4 stages
//   warps 1, 3  MMA issuers (N = 256), warp 1 for the even groups and accumulator 0, warp 3 for the
//               odd ones and accumulator 1: while one's four products run, the other
//               passes its waits (90 cycles each, even when there is nothing to wait for).
//               One commit per group both frees the stage and publishes the partial sums.
//   warp 2      scale producer (slots of four groups: 128 row scales, a gate and an up scale)
//   warps 4-11  promotion and epilogue.  Registers: 128 threads * 40 + 256 * 232 <= 384 * 168.
//
// Measured: 223-251 us at 8192 x 2048 x 7168 over the machines seen (0.57-0.65 of the FP8 peak), 38-42
// us at 1000 rows; for power-of-two scales the tensor core applies them in 178-184 and 29 us
// (gemm_ue8m0.cuh).  The promotion loop bounds it (tensor pipe about half busy): about 900 cycles per
// group against 512 of MMAs, of which the 64 packed FMAs per thread are 260.  Three warpgroups on 96
// columns (277 us) and four at 112 registers (250 us) measured slower; one issuer and per-thread
// arrivals 233 us.
struct GatedArgs {
  const float* sA;      // group-major [G][ld_sa]
  int64_t ld_sa;
  const float* sW;      // [2N / 128][G]
  __nv_bfloat16* h;     // [M, N]
  int64_t ldh;
  __nv_bfloat16* gu;    // [M, 2N] when GU
  int64_t ld_gu, M, N;
  int G;
  int mt, nt, n_fastest;
};

struct GatedCfg {
  static constexpr int kTileM = 128, kTileN = 128, kN = 2 * kTileN, kStages = 4, kAccBufs = 2;
  static constexpr int kSets = 2, kEpiThreads = 128 * kSets, kThreads = 128 + kEpiThreads;
  static constexpr int kSetCols = kTileN / kSets;       // columns of h per warpgroup
  static constexpr int kRegsCtl = 40, kRegsEpi = 232;
  static constexpr uint32_t kABytes = 128 * kBK, kBBytes = kN * kBK, kStageTx = kABytes + kBBytes;
  // Scales of four groups of one tile: [128 rows][4], then the gate's and the up projection's [4].
  static constexpr int kSlotGroups = 4, kScaleSlots = 5;
  static constexpr uint32_t kSlotFloats = kSlotGroups * (128 + 2);
  static constexpr uint32_t a = 0;
  static constexpr uint32_t b = a + kStages * kABytes;
  static constexpr uint32_t sring = b + kStages * kBBytes;
  static constexpr uint32_t bars = sring + 4 * kScaleSlots * kSlotFloats;
  // full[S], empty[S], tempty[2], drain[2], sfull[R], sempty[R]
  static constexpr uint32_t misc = align_up(bars + 8 * (2 * kStages + 2 * kAccBufs + 2 * kScaleSlots), 16);
  static constexpr uint32_t smem_bytes = misc + 16 + 1024;
  static_assert(kABytes % 1024 == 0 && kBBytes % 1024 == 0 && kTileN * kBK % 1024 == 0, "swizzle atoms");
  static_assert(sring % 16 == 0 && kSlotFloats % 4 == 0, "float4 reads of the scales");
  static_assert(kStages % kAccBufs == 0, "a stage barrier's phase outlives the epilogue's wait for it");
  static_assert(kAccBufs * kN <= static_cast<int>(kTmemCols) && kSetCols == 64, "accumulators; a set's columns");
  static_assert(128 * kRegsCtl + kEpiThreads * kRegsEpi <= kThreads * 168, "register split");
  static_assert(smem_bytes <= 232448, "fits the 227 KB opt-in shared memory");
};

// Two FP32 pairs of a column run, rounded to bf16, as 16 bytes.
__device__ __forceinline__ uint4 bf16x8(const float2& a, const float2& b, const float2& c, const float2& d) {
  __nv_bfloat162 h0 = __float22bfloat162_rn(a), h1 = __float22bfloat162_rn(b);
  __nv_bfloat162 h2 = __float22bfloat162_rn(c), h3 = __float22bfloat162_rn(d);
  return make_uint4(*reinterpret_cast<uint32_t*>(&h0), *reinterpret_cast<uint32_t*>(&h1),
                    *reinterpret_cast<uint32_t*>(&h2), *reinterpret_cast<uint32_t*>(&h3));
}

template <bool GU>
__global__ void __launch_bounds__(GatedCfg::kThreads, 1)
    gemm_fp8_gated_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                          const GatedArgs p) {
  using Cfg = GatedCfg;
  constexpr int S = Cfg::kStages, NB = Cfg::kAccBufs, R = Cfg::kScaleSlots;
  constexpr int SG = Cfg::kSlotGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::bars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto drain_bar = [&](int b) { return bar0 + 8u * (2 * S + NB + b); };
  auto sfull_bar = [&](int r) { return bar0 + 8u * (2 * S + 2 * NB + r); };
  auto sempty_bar = [&](int r) { return bar0 + 8u * (2 * S + 2 * NB + R + r); };
  float* sring = reinterpret_cast<float*>(smem + Cfg::sring);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(tempty_bar(b), Cfg::kEpiThreads / 32);   // one arrival a warp
      mbar_init(drain_bar(b), 1);
    }
    for (int r = 0; r < R; ++r) {
      mbar_init(sfull_bar(r), 32);                 // one cp.async arrival per producer lane
      mbar_init(sempty_bar(r), Cfg::kEpiThreads / 32);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int tiles = p.mt * p.nt;
  const int n_tiles = (tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  auto tile_at = [&](int i, int64_t& row0, int64_t& col0) {
    const int t = blockIdx.x + i * gridDim.x;
    const int fast = p.n_fastest ? p.nt : p.mt;
    const int q = t / fast, r = t - q * fast;
    row0 = static_cast<int64_t>(p.n_fastest ? q : r) * Cfg::kTileM;
    col0 = static_cast<int64_t>(p.n_fastest ? r : q) * Cfg::kTileN;
  };

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsCtl));
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      const bool leader = elect_one();
      uint32_t it = 0, s = 0, phase = 1;                   // of the empty barriers
      bool ok = true;
      for (int i = 0; ok && i < n_tiles; ++i) {
        int64_t row0, col0;
        tile_at(i, row0, col0);
        const int32_t row = static_cast<int32_t>(row0);
        const int32_t gate = static_cast<int32_t>(col0), up = static_cast<int32_t>(p.N + col0);
        for (int g = 0; g < G; ++g, ++it) {
          if (!mbar_wait_warp(empty_bar(s), phase, kSiteProducer, abort_flag)) { ok = false; break; }
          const uint32_t a = sbase + Cfg::a + s * Cfg::kABytes, b = sbase + Cfg::b + s * Cfg::kBBytes;
          if (leader) {
            mbar_arrive_expect_tx(full_bar(s), Cfg::kStageTx);
            tma_load_2d(a, &tmA, full_bar(s), g * kBK, row);
            tma_load_2d(b, &tmW, full_bar(s), g * kBK, gate);
            tma_load_2d(b + Cfg::kTileN * kBK, &tmW, full_bar(s), g * kBK, up);
          }
          if (++s == S) s = 0, phase ^= 1;
        }
      }
      // every issued load lands before the CTA can exit (bounded; loads end on their own)
      for (uint32_t j = it > S ? it - S : 0; j < it; ++j) mbar_wait(full_bar(j % S), (j / S) & 1u, kSiteDrain, nullptr);
      __syncwarp();
    } else if (warp == 1 || warp == 3) {
      // ---------------------------------------------------------- MMA issuers
      // (whole warps with one lane issuing, so that the operands are in uniform registers)
      constexpr uint32_t idesc = idesc_e4m3_f32(Cfg::kTileM, Cfg::kN);
      const int64_t total = static_cast<int64_t>(n_tiles) * G;
      const uint32_t buf = warp >> 1, d = tmem_base + buf * Cfg::kN;
      const uint64_t a0 = smem_desc_k_sw128(sbase + Cfg::a), b0 = smem_desc_k_sw128(sbase + Cfg::b);
      const bool leader = elect_one();
      uint32_t s = buf, phase = 0, acc_phase = 1;          // of the full barriers; of tempty
      for (int64_t it = buf; it < total; it += NB) {
        // the operands first (long in place), then the accumulator
        if (!mbar_wait_warp(full_bar(s), phase, kSiteMmaFull, abort_flag)) break;
        if (!mbar_wait_warp(tempty_bar(buf), acc_phase, kSiteMmaEmpty, abort_flag)) break;
        tc_fence_after();
        const uint64_t a = a0 + s * (Cfg::kABytes >> 4), b = b0 + s * (Cfg::kBBytes >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk) mma_f8<1>(d, a + 2 * kk, b + 2 * kk, idesc, kk > 0);
          mma_commit<1>(empty_bar(s));             // frees the stage and publishes the partial
        }
        acc_phase ^= 1;
        s += NB;
        if (s >= S) s -= S, phase ^= 1;
      }
      if (leader) {
        mma_commit<1>(drain_bar(buf));
        mbar_wait(drain_bar(buf), 0, kSiteDrain, nullptr);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------- scale producer
      uint32_t sl = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_tiles; ++i) {
        int64_t row0, col0;
        tile_at(i, row0, col0);
        const float* sW_tile = p.sW + (col0 + (lane & 1) * p.N) / 128 * G;   // lane 0 gate, 1 up
        for (int g0 = 0; g0 < G; g0 += SG, ++sl) {
          const int r = sl % R;
          if (!mbar_wait(sempty_bar(r), ((sl / R) & 1u) ^ 1u, kSiteScales, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t slot = sbase + Cfg::sring + 4u * Cfg::kSlotFloats * r;
          for (int k = 0; k < SG && g0 + k < G; ++k) {
            const float* sa_g = p.sA + static_cast<int64_t>(g0 + k) * p.ld_sa;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t m = row0 + 32 * j + lane;
              cp_async_4(slot + 4u * (SG * (32 * j + lane) + k), sa_g + (m < p.M ? m : 0), m < p.M);
            }
            if (lane < 2) cp_async_4(slot + 4u * (SG * (128 + lane) + k), sW_tile + g0 + k, true);
          }
          cp_async_arrive(sfull_bar(r));
        }
      }
      cp_async_wait_all();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsEpi));
    // ------------------------------------------------------------ promotion + epilogue
    // With two warps on a scheduler every dependent instruction of this loop costs its whole
    // latency, so it is kept short: running indices instead of divisions, one vector load for four
    // groups' scales, one arrival per warp, one vote per wait.
    const int quad = warp & 3, set = (warp - kEpiWarp0) >> 2;
    const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + set * Cfg::kSetCols;
    uint32_t s = 0, phase = 0, buf = 0, r = 0, rphase = 0;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int site) {      // warp-uniform outcome
      if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar, parity, site, abort_flag));
    };
    for (int i = 0; i < n_tiles; ++i) {
      float2 ag[32], au[32];                    // columns 2j, 2j + 1 of the gate's and up's 64
#pragma unroll
      for (int j = 0; j < 32; ++j) ag[j] = au[j] = make_float2(0.0f, 0.0f);
      for (int g0 = 0; g0 < G; g0 += SG) {
        wait(sfull_bar(r), rphase, kSiteScales);
        const float4* slot = reinterpret_cast<const float4*>(sring + Cfg::kSlotFloats * r);
        const float4 sa = slot[32 * quad + lane], sg = slot[128], su = slot[129];
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty_bar(r));         // the slot is in registers
        if (++r == R) r = 0, rphase ^= 1;
        const float cg4[4] = {sa.x * sg.x, sa.y * sg.y, sa.z * sg.z, sa.w * sg.w};
        const float cu4[4] = {sa.x * su.x, sa.y * su.y, sa.z * su.z, sa.w * su.w};
#pragma unroll
        for (int k = 0; k < SG; ++k) {
          if (g0 + k >= G) break;
          // the group's MMAs have completed: the commit on its stage's barrier (this wait cannot
          // lag by a phase: group it + S needs the accumulator freed after group it + S - 2)
          wait(empty_bar(s), phase, kSiteEpilogue);
          if (++s == S) s = 0, phase ^= 1;
          const uint32_t taddr = taddr0 + buf * Cfg::kN;
          if (ok) {
            tc_fence_after();
            const float2 cg = make_float2(cg4[k], cg4[k]), cu = make_float2(cu4[k], cu4[k]);
            uint32_t v[64];
            tmem_ld_64cols(taddr, v);
            tmem_ld_wait_regs(v);
            promote_chunk<false>(ag, v, cg, cg, nullptr);
            promote_chunk<false>(ag + 16, v + 32, cg, cg, nullptr);
            tmem_ld_64cols(taddr + Cfg::kTileN, v);
            tmem_ld_wait_regs(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(buf));   // free for group g + 2
            promote_chunk<false>(au, v, cu, cu, nullptr);
            promote_chunk<false>(au + 16, v + 32, cu, cu, nullptr);
          }
          buf ^= 1;
        }
      }
      int64_t row0, col0;
      tile_at(i, row0, col0);
      const int64_t m0 = row0 + 32 * quad, n0 = col0 + Cfg::kSetCols * set;
      if (!ok || m0 >= p.M) continue;         // warp-uniform
      const bool row_ok = m0 + lane < p.M;
      uint4 v[8];
      if constexpr (GU) {
        uint8_t* grow = reinterpret_cast<uint8_t*>(p.gu + (m0 + lane) * p.ld_gu + n0);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bf16x8(ag[4 * j], ag[4 * j + 1], ag[4 * j + 2], ag[4 * j + 3]);
        store_rows_by_quads(v, grow, row_ok);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bf16x8(au[4 * j], au[4 * j + 1], au[4 * j + 2], au[4 * j + 3]);
        store_rows_by_quads(v, grow + 2 * p.N, row_ok);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        ag[j].x = silu_mul(ag[j].x, au[j].x);
        ag[j].y = silu_mul(ag[j].y, au[j].y);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = bf16x8(ag[4 * j], ag[4 * j + 1], ag[4 * j + 2], ag[4 * j + 3]);
      store_rows_by_quads(v, reinterpret_cast<uint8_t*>(p.h + (m0 + lane) * p.ldh + n0), row_ok);
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<1>(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------- backward
//
// From dh [M, N] and the stored g, u (bf16 [M, 2N]):
//
//   sg = 1 / (1 + exp(-g))
//   dg = dh u sg (1 + g (1 - sg)),   du = dh g sg          (FP32, rounded to bf16)
//
// and of D = [dg | du] [M, 2N] both quantizations the two gradient products need: 1x128
// along the columns (q, s: dX = D W) and along the rows (qt, st: dW = D^T X), as
// fp8q_quant_act_dual makes them.  D itself is never written: 6 bytes read per element of
// h and 4 written, against 6 + 4 + 4 + 4 for an elementwise pass followed by the quantizer.
// Rows past M read as zeros, so qt and st cover M rounded up to 128 rows (zero codes,
// which add nothing to dW).
//
// Measured: 44 us (power-of-two scales) at 8192 x 2048, 0.58 of HBM; it issues 61 % of the time.
// With 256 threads per block, each quantizing both halves in turn, it took 50 us.
//
// Grid: one block of 512 threads per 128 x 128 tile of h, columns fastest, two to an SM.  The
// three bf16 input tiles come by TMA (two boxes of 64 columns each); dg replaces g and du
// replaces u in shared memory, and each is then quantized by the row and column passes of the
// quantizer, dg by the first eight warps and du by the others.
constexpr int kGatedBwdThreads = 512;
constexpr int kGatedBwdSmem = 3 * kDualTileBytes + 16 + 1024;
constexpr unsigned int kSiteGatedBwd = 10;

struct GatedBwdArgs {
  uint8_t* q;           // [M, 2N]
  float* s;             // [2N / 128][ld_s]
  uint8_t* qt;          // [2N, ceil128(M)]
  float* st;            // [ceil(M / 128)][ld_st]
  int64_t ldq, ld_s, ldqt, ld_st, M, N;
};

// dg and du of one bf16 pair each, from words of dh, g and u.
__device__ __forceinline__ void gated_grad_pair(uint32_t d, uint32_t& g, uint32_t& u) {
  auto one = [](float dh, float gv, float uv, float& dg, float& du) {
    const float sg = sigmoid(gv);
    const float ds = dh * sg;
    du = ds * gv;
    dg = ds * uv * fmaf(gv, 1.0f - sg, 1.0f);
  };
  float2 dg, du;
  one(bf16lo(d), bf16lo(g), bf16lo(u), dg.x, du.x);
  one(bf16hi(d), bf16hi(g), bf16hi(u), dg.y, du.y);
  __nv_bfloat162 a = __float22bfloat162_rn(dg), b = __float22bfloat162_rn(du);
  g = *reinterpret_cast<uint32_t*>(&a);
  u = *reinterpret_cast<uint32_t*>(&b);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

template <bool POW2>
__global__ void __launch_bounds__(kGatedBwdThreads, 2)
    gated_backward_quant_kernel(const __grid_constant__ CUtensorMap tmDh, const __grid_constant__ CUtensorMap tmGu,
                                const GatedBwdArgs p) {
  extern __shared__ uint8_t gbwd_raw[];
  const uint32_t tile = (smem_u32(gbwd_raw) + 1023u) & ~1023u;     // g, u, dh
  const uint32_t bar = tile + 3 * kDualTileBytes;
  const uint32_t nb = static_cast<uint32_t>(p.N / 128);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x % nb) * 128, m0 = static_cast<int64_t>(blockIdx.x / nb) * 128;
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar, 3 * kDualTileBytes);
    const int32_t y = static_cast<int32_t>(m0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t xg = static_cast<int32_t>(n0 + 64 * h), xu = static_cast<int32_t>(p.N + n0 + 64 * h);
      const uint32_t at = tile + h * (kDualTileBytes / 2);
      tma_load_2d(at, &tmGu, bar, xg, y);
      tma_load_2d(at + kDualTileBytes, &tmGu, bar, xu, y);
      tma_load_2d(at + 2 * kDualTileBytes, &tmDh, bar, xg, y);
    }
  }
  // bounded (the loads end on their own); a timeout is recorded and the tile skipped
  if (!__syncthreads_and(mbar_wait(bar, 0, kSiteGatedBwd, nullptr))) return;

  // the elementwise part, in place (the tiles share one swizzle, so equal offsets are equal
  // elements)
#pragma unroll 2
  for (int j = 0; j < 2048 / kGatedBwdThreads; ++j) {
    const uint32_t at = tile + 16u * (threadIdx.x + kGatedBwdThreads * j);
    const uint4 d = ld_shared_v4(at + 2 * kDualTileBytes);
    uint4 g = ld_shared_v4(at), u = ld_shared_v4(at + kDualTileBytes);
    gated_grad_pair(d.x, g.x, u.x);
    gated_grad_pair(d.y, g.y, u.y);
    gated_grad_pair(d.z, g.z, u.z);
    gated_grad_pair(d.w, g.w, u.w);
    st_shared_v4(at, g);
    st_shared_v4(at + kDualTileBytes, u);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, l4 = lane & 3;
  const int half = threadIdx.x >> 8, warp = (threadIdx.x >> 5) & 7;
  const uint32_t mine = tile + half * kDualTileBytes;
  const int64_t k0 = half * p.N + n0;
  dual_rows_pass<POW2, true>(lane, warp, l4, mine, m0, p.M, k0 / 128, k0, p.q, p.ldq, p.s, p.ld_s);
  dual_columns_pass<POW2>(lane, warp, l4, mine, m0, k0, p.qt, p.ldqt, p.st, p.ld_st);
}

// ---------------------------------------------------------------- rows and columns, any row count
//
// quant_act_dual_kernel for any number of rows: the tile's rows from M on read as zeros, are
// not written to q and s, and give zero codes in qt (and scale 1 where a whole tile of a column is
// zero), as the backward kernel above treats D.  Grid and shared memory as there.
template <bool POW2>
__global__ void __launch_bounds__(256, 5)
    quant_act_dual_padded_kernel(const __grid_constant__ CUtensorMap tmx, int64_t M, uint8_t* __restrict__ q,
                                 int64_t ldq, float* __restrict__ s, int64_t lds, uint8_t* __restrict__ qt,
                                 int64_t ldqt, float* __restrict__ st, int64_t ldst, uint32_t G) {
  extern __shared__ uint8_t padded_raw[];
  const uint32_t tile = (smem_u32(padded_raw) + 1023u) & ~1023u;
  const uint32_t bar = tile + kDualTileBytes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l4 = lane & 3;
  const int64_t g = blockIdx.x % G, m0 = static_cast<int64_t>(blockIdx.x / G) * 128;
  const int64_t k0 = g * 128;
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar, kDualTileBytes);
    tma_load_2d(tile, &tmx, bar, static_cast<int32_t>(k0), static_cast<int32_t>(m0));
    tma_load_2d(tile + kDualTileBytes / 2, &tmx, bar, static_cast<int32_t>(k0 + 64), static_cast<int32_t>(m0));
  }
  if (!__syncthreads_and(mbar_wait(bar, 0, kSiteDual, nullptr))) return;
  dual_rows_pass<POW2, true>(lane, warp, l4, tile, m0, M, g, k0, q, ldq, s, lds);
  dual_columns_pass<POW2>(lane, warp, l4, tile, m0, k0, qt, ldqt, st, ldst);
}

}  // namespace fp8q
