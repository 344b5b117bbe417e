// The products for few rows: INT8 (plain and gated) and the gated block-scaled FP8 product for
// decode batches and single tokens (sm_100a: tcgen05 + TMEM + TMA, clusters).
//
// With few rows of A the weight's bytes bound the product, and a grid of 128-row tiles of A
// would use a few SMs only.  So the operands change places: the tensor core's 128 rows are
// rows of the weight, its MP columns are rows of A (MP = 16 .. 128, rows past M read as
// zeros), and K is split over the CTAs of a cluster of at most four, so that up to two CTAs per SM
// stream the weight (a gated product of N = 2048 has 32 tiles: 128 CTAs in all).  Their partial sums meet in shared memory: each CTA leaves its
// [MP][128] partials in its own, the cluster synchronizes, and each CTA sums a slice of the outputs
// over the cluster in CTA order (a fixed order; INT32 sums are exact in any) and finishes it:
// one launch, no workspace, no atomics.
//
// GATED: the 128 weight rows are 64 gate rows and the same 64 up rows (two TMA boxes).
//
//   warp 0      TMA producer: weight [128 x 128 B] and A [MP x 128 B] per 128 K-elements
//   warp 1      TMEM owner and MMA issuer.  INT8: one accumulator over the CTA's K range.
//               FP8: a fresh accumulator (of four) per group, promoted by the epilogue.
//   warp 2      FP8: scale producer, MP row scales and the two weight scales per group
//               INT8: puts the tile's row and weight scales into shared memory
//   warp 3      idle; FP8 whose scales shall be powers of two: checks them
//   warps 4-7   epilogue: thread t owns weight row t of the tile.  FP8: per group
//               acc[m] += (P sW) sA[m] in FP32 registers.
// Measured: INT8 1 x 7168 x 2048 in 7.1 us, 64 x 7168 x 7168 in 13.8 us (8 us of streaming at the
// HBM rate, 2 of launch, the rest joining the sums); FP8 gated 16 x 2048 x 7168 in 10.0 us (the
// wide kernel: 31).  Against the wide kernels at more rows: beside the rule that chooses.
//
// All eight warps then sum the slices.  Two CTAs fit on an SM (about 100 KB, 128 registers).
//
// A decode step's product lasts a few microseconds, so what is not streaming counts (cycles of 7900
// at 1 x 7168 x 2048 before: 1100 until the first load was issued, 1400 in a barrier that waited
// for the outputs to be written): the first loads go out before the CTA has synchronized, the
// scales are in shared memory before they are needed, and the last cluster barrier orders nothing
// but the reads of the partials.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include "ptx.cuh"
#include "gemm.cuh"
#include "gemm_ue8m0.cuh"
#include "int8.cuh"

namespace fp8q {

enum SkinnyKind { kSkinnyInt8 = 0, kSkinnyFp8 = 1 };

struct SkinnyArgs {
  const float* sA;      // INT8: [M]; FP8: group-major [G][ld_sa]
  int64_t ld_sa;
  const float* sB;      // INT8: a scale per weight row; FP8: [2N / 128][G]
  void* C;
  int64_t ldc;
  __nv_bfloat16* gu;    // FP8: g and u in bf16 when set
  int64_t ld_gu, M, N;
  int G;                // groups of 128 K-elements
  int nt;               // weight tiles
  int split;            // CTAs per cluster, at most kMaxSplit
  int vec;              // C takes four elements at a time
  int pow2;             // FP8: report scales that are not powers of two
};

constexpr int kMaxSplit = 4;

template <int KIND, int MP>
struct SkinnyCfg {
  static constexpr int kThreads = 256;
  static constexpr int kStages = MP == 16 ? 5 : (MP == 128 ? 3 : 4);
  static constexpr int kAccBufs = KIND == kSkinnyFp8 ? 4 : 1;
  static constexpr uint32_t kAccCols = kAccBufs * MP < 32 ? 32 : kAccBufs * MP;   // a power of two
  // FP8: scales of one group per slot; INT8: one slot, the tile's row scales and 128 weight scales
  static constexpr int kScaleSlots = KIND == kSkinnyFp8 ? 8 : 1;
  static constexpr uint32_t kSlotFloats = KIND == kSkinnyFp8 ? MP + 4 : MP + 128;
  static constexpr uint32_t kWBytes = 128 * kBK, kABytes = MP * kBK, kStageTx = kWBytes + kABytes;
  static constexpr uint32_t w = 0;
  static constexpr uint32_t a = w + kStages * kWBytes;
  static constexpr uint32_t sring = a + kStages * kABytes;
  static constexpr uint32_t bars = sring + 4 * kScaleSlots * kSlotFloats;
  // full[S], empty[S], tfull[NB], tempty[NB], sfull[R], sempty[R], drain
  static constexpr uint32_t misc = align_up(bars + 8 * (2 * kStages + 2 * kAccBufs + 2 * kScaleSlots + 1), 16);
  static constexpr uint32_t smem_bytes = misc + 16 + 1024;
  static constexpr uint32_t part = 0;                      // [MP][128] partials, over the ring
  static_assert(MP * 128 * 4 <= kStages * (kWBytes + kABytes), "the partials fit in the ring");
  static_assert(kABytes % 1024 == 0 && a % 1024 == 0, "swizzle atoms");
  static_assert(2 * (smem_bytes + 1024) <= 233472, "two CTAs per SM");
  static_assert(kAccCols <= 256, "two CTAs share the tensor memory");
  static_assert(KIND == kSkinnyInt8 || MP <= 64, "FP8 keeps MP running sums in registers");
};

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint2 bf16x4(const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// TMEM columns of this warp's lanes into registers, by the count.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_16cols(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32cols(taddr, r); }

// The wait of a 16-column load, naming its registers (see tmem_ld_wait_regs).
__device__ __forceinline__ void tmem_ld_wait_regs(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

template <int KIND, bool GATED, bool OUT_BF16, int MP>
__global__ void __launch_bounds__(256, 2)
    gemm_skinny_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                       const SkinnyArgs p) {
  using Cfg = SkinnyCfg<KIND, MP>;
  constexpr bool FP8 = KIND == kSkinnyFp8;
  static_assert(GATED || !FP8, "the plain FP8 product has its own kernels");
  static_assert(OUT_BF16 || !GATED, "the gated product is bf16");
  constexpr int S = Cfg::kStages, NB = Cfg::kAccBufs, R = Cfg::kScaleSlots;
  constexpr int kCols = GATED ? 64 : 128;                  // output columns per tile
  constexpr int kChunk = MP < 32 ? 16 : 32;                // TMEM columns per load
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::bars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + NB + b); };
  auto sfull_bar = [&](int r) { return bar0 + 8u * (2 * S + 2 * NB + r); };
  auto sempty_bar = [&](int r) { return bar0 + 8u * (2 * S + 2 * NB + R + r); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 2 * NB + 2 * R);
  float* sring = reinterpret_cast<float*>(smem + Cfg::sring);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int unit = blockIdx.x / p.split;
  const int64_t col0 = static_cast<int64_t>(unit % p.nt) * kCols, row0 = static_cast<int64_t>(unit / p.nt) * MP;
  const int g0 = static_cast<int>(static_cast<int64_t>(p.G) * rank / p.split);
  const int n_g = static_cast<int>(static_cast<int64_t>(p.G) * (rank + 1) / p.split) - g0;   // >= 1

  auto load_stage = [&](int it) {
    const int s = it % S;
    mbar_arrive_expect_tx(full_bar(s), Cfg::kStageTx);
    const uint32_t w = sbase + Cfg::w + s * Cfg::kWBytes;
    const int32_t x = (g0 + it) * kBK;
    tma_load_2d(w, &tmW, full_bar(s), x, static_cast<int32_t>(col0));
    if (GATED) tma_load_2d(w + 64 * kBK, &tmW, full_bar(s), x, static_cast<int32_t>(p.N + col0));
    tma_load_2d(sbase + Cfg::a + s * Cfg::kABytes, &tmA, full_bar(s), x, static_cast<int32_t>(row0));
  };
  const int n_first = n_g < S ? n_g : S;                   // stages that wait for nothing
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 128);
    }
    for (int r = 0; r < R; ++r) {
      mbar_init(sfull_bar(r), 32);
      mbar_init(sempty_bar(r), 128);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    for (int it = 0; it < n_first; ++it) load_stage(it);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_slot), Cfg::kAccCols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // -------------------------------------------------------------- TMA producer
    // (here and in the issuer: whole warps with one lane issuing, so that the operands are in
    // uniform registers)
    __syncwarp();
    const bool leader = elect_one();
    int it = n_first;
    for (; it < n_g; ++it) {
      if (!mbar_wait_warp(empty_bar(it % S), ((it / S) & 1u) ^ 1u, kSiteProducer, abort_flag)) break;
      if (leader) load_stage(it);
    }
    // every issued load lands before the ring is reused (bounded; loads end on their own)
    for (int j = it > S ? it - S : 0; j < it; ++j) mbar_wait(full_bar(j % S), (j / S) & 1u, kSiteDrain, nullptr);
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = FP8 ? idesc_e4m3_f32(128, MP) : idesc_s8_s32(128, MP);
    const uint64_t w0 = smem_desc_k_sw128(sbase + Cfg::w), a0 = smem_desc_k_sw128(sbase + Cfg::a);
    const bool leader = elect_one();
    bool ok = true;
    for (int it = 0; it < n_g; ++it) {
      const int s = it % S, b = it % NB;
      ok = mbar_wait_warp(full_bar(s), (it / S) & 1u, kSiteMmaFull, abort_flag);
      if (ok && FP8) ok = mbar_wait_warp(tempty_bar(b), ((it / NB) & 1u) ^ 1u, kSiteMmaEmpty, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint64_t w = w0 + s * (Cfg::kWBytes >> 4), a = a0 + s * (Cfg::kABytes >> 4);
      const uint32_t d = tmem_base + b * MP;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk) {
          if (FP8) mma_f8<1>(d, w + 2 * kk, a + 2 * kk, idesc, kk > 0);
          else mma_i8<1>(d, w + 2 * kk, a + 2 * kk, idesc, it > 0 || kk > 0);
        }
        mma_commit<1>(empty_bar(s));
        if (FP8) mma_commit<1>(tfull_bar(b));
      }
    }
    if (leader) {
      if (!FP8 && ok) mma_commit<1>(tfull_bar(0));
      mma_commit<1>(drain_bar);
      mbar_wait(drain_bar, 0, kSiteDrain, nullptr);
    }
  } else if (FP8 && warp == 2) {
    // -------------------------------------------------------------- scale producer
    const float* sW = p.sB + (col0 + (lane & 1) * p.N) / 128 * p.G;        // lane 0 gate, 1 up
    for (int it = 0; it < n_g; ++it) {
      const int r = it % R;
      if (!mbar_wait(sempty_bar(r), ((it / R) & 1u) ^ 1u, kSiteScales, abort_flag)) break;
      const uint32_t slot = sbase + Cfg::sring + 4u * Cfg::kSlotFloats * r;
      const float* sa = p.sA + static_cast<int64_t>(g0 + it) * p.ld_sa;
#pragma unroll
      for (int j = 0; j < (MP + 31) / 32; ++j) {
        const int64_t m = row0 + 32 * j + lane;
        if (32 * j + lane < MP) cp_async_4(slot + 4u * (32 * j + lane), sa + (m < p.M ? m : 0), m < p.M);
      }
      if (lane < 2) cp_async_4(slot + 4u * (MP + lane), sW + g0 + it, true);
      cp_async_arrive(sfull_bar(r));
    }
    cp_async_wait_all();
  } else if (FP8 && warp == 3) {
    if (p.pow2) {
      bool bad = false;
      const float* sW = p.sB + (col0 + (lane & 1) * p.N) / 128 * p.G + g0;
      for (int i = lane >> 1; i < n_g; i += 16) ue8m0_of(__ldg(sW + i), bad);
      for (int it = 0; it < n_g; ++it)
        for (int64_t m = row0 + lane; m < row0 + MP && m < p.M; m += 32)
          ue8m0_of(__ldg(p.sA + static_cast<int64_t>(g0 + it) * p.ld_sa + m), bad);
      if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) record_error((kSiteScaleFormat << 8) | kErrScale);
    }
  } else if (!FP8 && warp == 2) {
    // read after the cluster barrier below
    for (int m = lane; m < MP; m += 32) sring[m] = row0 + m < p.M ? __ldg(p.sA + row0 + m) : 0.0f;
    for (int c = lane; c < 128; c += 32) {
      const bool up = c >= kCols;                          // GATED: 64 gate scales, 64 up scales
      const int64_t n = col0 + (up ? c - kCols : c);
      sring[MP + c] = n < p.N ? __ldg(p.sB + (up ? p.N : 0) + n) : 0.0f;
    }
  }

  // The CTA's partials, [m][weight row].  The ring is free to hold them: the last group's
  // products have completed, and with them every load.
  uint32_t* part = reinterpret_cast<uint32_t*>(smem + Cfg::part);
  if (warp >= 4) {
    const int quad = warp & 3;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * quad) << 16);
    uint32_t* mine = part + 32 * quad + lane;
    if constexpr (FP8) {
      float2 acc[MP / 2];
#pragma unroll
      for (int j = 0; j < MP / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      bool ok = true;
      for (int it = 0; it < n_g; ++it) {
        const int r = it % R, b = it % NB;
        if (ok) ok = mbar_wait(sfull_bar(r), (it / R) & 1u, kSiteScales, abort_flag);
        if (ok) ok = mbar_wait(tfull_bar(b), (it / NB) & 1u, kSiteEpilogue, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        const float* slot = sring + Cfg::kSlotFloats * r;
        const float sw = slot[MP + (quad >> 1)];           // rows 0-63 gate, 64-127 up
        const float2 sw2 = make_float2(sw, sw);
#pragma unroll
        for (int c = 0; c < MP; c += kChunk) {
          uint32_t v[kChunk];
          tmem_ld_cols(taddr + b * MP + c, v);
          tmem_ld_wait_regs(v);
          if (c + kChunk == MP) {
            tc_fence_before();
            mbar_arrive(tempty_bar(b));
          }
#pragma unroll
          for (int j = 0; j < kChunk; j += 4) {
            const float4 sa = *reinterpret_cast<const float4*>(slot + c + j);
            const float2 p0 = make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            const float2 p1 = make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
            float2& a0 = acc[(c + j) / 2];
            float2& a1 = acc[(c + j) / 2 + 1];
            a0 = __ffma2_rn(__fmul2_rn(p0, sw2), make_float2(sa.x, sa.y), a0);
            a1 = __ffma2_rn(__fmul2_rn(p1, sw2), make_float2(sa.z, sa.w), a1);
          }
        }
        mbar_arrive(sempty_bar(r));
      }
#pragma unroll
      for (int j = 0; j < MP / 2; ++j) {
        mine[128 * (2 * j)] = __float_as_uint(acc[j].x);
        mine[128 * (2 * j + 1)] = __float_as_uint(acc[j].y);
      }
    } else {
      const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(tfull_bar(0), 0, kSiteEpilogue, abort_flag));
      if (ok) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < MP; c += kChunk) {
          uint32_t v[kChunk];
          tmem_ld_cols(taddr + c, v);
          tmem_ld_wait_regs(v);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) mine[128 * (c + j)] = v[j];
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();

  // ------------------------------------------------------------------ sum and finish
  // Four consecutive columns of a row per thread and step, so that few steps wait for the
  // other CTAs' shared memory.
  const int rows = static_cast<int>(p.M - row0 < MP ? p.M - row0 : MP);
  const uint32_t part_u32 = sbase + Cfg::part;
  auto total = [&](int m, int r, float (&t)[4]) {          // over the cluster, in CTA order
    uint4 v[kMaxSplit];
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s)
      v[s] = s < p.split ? ld_cluster_v4(map_shared_rank(part_u32 + 4u * (128 * m + r), s)) : make_uint4(0, 0, 0, 0);
    uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int s = 1; s < kMaxSplit; ++s) {
      const uint32_t a[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = FP8 ? __float_as_uint(__uint_as_float(w[j]) + __uint_as_float(a[j])) : w[j] + a[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = FP8 ? __uint_as_float(w[j]) : __int2float_rn(static_cast<int>(w[j]));
  };
  for (int e = rank * Cfg::kThreads + threadIdx.x; e < rows * (kCols / 4); e += p.split * Cfg::kThreads) {
    const int m = e / (kCols / 4), c = 4 * (e % (kCols / 4));
    const int64_t n = col0 + c, row = row0 + m;
    const int left = static_cast<int>(p.N - n < 4 ? p.N - n : 4);
    if (left <= 0) continue;
    float v[4], u[4];
    total(m, c, v);
    if constexpr (GATED) total(m, 64 + c, u);
    if constexpr (!FP8) {
      const float sa = sring[m];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = (v[j] * sa) * sring[MP + c + j];
        if (GATED) u[j] = (u[j] * sa) * sring[MP + 64 + c + j];
      }
    }
    if constexpr (GATED) {
      if constexpr (FP8) {
        if (p.gu != nullptr) {                             // N % 128 == 0, rows on 16 bytes
          *reinterpret_cast<uint2*>(p.gu + row * p.ld_gu + n) = bf16x4(v);
          *reinterpret_cast<uint2*>(p.gu + row * p.ld_gu + p.N + n) = bf16x4(u);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = silu_mul(v[j], u[j]);
    }
    if (OUT_BF16) {
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.C) + row * p.ldc + n;
      if (p.vec && left == 4) {
        *reinterpret_cast<uint2*>(out) = bf16x4(v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) out[j] = __float2bfloat16_rn(v[j]);
      }
    } else {
      float* out = reinterpret_cast<float*>(p.C) + row * p.ldc + n;
      if (p.vec && left == 4) {
        *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) out[j] = v[j];
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  // The partials stay until all have read them (each read has been used: nothing to order).
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem_base, Cfg::kAccCols);
  }
}

}  // namespace fp8q
