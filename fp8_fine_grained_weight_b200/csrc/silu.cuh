// The activation of the gated feed-forward kernels.
#pragma once

namespace fp8q {

// 1 / (1 + exp(-g)) by the hardware's base-2 exponential and reciprocal: exp within 2 + 0.75 |g|
// units of 2^-23 (2^-22 for ex2, the rounding of g log2(e) and of the constant), the sum rounded
// once, the reciprocal within one unit.  For g < -87.3 the divisor passes 2^126 and the result is
// returned as 0; silu(g) is above -1.2e-36 there.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid(g) * u; }

}  // namespace fp8q
