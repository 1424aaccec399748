// What the forms of the int8 product share: how an int32 sum becomes an output.
#pragma once

#include "moe_internal.cuh"

namespace moe {
namespace i8 {

// g / (1 + exp(-g)), g >= -80, for results rounded to bf16: off by a few 2^-22
// relative, and by 1.6 |g| 2^-24 from the exponent (exactly g far out).
__device__ __forceinline__ float quick_silu(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r;
}

// y = silu(g) * u, to the precision of an output of type O. Far below zero
// exp(-g) leaves binary32 before g exp(g) does: there 1 + exp(-g) is exp(-g) (to
// e^-80), and half of the exponent at a time keeps every factor normal. One
// look at the lowest of eight values is what that costs the others (4096 x 2048
// x 1024 bf16 32.8 us with or without; a look at each 36.9).
template <typename O, int kN>
__device__ __forceinline__ void swiglu(const float (&g)[kN], const float (&u)[kN], float* y) {
  float low = g[0];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    low = fminf(low, g[i]);
    y[i] = (sizeof(O) == 2 ? quick_silu(g[i]) : g[i] / (1.f + expf(-g[i]))) * u[i];
  }
  if (low < -80.f) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float h = expf(0.5f * g[i]);
      if (g[i] < -80.f) y[i] = g[i] * h * u[i] * h;
    }
  }
}
template <typename O>
__device__ __forceinline__ float swiglu(float g, float u) {
  const float gs[1] = {g}, us[1] = {u};
  float y[1];
  swiglu<O>(gs, us, y);
  return y[0];
}

__device__ __forceinline__ void put(float* y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

}  // namespace i8

// Dense products of up to kFewRows rows, of kFewBytes together (gemm_i8_few.cu).
constexpr int kFewRows = 8;
constexpr int64_t kFewBytes = 96 * 1024;
cudaError_t launch_gemm_i8_few(const GemmI8Args& a);

}  // namespace moe
