// What the forms of the int8 product share: how an int32 sum becomes an output.
#pragma once

#include "moe_internal.cuh"

namespace moe {
namespace i8 {

// g / (1 + exp(-g)) for results rounded to bf16: off by a few 2^-22 relative,
// and by 1.6 |g| 2^-24 from the exponent (exactly g or 0 far out).
__device__ __forceinline__ float quick_silu(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r;
}

// silu(g) * u, to the precision of an output of type O
template <typename O>
__device__ __forceinline__ float swiglu(float g, float u) {
  return (sizeof(O) == 2 ? quick_silu(g) : g / (1.f + expf(-g))) * u;
}

__device__ __forceinline__ void put(float* y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

}  // namespace i8

// Dense products of up to kFewRows rows, of kFewBytes together (gemm_i8_few.cu).
constexpr int kFewRows = 8;
constexpr int64_t kFewBytes = 96 * 1024;
cudaError_t launch_gemm_i8_few(const GemmI8Args& a);

}  // namespace moe
