// Rows to int8 with one scale each: scale = max |x| * (1 / 127), q = x / scale
// rounded to nearest even. The reciprocal, the product and the quotient are
// correctly rounded ones, so that the result is defined to the bit.
//
// One block per row (of all rows, or of the filled rows of windows).
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float load_x(const T* p) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
  else return *p;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
quant_i8_kernel(const T* __restrict__ x, int64_t rows, int cols, RowWindows win, int8_t* __restrict__ q,
                float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / 32];
  int64_t row0;
  const int n = window_rows(win, blockIdx.y, rows, &row0);
  for (int r = blockIdx.x; r < n; r += gridDim.x) {
    const T* xr = x + (row0 + r) * cols;
    // |x| as bits: ordered like the values, NaN and infinity above all numbers
    uint32_t m = 0;
    for (int i = threadIdx.x; i < cols; i += kThreads) m = max(m, __float_as_uint(load_x(xr + i)) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    __syncthreads();
    const bool bad = m >= 0x7F800000u;
    const float s = bad ? __int_as_float(0x7fc00000) : (m == 0 ? 1.f : fmaxf(__fmul_rn(__uint_as_float(m), 1.f / 127.f), 0x1p-126f));
    if (threadIdx.x == 0) scale[row0 + r] = s;
    for (int i = threadIdx.x; i < cols; i += kThreads)
      q[(row0 + r) * cols + i] = bad ? 0 : (int8_t)__float2int_rn(__fdiv_rn(load_x(xr + i), s));
  }
}

}  // namespace

cudaError_t launch_quant_i8(int64_t rows, int64_t cols, int32_t dtype, const void* x, const RowWindows& win,
                            int8_t* q, float* scale, int num_sms, cudaStream_t stream) {
  const int64_t most = (8 * num_sms + win.experts - 1) / win.experts;
  const dim3 grid((unsigned)(rows < most ? rows : most), win.experts);
  if (dtype == MOE_BF16)
    quant_i8_kernel<<<grid, kThreads, 0, stream>>>((const __nv_bfloat16*)x, rows, (int)cols, win, q, scale);
  else
    quant_i8_kernel<<<grid, kThreads, 0, stream>>>((const float*)x, rows, (int)cols, win, q, scale);
  return cudaGetLastError();
}

}  // namespace moe
