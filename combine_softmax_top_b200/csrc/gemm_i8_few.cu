// int8 products of up to eight dense rows (a few decoded tokens), without tensor
// cores: every weight is read once, and what counts is that all SMs read at
// once and soon. A warp takes kCh channels and goes along K 512 bytes at a time,
// 16 a lane: kCh loads of weights in flight for each step, the rows' pieces
// from shared memory, four-way integer dot products, and one integer reduction
// over the warp for every sum. Bound by latency and then by HBM.
//
// The tensor-core form needs 3.6 us for one slab of K (barriers, tensor memory,
// tensor maps) and 0.24 us for each further one. Here one row of 7168 x 2048
// takes 4.5 us against 8.9 (3.3 against 8.4 with the weights in L2), of 4096 x 7168
// 7.6 against 12.3 (4.4 against 10.7), where HBM alone would allow 2.2 and 4.5;
// launch_gemm_i8 says from where on the tensor cores are ahead.
#include "gemm_i8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStep = 512;   // bytes of K a warp takes at a time

__device__ __forceinline__ int dot16(int4 a, int4 b, int s) {
  s = __dp4a(a.x, b.x, s);
  s = __dp4a(a.y, b.y, s);
  s = __dp4a(a.z, b.z, s);
  return __dp4a(a.w, b.w, s);
}

template <int kM, int kCh, bool kUp, typename O>
__global__ void __launch_bounds__(kThreads, 2) gemm_i8_few_kernel(GemmI8Args a) {
  // loads in flight a lane, for two blocks an SM
  constexpr int kLoads = kM > 4 ? 8 : 16, kEach = kCh * (kUp ? 2 : 1), kUnroll = kLoads > kEach ? kLoads / kEach : 1;
  extern __shared__ int4 sx[];   // [M][K / 16]
  const int lane = threadIdx.x & 31;
  const int K16 = (int)(a.d.K / 16);
  const int N = (int)a.d.N;
  const int4* x = reinterpret_cast<const int4*>(a.x);
  const int M = (int)a.d.M;   // rows past the last repeat the first
  for (int i = threadIdx.x; i < M * K16; i += kThreads) sx[i] = __ldg(x + i);
  __syncthreads();
  const int warps = gridDim.x * kWarps;
  for (int64_t c0 = (int64_t)(blockIdx.x * kWarps + (threadIdx.x >> 5)) * kCh; c0 < N; c0 += (int64_t)warps * kCh) {
    int acc[kM][kCh] = {}, up[kM][kUp ? kCh : 1] = {};
#pragma unroll kUnroll
    for (int k = lane; k < K16; k += kStep / 16) {
      int4 w[kCh], u[kUp ? kCh : 1];
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        const int64_t at = (c0 + c < N ? c0 + c : c0) * K16 + k;   // channels past the last: the first once more
        w[c] = __ldcs(reinterpret_cast<const int4*>(a.w) + at);
        if (kUp) u[c] = __ldcs(reinterpret_cast<const int4*>(a.wu) + at);
      }
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int4 xv = sx[(m < M ? m : 0) * K16 + k];
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          acc[m][c] = dot16(xv, w[c], acc[m][c]);
          if (kUp) up[m][c] = dot16(xv, u[c], up[m][c]);
        }
      }
    }
    // lane m * kCh + c finishes row m, channel c
    int mine = 0, mine_up = 0;
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        const int s = __reduce_add_sync(0xffffffffu, acc[m][c]);
        const int t = kUp ? __reduce_add_sync(0xffffffffu, up[m][c]) : 0;
        if (lane == m * kCh + c) { mine = s; mine_up = t; }
      }
    const int m = lane / kCh;
    const int64_t n = c0 + lane % kCh;
    if (m < M && n < N) {
      const float xs = __ldg(a.xs + m);
      float v = (float)mine * __ldg(a.ws + n) * xs;
      if (kUp) v = i8::swiglu<O>(v, (float)mine_up * __ldg(a.wus + n) * xs);
      i8::put(reinterpret_cast<O*>(a.y) + (int64_t)m * N + n, v);
    }
  }
}

template <int kM, int kCh, bool kUp, typename O>
cudaError_t go(const GemmI8Args& a) {
  const int64_t need = ceil_div(ceil_div(a.d.N, kCh), kWarps), most = 2 * (int64_t)a.num_sms;
  const unsigned grid = (unsigned)(need < most ? need : most);
  const size_t smem = (size_t)(a.d.M * a.d.K);   // at most kFewBytes
  auto* kernel = gemm_i8_few_kernel<kM, kCh, kUp, O>;
  if (smem > 48 * 1024) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewBytes);
    if (err != cudaSuccess) return err;
  }
  kernel<<<grid, kThreads, smem, a.stream>>>(a);
  return cudaGetLastError();
}

template <int kM, int kCh>
cudaError_t by_form(const GemmI8Args& a) {
  const bool f32 = a.d.out_dtype == MOE_F32;
  if (a.wu) return f32 ? go<kM, kCh, true, float>(a) : go<kM, kCh, true, __nv_bfloat16>(a);
  return f32 ? go<kM, kCh, false, float>(a) : go<kM, kCh, false, __nv_bfloat16>(a);
}

template <int kM>
cudaError_t by_channels(const GemmI8Args& a) {
  // four channels a warp while that leaves every SM some (7168 channels: 12
  // warps an SM), else one
  return a.d.N >= 16 * (int64_t)a.num_sms ? by_form<kM, 4>(a) : by_form<kM, 1>(a);
}

}  // namespace

cudaError_t launch_gemm_i8_few(const GemmI8Args& a) {
  if (a.d.M == 1) return by_channels<1>(a);
  if (a.d.M == 2) return by_channels<2>(a);
  return a.d.M <= 4 ? by_channels<4>(a) : by_channels<8>(a);
}

}  // namespace moe
