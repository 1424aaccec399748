// int8 products over dense rows or expert windows: exact int32 sums, scaled in
// fp32 and rounded once.
//
// One block computes tiles of 64 rows x 64 channels with the four-way integer
// dot product; each of its 256 threads holds 4 x 4 sums (twice with an up
// projection).
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kThreads = 256, kWords = 16;   // K step: 16 words of 4 bytes

template <bool kUp, typename O>
__global__ void __launch_bounds__(kThreads) gemm_i8_kernel(GemmI8Args a) {
  __shared__ int sx[kTile][kWords + 1], sw[kTile][kWords + 1], su[kTile][kWords + 1];
  const int e = blockIdx.z, n0 = blockIdx.x * kTile;
  const int64_t N = a.d.N, K = a.d.K;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int64_t row0;
  const int rows = window_rows(a.win, e, a.d.M, &row0);
  for (int64_t m0 = (int64_t)blockIdx.y * kTile; m0 < rows; m0 += (int64_t)gridDim.y * kTile) {
    int acc[4][4] = {}, up[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += 4 * kWords) {
      // each thread moves one 16-byte piece of each tile (K is a multiple of 16)
      const int r = threadIdx.x >> 2, p = threadIdx.x & 3;
      const int64_t k = k0 + 16 * p;
      int4 vx = make_int4(0, 0, 0, 0), vw = vx, vu = vx;
      if (k < K) {
        if (m0 + r < rows) vx = *reinterpret_cast<const int4*>(a.x + (row0 + m0 + r) * K + k);
        if (n0 + r < N) {
          vw = *reinterpret_cast<const int4*>(a.w + ((int64_t)e * N + n0 + r) * K + k);
          if (kUp) vu = *reinterpret_cast<const int4*>(a.wu + ((int64_t)e * N + n0 + r) * K + k);
        }
      }
      __syncthreads();
      const int* px = &vx.x;
      const int* pw = &vw.x;
      const int* pu = &vu.x;
      for (int i = 0; i < 4; ++i) {
        sx[r][4 * p + i] = px[i];
        sw[r][4 * p + i] = pw[i];
        if (kUp) su[r][4 * p + i] = pu[i];
      }
      __syncthreads();
      for (int kk = 0; kk < kWords; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] = __dp4a(sx[ty + 16 * i][kk], sw[tx + 16 * j][kk], acc[i][j]);
            if (kUp) up[i][j] = __dp4a(sx[ty + 16 * i][kk], su[tx + 16 * j][kk], up[i][j]);
          }
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m >= rows || n >= N) continue;
        const float xs = a.xs[row0 + m];
        float v = (float)acc[i][j] * a.ws[(int64_t)e * N + n] * xs;
        if (kUp) v = v / (1.f + expf(-v)) * ((float)up[i][j] * a.wus[(int64_t)e * N + n] * xs);
        O* y = (O*)a.y + (row0 + m) * N + n;
        if constexpr (sizeof(O) == 2) *y = __float2bfloat16_rn(v);
        else *y = v;
      }
  }
}

}  // namespace

cudaError_t launch_gemm_i8(const GemmI8Args& a) {
  const int64_t nt = ceil_div(a.d.N, kTile), mt = ceil_div(a.d.M, kTile);
  const dim3 grid((unsigned)nt, (unsigned)(mt < 64 ? mt : 64), (unsigned)a.d.experts);
  const bool f32 = a.d.out_dtype == MOE_F32;
  if (a.wu) {
    if (f32) gemm_i8_kernel<true, float><<<grid, kThreads, 0, a.stream>>>(a);
    else gemm_i8_kernel<true, __nv_bfloat16><<<grid, kThreads, 0, a.stream>>>(a);
  } else {
    if (f32) gemm_i8_kernel<false, float><<<grid, kThreads, 0, a.stream>>>(a);
    else gemm_i8_kernel<false, __nv_bfloat16><<<grid, kThreads, 0, a.stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace moe
