// Rows to int8 with one scale each: scale = max |x| * (1 / 127), q = x / scale
// rounded to nearest even. The reciprocal, the product and the quotient are
// correctly rounded ones, so that the result is defined to the bit.
//
// Bound by HBM: 3 bytes an element of bf16 rows (5 of fp32), read once. A team
// of threads (part of a warp, a warp, or a block of four for rows beyond 8 KB)
// keeps its row in registers between the maximum and the quantisation, 16 bytes
// a thread and step; what a row has beyond the registers is read again. Warps
// with rows of their own meet no barrier, and while some reduce, the others'
// loads are in flight. 8192 x 7168 bf16: 30 us, 5.9 TB/s; one row 1.8 us.
//
// A division instruction sequence costs some twenty instructions an element,
// which would be the bound instead. With y the rounded reciprocal of s, one a
// row, q0 = x y is within two units of the quotient, q1 = q0 + (x - q0 s) y
// within one, and q2 = q1 + (x - q1 s) y, each an fma, is then the correctly
// rounded quotient (Markstein's theorem: y correctly rounded, q1 within one
// unit, the remainder exact). Rows whose remainders could leave the normal
// numbers are scaled by 2^64 first, which changes no quotient. Adding
// 1.5 * 2^23 rounds to an integer, ties to even, whose low byte is the code.
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxExperts = 1024;

// 16 bytes of consecutive elements, as loaded.
template <typename T>
struct Piece {
  static constexpr int kN = 16 / sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // |x| as bits, ordered like the values, NaN and infinity above all numbers:
  // of fp32 as they are, of bf16 two elements side by side (most_of joins them)
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) m = max(m, w[i] & 0x7FFFFFFFu);
      else m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    }
    return m;
  }
  static __device__ __forceinline__ uint32_t most_of(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    else return max(m & 0xFFFF0000u, m << 16);
  }
  template <bool kTiny>
  __device__ __forceinline__ void quantise(float s, float y, int8_t* q) const {
    const uint64_t y2 = ptx::two(y, y), minus_s = ptx::two(-s, -s), magic = ptx::two(12582912.f, 12582912.f);   // 1.5 * 2^23
    float t[kN];
#pragma unroll
    for (int i = 0; i < kN; i += 2) {   // two elements an instruction
      uint64_t x = ptx::two(at(i), at(i + 1));
      if (kTiny) x = ptx::mul2(x, ptx::two(0x1p64f, 0x1p64f));
      uint64_t v = ptx::mul2(x, y2);
      v = ptx::fma2(ptx::fma2(v, minus_s, x), y2, v);
      v = ptx::fma2(ptx::fma2(v, minus_s, x), y2, v);
      v = ptx::add2(v, magic);
      ptx::split(v, t[i], t[i + 1]);
    }
    uint32_t b[kN / 4];
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      b[i] = __byte_perm(__byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040),
                         __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040), 0x5410);
    store(b, q);
  }
  static __device__ __forceinline__ void store(const uint32_t (&b)[kN / 4], int8_t* q) {   // kN codes
    if constexpr (kN == 8) *reinterpret_cast<uint2*>(q) = make_uint2(b[0], b[1]);
    else *reinterpret_cast<uint32_t*>(q) = b[0];
  }
};

// kTeam threads a row, kKeep steps of it in registers.
template <typename T, int kTeam, int kKeep>
__global__ void __launch_bounds__(kThreads, kKeep <= 8 ? 8 : 5)
quant_i8_kernel(const T* __restrict__ x, int64_t rows, int cols, RowWindows win, int8_t* __restrict__ q,
                float* __restrict__ scale) {
  __shared__ uint32_t part[2][kThreads / 32];
  __shared__ int first[kMaxExperts + 1];   // rows of the windows before each window
  const int tid = threadIdx.x % kTeam, lane = threadIdx.x & 31;
  int total = (int)rows;
  if (win.offsets) {
    if (threadIdx.x < 32)
      window_prefix(win, rows, rows, [](int n) { return n; }, first);
    __syncthreads();
    total = first[win.experts];
  }
  constexpr int kTeams = kThreads / kTeam;
  int turn = 0;
  for (int64_t i0 = (int64_t)blockIdx.x * kTeams + threadIdx.x / 32 * (kTeam < 32 ? 32 / kTeam : 1) / (kTeam > 32 ? kTeam / 32 : 1);
       i0 < total; i0 += (int64_t)gridDim.x * kTeams, turn ^= 1) {
    // teams of one warp past the last row do that row once more, without storing
    const int64_t mine = i0 + (kTeam < 32 ? lane / kTeam : 0), i = mine < total ? mine : total - 1;
    const bool real = mine < total;
    int64_t r = i;
    if (win.offsets) {   // the last window that starts at or before row i (empty ones never do)
      int lo = 0, hi = win.experts - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      r = (int64_t)__ldg(win.offsets + lo) + (i - first[lo]);
    }
    const T* xr = x + r * cols;
    int8_t* qr = q + r * cols;
    Piece<T> kept[kKeep];
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < kKeep; ++g) {
      const int c = (g * kTeam + tid) * Piece<T>::kN;
      if (c < cols) kept[g].load(xr + c);
      else kept[g].zero();
    }
#pragma unroll
    for (int g = 0; g < kKeep; ++g) m = kept[g].most(m);
    for (int c = (kKeep * kTeam + tid) * Piece<T>::kN; c < cols; c += kTeam * Piece<T>::kN) {
      Piece<T> more;
      more.load(xr + c);
      m = more.most(m);
    }
    m = Piece<T>::most_of(m);
    if constexpr (kTeam >= 32) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int off = kTeam / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
    if constexpr (kTeam > 32) {   // two slots in turn: one barrier a row
      if (lane == 0) part[turn][threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kTeam / 32; ++w) m = max(m, part[turn][w]);
    }
    const bool bad = m >= 0x7F800000u;
    const float s = bad ? __int_as_float(0x7fc00000)
                        : (m == 0 ? 1.f : fmaxf(__fmul_rn(__uint_as_float(m), 1.f / 127.f), 0x1p-126f));
    const bool tiny = s < 0x1p-60f;
    const float up = tiny ? s * 0x1p64f : s, y = __frcp_rn(up);
    if (!real) continue;
    if (tid == 0) scale[r] = s;
    auto put = [&](const Piece<T>& v, int c) {
      if (bad) {
        const uint32_t none[Piece<T>::kN / 4] = {};
        Piece<T>::store(none, qr + c);
      } else if (tiny) {
        v.template quantise<true>(up, y, qr + c);
      } else {
        v.template quantise<false>(up, y, qr + c);
      }
    };
#pragma unroll
    for (int g = 0; g < kKeep; ++g) {
      const int c = (g * kTeam + tid) * Piece<T>::kN;
      if (c < cols) put(kept[g], c);
    }
    for (int c = (kKeep * kTeam + tid) * Piece<T>::kN; c < cols; c += kTeam * Piece<T>::kN) {
      Piece<T> more;
      more.load(xr + c);
      put(more, c);
    }
  }
}

template <typename T, int kTeam, int kKeep>
cudaError_t go(int64_t rows, int64_t cols, const void* x, const RowWindows& win, int8_t* q, float* scale, int num_sms,
               cudaStream_t stream) {
  // as many blocks as are resident where each first has to add up the windows
  // (1024 rows in 256 windows: 9.9 us with twice as many, 7.8 us)
  const int64_t need = ceil_div(rows, kThreads / kTeam), most = (win.offsets ? 8 : 16) * (int64_t)num_sms;
  quant_i8_kernel<T, kTeam, kKeep>
      <<<(unsigned)(need < most ? need : most), kThreads, 0, stream>>>((const T*)x, rows, (int)cols, win, q, scale);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_cols(int64_t rows, int64_t cols, const void* x, const RowWindows& win, int8_t* q, float* scale,
                    int num_sms, cudaStream_t stream) {
  const int64_t bytes = cols * (int64_t)sizeof(T);
  // few rows: a block each, so that one row is not one warp's work
  const bool few = rows < 4 * (int64_t)num_sms;
  if (bytes <= 256 && !few) return go<T, 8, 2>(rows, cols, x, win, q, scale, num_sms, stream);
  if (bytes <= 1024) return go<T, 32, 2>(rows, cols, x, win, q, scale, num_sms, stream);
  if (!few) {
    if (bytes <= 2048) return go<T, 32, 4>(rows, cols, x, win, q, scale, num_sms, stream);
    if (bytes <= 4096) return go<T, 32, 8>(rows, cols, x, win, q, scale, num_sms, stream);
    if (bytes <= 8192) return go<T, 32, 16>(rows, cols, x, win, q, scale, num_sms, stream);
  }
  if (bytes <= 16384) return go<T, 128, 8>(rows, cols, x, win, q, scale, num_sms, stream);
  return go<T, 128, 16>(rows, cols, x, win, q, scale, num_sms, stream);
}

}  // namespace

cudaError_t launch_quant_i8(int64_t rows, int64_t cols, int32_t dtype, const void* x, const RowWindows& win,
                            int8_t* q, float* scale, int num_sms, cudaStream_t stream) {
  return dtype == MOE_BF16 ? by_cols<__nv_bfloat16>(rows, cols, x, win, q, scale, num_sms, stream)
                           : by_cols<float>(rows, cols, x, win, q, scale, num_sms, stream);
}

}  // namespace moe
