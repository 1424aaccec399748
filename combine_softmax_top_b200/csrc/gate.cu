// The gate: routing with softmax or sigmoid scores, a balance bias, expert
// groups, top-k and renormalised, scaled weights; and its gradient.
//
// gate_kernel gives a token a set of S lanes: a warp, or for many tokens a half
// or a quarter of one, which shares the work that does not grow with E. Lane i
// holds `per` = ceil(E / S) consecutive experts from i * per on, so that for
// most groupings a group is a power-of-two set of lanes. Each lane sorts 32-bit
// keys that order like its choice values c, their low 6 to 10 bits given to the
// expert (a sorting network of min and max, two instructions a comparison), and
// each of the topk rounds takes the largest head with one reduction, which
// names the expert too, and pops it (two heads in registers, the rest of a list in
// shared memory: 32768 x 128 bf16 8.5 us, all in registers 10.1).
//
// What is chosen has to be what binary64 chooses. The keys drop low bits and
// c = s + bias carries binary32 roundings, so the chosen values (and the best
// one left) are compared once more with the bounds of both. Where two
// neighbours are closer than that, every candidate that could still belong to
// the topk is popped, one to a lane, and these are ordered in binary64. Groups
// at the border of the open ones closer than that are ranked in binary64, by the
// experts that can be their best, and all else is done over (few tokens, kClose),
// or the token is chosen in binary64 altogether (choose_exactly). Without a bias
// c is the logit itself; bf16 logits then lose nothing in the keys and need no
// second look.
//
// For many tokens neither HBM nor issue is the bound, but rounds of warps, each
// with its load uncovered: 709 warp instructions a token of 256 f32 logits with a
// bias and groups take 69 % of the issue slots (40 registers: 48 warps an SM for
// 55 tokens an SM of 8192), 143 of 128 bf16 ones 52 % (69 to 72 registers: 28 warps
// an SM for 55). For few it is latency. One token 2.7 us, 8192 x 256 f32 8.8 us, 32768
// x 128 bf16 8.2 us (1.0 and 1.0 TB/s of logits, where HBM would allow 6.5).
//
// gate_backward_kernel writes what every expert gets (zero, or -p_e dot for a
// plain softmax) 16 bytes a lane, then the chosen experts' derivatives over it.
// The row is read only for a plain softmax, once where registers hold it. 8192 x
// 256 f32, renormalised: 3.4 us (2.7 TB/s); 32768 x 128 bf16, plain softmax, 4.9 us
// (3.9 TB/s), both mostly launch and latency; 32768 x 1024 f32 42 us (6.4 TB/s).
#include <algorithm>
#include <type_traits>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kNoKey = 0u;
constexpr uint32_t kLeastKey = 0x00800000u;   // of the lowest number; -infinity's is below

// 32-bit key that orders like the number, -0 below +0
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
  else return *p;
}

template <typename T>
__device__ __forceinline__ void store_grad(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(v);
  else *p = v;
}

// four elements at an address that is a multiple of their size
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 q = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(q.x << 16);
  v[1] = __uint_as_float(q.x & 0xFFFF0000u);
  v[2] = __uint_as_float(q.y << 16);
  v[3] = __uint_as_float(q.y & 0xFFFF0000u);
}
template <int kW, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[kW]) {
  if constexpr (kW == 1) {
    v[0] = load_logit(p);
  } else {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if constexpr (kW == 4) {
        v[b] = __uint_as_float(w[b]);
      } else {
        v[2 * b] = __uint_as_float(w[b] << 16);
        v[2 * b + 1] = __uint_as_float(w[b] & 0xFFFF0000u);
      }
    }
  }
}
template <int kW, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[kW]) {
  if constexpr (kW == 1) {
    store_grad(p, v[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if constexpr (kW == 4) {
        w[b] = __float_as_uint(v[b]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * b], v[2 * b + 1]);
        w[b] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Reductions over the S lanes of a token (all 32 lanes take part).
template <int S, typename V>
__device__ __forceinline__ V sub_sum(V v) {
#pragma unroll
  for (int off = S / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
template <int S>
__device__ __forceinline__ float sub_max(float v) {
  if constexpr (S == 32) {   // a NaN gives way to a number, as in fmaxf
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
  } else {
#pragma unroll
    for (int off = S / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
    return v;
  }
}
template <int S>
__device__ __forceinline__ uint32_t sub_max(uint32_t v) {
  if constexpr (S == 32) {
    return __reduce_max_sync(kFull, v);
  } else {
#pragma unroll
    for (int off = S / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(kFull, v, off));
    return v;
  }
}
// Whether p holds in any of the token's lanes.
template <int S>
__device__ __forceinline__ bool sub_any(bool p) {
  const uint32_t all = __ballot_sync(kFull, p);
  if constexpr (S == 32) return all != 0u;
  return ((all >> ((threadIdx.x & 31) / S * S)) & ((1u << (S & 31)) - 1u)) != 0u;
}

// exp(x), x <= 0, for a gradient of type T: binary32's own for binary32. What is
// rounded to bf16 takes the quick one, off by (4 + 1.5 |x|) 2^-24 relative (see
// quick_exp): 2^-17 for the smallest normal result, half a step of bf16 is 2^-8.
// For binary32 that would be up to 134 half-units, where expf has 4 (8192 x 256
// 3.8 us, 32768 x 1024 42 us: 6.4 TB/s).
template <typename T>
__device__ __forceinline__ float grad_exp(float x) {
  return sizeof(T) == 2 ? __expf(x) : expf(x);
}

constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float quick_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// exp for the choice: off by (4 + 1.5 |x|) 2^-24 relative at most (ex2.approx:
// 2^-22; its argument is rounded twice, 2^-24 |x| / ln 2 each with a factor ln 2)
__device__ __forceinline__ float quick_exp(float x) { return quick_exp2(x * kLog2E); }
// 1 / x, x >= 1 (0 for infinity): off by 2^-23 relative at most
__device__ __forceinline__ float quick_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Terms a_j of the chosen scores (lane j holds logit l of slot j, `live` if it
// takes part), equal to s_j up to a common factor, so that a_j / sum a is the
// renormalised score. The factor keeps the largest term near 1, where the
// scores themselves would underflow: exp(l - max) for softmax; for sigmoid,
// with m = min(0, max l), exp(-m) s = exp(l - m) / (1 + exp(l)).
template <bool kSigmoid, int S>
__device__ __forceinline__ float renorm_term(float l, bool live) {
  const float top = sub_max<S>(live ? l : -INFINITY);
  if (!live) return 0.f;
  if (!kSigmoid) return expf(l - top);
  return (l > 0.f ? 1.f : expf(l - fminf(top, 0.f))) / (1.f + expf(-fabsf(l)));
}

// 64-bit key that orders like the number
__device__ __forceinline__ uint64_t order_key(double f) {
  const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// The two best choice values in binary64 of those of this lane's `mine` experts
// that are in `mask` (bias or scores, never logits); row and bias from its first on.
template <typename T, bool kSigmoid, int S>
__device__ __noinline__ double2 best_exactly(const T* row, const float* bias, int mine, uint32_t mask, float top) {
  double z = 1.0;
  if (!kSigmoid) {
    z = 0.0;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) z += exp((double)load_logit(row + i) - (double)top);
    z = sub_sum<S>(z);
  }
  double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 1
  for (; mask; mask &= mask - 1) {
    const int i = __ffs(mask) - 1;
    const double l = load_logit(row + i);
    const double s = kSigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / z;
    const double v = bias ? s + (double)__ldg(bias + i) : s;
    b2 = fmax(b2, fmin(b1, v));
    b1 = fmax(b1, v);
  }
  __syncwarp();
  return make_double2(b1, b2);
}

// The choice in binary64, lane j < k returning slot j's expert. n: experts of a
// group. c: E doubles of shared memory of this warp.
template <typename T, bool kSigmoid>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, int E, int k, int n, moe_gate_desc g,
                                           float top, double* c) {
  const int lane = threadIdx.x & 31;
  const bool ranks = g.groups > 1 && g.group_best == 2;   // groups are ranked by scores
  double z = 1.0;
  if (!kSigmoid && (bias || ranks)) {
    z = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) z += exp((double)load_logit(row + e) - (double)top);
    z = sub_sum<32>(z);
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const double l = load_logit(row + e);
    const double s = !bias && !ranks ? l : kSigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / z;
    c[e] = bias ? s + (double)bias[e] : s;
  }
  __syncwarp();
  uint32_t open = kFull;
  if (g.groups > 1) {
    double b1 = -INFINITY, b2 = -INFINITY;
    int share = 1;   // lanes of a group: lane h, h + 32 / share, ... look at group h
    while (2 * share * g.groups <= 32) share *= 2;
    const int h = lane & (32 / share - 1);
    if (h < g.groups) {
#pragma unroll 4
      for (int i = lane / (32 / share); i < n; i += share) {
        const double v = c[h * n + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
    }
    for (int off = 16; off >= 32 / share; off >>= 1) {
      const double o1 = __shfl_xor_sync(kFull, b1, off), o2 = __shfl_xor_sync(kFull, b2, off);
      b2 = fmax(fmax(b2, o2), fmin(b1, o1));
      b1 = fmax(b1, o1);
    }
    const double r = g.group_best == 2 ? b1 + b2 : b1;
    int above = 0;
    for (int h = 0; h < g.groups; ++h) {
      const double o = __shfl_sync(kFull, r, h);
      above += o > r || (o == r && h < lane);
    }
    open = __ballot_sync(kFull, lane < g.groups && above < g.topk_groups);
    __syncwarp();
  }
  // keys in place of the values, 0 in closed groups; each lane's own from here on
  for (int e = lane; e < E; e += 32) {
    const bool in = g.groups == 1 || ((open >> (e / n)) & 1u);
    const uint64_t key = in ? order_key(ranks && !bias ? (double)load_logit(row + e) : c[e]) : 0;
    c[e] = __longlong_as_double((long long)key);
  }
  uint64_t best;
  int who;
  auto look = [&]() {   // this lane's largest, the lowest index of equals
    best = 0;
    who = INT32_MAX;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
      const uint64_t q = (uint64_t)__double_as_longlong(c[e]);
      if (q > best) { best = q; who = e; }
    }
  };
  look();
  int sel = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(best >> 32));
    const bool in = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(kFull, in ? (uint32_t)best : 0u);
    const int e = (int)__reduce_min_sync(kFull, in && (uint32_t)best == lo ? (uint32_t)who : 0xFFFFFFFFu);
    if (lane == j) sel = e;
    if (who == e) {
      c[e] = __longlong_as_double(0);
      look();
    }
  }
  __syncwarp();
  return sel;
}

// Odd-even merge sort of key[kLo .. kLo + kN), largest first.
template <int kLo, int kN, int kStep, int NV>
__device__ __forceinline__ void merge_descending(uint32_t (&key)[NV]) {
  if constexpr (2 * kStep < kN) {
    merge_descending<kLo, kN, 2 * kStep>(key);
    merge_descending<kLo + kStep, kN, 2 * kStep>(key);
  }
#pragma unroll
  for (int i = 2 * kStep < kN ? kLo + kStep : kLo; i + kStep < kLo + kN; i += 2 * kStep) {
    const uint32_t a = key[i], b = key[i + kStep];
    key[i] = max(a, b);
    key[i + kStep] = min(a, b);
  }
}
template <int kLo, int kN, int NV>
__device__ __forceinline__ void sort_descending(uint32_t (&key)[NV]) {
  if constexpr (kN > 1) {
    sort_descending<kLo, kN / 2>(key);
    sort_descending<kLo + kN / 2, kN / 2>(key);
    merge_descending<kLo, kN, 1>(key);
  }
}

// What the kernel needs of a grouping.
struct Groups {
  int n;      // experts of a group
  int span;   // lanes of a group, a power of two, or 0: groups are not sets of lanes
  int scratch;   // doubles of shared memory a warp
};

// s of one logit for the choice, within err0 (below) of its value.
template <bool kSigmoid>
__device__ __forceinline__ float quick_score(float l, float top, float inv_z) {
  return kSigmoid ? quick_rcp(1.f + quick_exp(-l)) : quick_exp(l - top) * inv_z;
}

// NV slots of a lane, the first `per` of them used; S lanes a token. kClose: there
// are groups ranked by scores, and those too close to tell are ranked in binary64
// before all else is done over. It costs registers (32768 x 160 with groups 24.3
// us, 21.8 without) and spares choose_exactly (8192 x 256 with one such token 9.0
// us, 12.1 without), so that it is for a warp a token, where few tokens do not
// hide one that takes long.
template <typename T, bool kSigmoid, int NV, int S, bool kClose>
__global__ void __launch_bounds__(kWarps * 32, kClose && NV <= 8 ? 12 : 1)
gate_kernel(const T* __restrict__ logits, const float* __restrict__ bias, int tokens, int E, int per, int k,
            int shared, int renorm, moe_gate_desc g, Groups gr, int32_t* __restrict__ topk_idx,
            float* __restrict__ topk_w, Header* hdr) {
  constexpr int kBits = NV * S <= 64 ? 6 : NV * S <= 128 ? 7 : NV * S <= 256 ? 8 : NV * S <= 512 ? 9 : 10;
  constexpr uint32_t kIdx = (1u << kBits) - 1u;
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31;
  const int li = lane % S, base = lane - li;   // place among the token's lanes, and their first
  double* scratch = smem + (threadIdx.x >> 5) * gr.scratch;
  const int warp_t = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / S);
  if (warp_t >= tokens) return;
  const int t = min(warp_t + lane / S, tokens - 1);   // lanes past the last token do it once more
  const bool mine_to_store = warp_t + lane / S < tokens;
  const T* row = logits + (int64_t)t * E;
  const int e0 = li * per;
  const int mine = max(0, min(per, E - e0));   // experts of this lane

  uint32_t ranked = 0;   // kClose: open groups, once they had to be ranked in binary64 (never none)
again:
  float l[NV], c[NV];   // logits, choice values
  // wide loads where every lane's part starts on a boundary and none is cut
  const bool wide = E == S * NV;
  if (wide) {
#pragma unroll
    for (int v = 0; v < NV; v += 4) {
      float q[4];
      load4(row + e0 + v, q);
#pragma unroll
      for (int b = 0; b < 4; ++b) l[v + b] = q[b];
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) l[v] = v < mine ? load_logit(row + e0 + v) : 0.f;
  }
  if (bias) {   // c holds the bias until the scores are there
    if (wide) {
#pragma unroll
      for (int v = 0; v < NV; v += 4) {
        float q[4];
        load4(bias + e0 + v, q);
#pragma unroll
        for (int b = 0; b < 4; ++b) c[v + b] = q[b];
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) c[v] = v < mine ? __ldg(bias + e0 + v) : 0.f;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) c[v] = 0.f;
  }
  uint64_t zeros = 0;   // two zeros, which stay that unless a value is not finite
  auto check = [&](const float (&x)[NV]) {
#pragma unroll
    for (int v = 0; v < NV; v += 2) zeros = ptx::fma2(ptx::two(x[v], x[v + 1]), 0ull, zeros);
  };
  check(l);
  if (bias) check(c);
  float zero, zero1;
  ptx::split(zeros, zero, zero1);
  const bool dead = sub_any<S>(zero + zero1 != 0.f);
  if (dead) {   // goes along as a row of zeros
#pragma unroll
    for (int v = 0; v < NV; ++v) l[v] = c[v] = 0.f;
    if (li == 0 && mine_to_store) latch_error(hdr, MOE_ERR_NONFINITE, (uint32_t)t);
  }
  if (!wide) {   // slots without an expert stay below all others
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v >= mine) l[v] = c[v] = -INFINITY;
  }
  const bool lossless = sizeof(T) == 2 && !bias;   // the keys tell all choice values apart
  const bool scores = bias || (g.groups > 1 && g.group_best == 2);
  float top = 0.f, z = 1.f, inv_z = 1.f;
  if (!kSigmoid && (scores || !renorm)) {
    top = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v) top = fmaxf(top, l[v]);
    top = sub_max<S>(top);
    float part = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) part += quick_exp(l[v] - top);
    z = sub_sum<S>(part);
    inv_z = 1.f / z;
  }
  // err0 + err1 |c|: how far c can be from its binary64 value, with exp off by
  // (4 + 1.5 |x|) 2^-24 relative (ex2 and the rounding of its argument) and the
  // reciprocal by 2^-23.
  // Sigmoid: s (1 - s) times the former is below 1.6 * 2^-24, the sum adds
  // 2^-24, the reciprocal 2^-23: 4.6 * 2^-24. Softmax: over z the errors of exp
  // average to at most 10.5 * 2^-23 (of 1024 terms), and the sum has a depth of
  // at most 37: below 2^-17 of the largest score 1 / z in all. The sum with the
  // bias: 2^-24 |c|. Weights that are not renormalised are divided by this z too:
  // at most those 10.5 * 2^-23 beside the roundings of the sum.
  const float err0 = scores ? (kSigmoid ? 5.f * 0x1p-24f : 0x1p-17f * inv_z) : 0.f;
  const float err1 = bias ? 0x1p-23f : 0.f;
  auto logits_choose = [&]() {   // -0 and +0 are one value
#pragma unroll
    for (int v = 0; v < NV; v += 2) ptx::split(ptx::add2(ptx::two(l[v], l[v + 1]), 0ull), c[v], c[v + 1]);
  };
  if (scores) {
#pragma unroll
    for (int v = 0; v < NV; v += 2) {   // quick_score, two at a time
      const uint64_t x = ptx::two(l[v], l[v + 1]), b = ptx::two(c[v], c[v + 1]);
      float p, q;
      if (kSigmoid) {
        ptx::split(ptx::mul2(x, ptx::two(-kLog2E, -kLog2E)), p, q);
        ptx::split(ptx::add2(ptx::two(quick_exp2(p), quick_exp2(q)), ptx::two(1.f, 1.f)), p, q);
        ptx::split(ptx::add2(ptx::two(quick_rcp(p), quick_rcp(q)), b), c[v], c[v + 1]);
      } else {
        ptx::split(ptx::mul2(ptx::add2(x, ptx::two(-top, -top)), ptx::two(kLog2E, kLog2E)), p, q);
        ptx::split(ptx::fma2(ptx::two(quick_exp2(p), quick_exp2(q)), ptx::two(inv_z, inv_z), b), c[v], c[v + 1]);
      }
    }
  } else {
    logits_choose();
  }

  // groups: the slots of closed ones go below all others
  bool unsure = false;
  if (g.groups > 1) {
    float b1 = -INFINITY, b2 = -INFINITY;
    auto take = [&](float v) {
      b2 = fmaxf(b2, fminf(b1, v));
      b1 = fmaxf(b1, v);
    };
    int gi = li;   // this lane's group
    if (gr.span) {   // a group is an aligned set of lanes, all of them full
      gi = li >> (__ffs(gr.span) - 1);
#pragma unroll
      for (int v = 0; v < NV; ++v) take(c[v]);
      for (int off = 1; off < gr.span; off <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, b1, off), o2 = __shfl_xor_sync(kFull, b2, off);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
    } else {         // any other grouping: lane i looks at group i
      float* row_c = reinterpret_cast<float*>(scratch) + lane / S * E;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine) row_c[e0 + v] = c[v];
      __syncwarp();
      if (li < g.groups)
        for (int i = 0; i < gr.n; ++i) take(row_c[li * gr.n + i]);
      __syncwarp();
    }
    const bool two = g.group_best == 2;
    const float r = two ? b1 + b2 : b1;
    const float e = two ? 2.f * err0 + err1 * (fabsf(b1) + fabsf(b2)) + 0x1p-23f * fabsf(r)
                        : (scores ? err0 + err1 * fabsf(b1) : 0.f);
    const float lo = r - e, hi = r + e;
    // a group is open if fewer than topk_groups others may be above it; its lanes
    // share the comparisons
    const int step = gr.span ? gr.span : 1;
    int above = 0, may = 0;
    for (int h0 = 0; h0 < g.groups; h0 += step) {
      const int h = h0 + (li & (step - 1)), src = base + h * step;
      if (scores) {
        const float olo = __shfl_sync(kFull, lo, src), ohi = __shfl_sync(kFull, hi, src);
        above += h < g.groups && olo > hi;       // not of itself
        may += h < g.groups && !(ohi < lo);      // of itself too
      } else {   // exact: ties to the lowest group
        const float o = __shfl_sync(kFull, r, src);
        above += h < g.groups && (o > r || (o == r && h < gi));
      }
    }
    for (int off = 1; off < step; off <<= 1) {
      above += __shfl_xor_sync(kFull, above, off);
      may += __shfl_xor_sync(kFull, may, off);
    }
    may = scores ? may - 1 : above;
    const bool in = gi < g.groups;
    unsure = in && may >= g.topk_groups && above < g.topk_groups;
    if (kClose && ranked) {
      may = (ranked >> (gi & 31)) & 1u ? 0 : g.topk_groups;
      unsure = false;
    } else if (kClose && gr.span && __any_sync(kFull, unsure && !dead)) {
      // Too close to tell: from the values that can be a group's best two in
      // binary64, then once more from the start, so that no registers wait
      uint32_t mask = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine && !(c[v] < b2 - 4.f * (err0 + err1 * (fabsf(b2) + fabsf(c[v]))))) mask |= 1u << v;
      double2 b = best_exactly<T, kSigmoid, S>(row + e0, bias ? bias + e0 : nullptr, mine, mask, top);
      for (int off = 1; off < step; off <<= 1) {
        const double o1 = __shfl_xor_sync(kFull, b.x, off), o2 = __shfl_xor_sync(kFull, b.y, off);
        b.y = fmax(fmax(b.y, o2), fmin(b.x, o1));
        b.x = fmax(b.x, o1);
      }
      const double rd = two ? b.x + b.y : b.x;
      int over = 0;   // groups above, ties to the lowest
#pragma unroll 1
      for (int h = 0; h < g.groups; ++h) {
        const double o = __shfl_sync(kFull, rd, base + h * step);
        over += o > rd || (o == rd && h < gi);
      }
      const bool open = in && over < g.topk_groups;
      ranked = 0;
#pragma unroll 1
      for (int h = 0; h < g.groups; ++h)
        ranked |= (__shfl_sync(kFull, (int)open, base + h * step) ? 1u : 0u) << h;
      if (dead || !ranked) ranked = kFull;
      goto again;
    }
    const uint32_t opens = __ballot_sync(kFull, in && may < g.topk_groups) >> base;
    if (!bias && scores) logits_choose();   // the scores only ranked the groups
    if (gr.span) {
      const bool open = may < g.topk_groups;
#pragma unroll
      for (int v = 0; v < NV; ++v) c[v] = open ? c[v] : -INFINITY;
    } else {
      int q = e0 / gr.n, at = e0 - q * gr.n;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (v < mine && !((opens >> q) & 1u)) c[v] = -INFINITY;
        if (++at == gr.n) { at = 0; ++q; }
      }
    }
  }

  uint32_t key[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) key[v] = (order_key(c[v]) & ~kIdx) | (kIdx - (uint32_t)(e0 + v));
  sort_descending<0, NV>(key);
  // the two largest stay in registers, the others wait in shared memory, two
  // kNoKey behind them (a lane's list is popped NV times at most)
  uint32_t* list = reinterpret_cast<uint32_t*>(scratch) + lane * (NV + 4);
#pragma unroll
  for (int v = 0; v < NV; v += 4)
    *reinterpret_cast<uint4*>(list + v) = make_uint4(key[v], key[v + 1], key[v + 2], key[v + 3]);
  *reinterpret_cast<uint2*>(list + NV) = make_uint2(kNoKey, kNoKey);
  uint32_t head = key[0], second = key[1];
  list += 2;
  uint32_t won = kNoKey;   // lane j: slot j's key (lane k: that of the best one left)
  auto pop = [&](uint32_t m, int j) {   // the largest head m, into lane j
    won = li == j ? m : won;
    if (head == m) {
      head = second;
      second = *list++;
    }
  };
  const int rounds = lossless ? k : min(k + 1, S);
#pragma unroll 1
  for (int j = 0; j < rounds; ++j) pop(sub_max<S>(head), j);
  int sel = won < kLeastKey ? -1 : (int)(kIdx - (won & kIdx));
  float lj = sel >= 0 ? load_logit(row + sel) : 0.f;
  unsure = sub_any<S>(unsure) && !dead;   // which groups are open
  if (!lossless) {
    float v = -INFINITY;
    if (sel >= 0) v = bias ? __ldg(bias + sel) + quick_score<kSigmoid>(lj, top, inv_z) : lj;
    const float next = __shfl_down_sync(kFull, v, 1);
    const int nsel = __shfl_down_sync(kFull, sel, 1);
    const float mag = fmaxf(fmaxf(fabsf(v), sel >= 0 && nsel >= 0 ? fabsf(next) : 0.f), 0x1p-126f);
    const float near = 2.f * (err0 + err1 * mag);       // between two choice values
    const float cut = mag * (float)(1u << kBits) * 0x1p-23f;   // and what the keys drop
    bool doubt = false;   // between lanes j and j + 1
    if (li + 1 < k) doubt = bias ? !(v - next > near) : !(v > next || (v == next && sel < nsel));
    if (li == k - 1) doubt = k == S || (nsel >= 0 && !(v - next > near + cut));
    doubt = sub_any<S>(doubt) && !dead && !unsure;
    if (__any_sync(kFull, doubt)) {
      // pop whatever may reach the last slot
      const uint32_t lim = order_key(__shfl_sync(kFull, v - (near + cut), base + k - 1) + 0.f);
      int n = rounds, most = rounds;   // popped of this token, and of any here
      uint32_t m = sub_max<S>(head);
      auto reaches = [&]() { return doubt && m >= kLeastKey && (m | kIdx) >= lim; };
      while (__any_sync(kFull, reaches() && n < S)) {
        const bool take = reaches() && n < S;
        pop(take ? m : ~0u, take ? n : -1);   // ~0 is no key: nothing is taken
        n += take;
        ++most;
        m = sub_max<S>(head);
      }
      unsure = unsure || reaches();   // more candidates than lanes
      const int cand = won < kLeastKey ? -1 : (int)(kIdx - (won & kIdx));
      double zd = 1.0;
      if (!kSigmoid && bias) {
        double part = 0.0;
#pragma unroll 1
        for (int i = 0; i < mine; ++i) part += exp((double)load_logit(row + e0 + i) - (double)top);
        zd = sub_sum<S>(part);
      }
      double c64 = -INFINITY;
      if (cand >= 0) {
        const double x = load_logit(row + cand);
        c64 = !bias ? x
                    : (kSigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / zd) + (double)__ldg(bias + cand);
      }
      int rank = 0;
      for (int i = 0; i < most; ++i) {
        const double o = __shfl_sync(kFull, c64, base + i);
        const int os = __shfl_sync(kFull, cand, base + i);
        rank += os >= 0 && (o > c64 || (o == c64 && os < cand));
      }
      int* slots = reinterpret_cast<int*>(scratch) + base;
      __syncwarp();
      if (doubt && cand >= 0 && rank < k) slots[rank] = cand;
      __syncwarp();
      if (doubt && !unsure && li < k) {
        sel = slots[li];
        lj = load_logit(row + sel);
      }
    }
  }
  uint32_t again = __ballot_sync(kFull, unsure);
  while (again) {   // a token at a time, by the whole warp
    const int src = __ffs(again) - 1, first = src - src % S;
    again &= ~((S == 32 ? kFull : (1u << (S & 31)) - 1u) << first);
    __syncwarp();
    const int s = choose_exactly<T, kSigmoid>(logits + (int64_t)__shfl_sync(kFull, t, first) * E, bias, E, k, gr.n,
                                              g, __shfl_sync(kFull, top, first), scratch);
    const int got = __shfl_sync(kFull, s, li);
    if (base == first && li < k) {
      sel = got;
      lj = load_logit(row + sel);
    }
    __syncwarp();
  }

  const bool live = li < k;
  float a;
  if (renorm) {
    a = renorm_term<kSigmoid, S>(lj, live);
    a /= k <= 8 ? sub_sum<8>(a) : sub_sum<S>(a);   // of the slots' lanes
  } else {
    a = kSigmoid ? 1.f / (1.f + expf(-lj)) : expf(lj - top) / z;
  }
  const int ks = k + shared;
  int32_t* idx = topk_idx + (int64_t)t * ks;
  float* out = topk_w + (int64_t)t * ks;
  if (mine_to_store && live) {
    idx[li] = dead ? li : sel;
    out[li] = dead ? __int_as_float(0x7fc00000) : g.scale * a;
  }
  if (mine_to_store && shared && li == 0) {
    idx[k] = E;
    out[k] = 1.f;
  }
}

// S lanes a token (topk <= S). Elements go kW at a time, 16 bytes where rows
// start on such a boundary, else one. In the former case a plain softmax keeps its
// row in NV > 0 registers a lane (E <= S NV): one exponential an element, not two.
template <typename T, bool kSigmoid, bool kRenorm, int S, int kW, int NV>
__global__ void __launch_bounds__(kWarps * 32)
gate_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                     const float* __restrict__ grad_w, int tokens, int E, int k, int shared, float scale,
                     T* __restrict__ grad_logits) {
  constexpr bool kEvery = !kSigmoid && !kRenorm;
  static_assert(!kEvery || (NV > 0) == (kW > 1), "a plain softmax's row is in registers where it is loaded wide");
  const int lane = threadIdx.x & 31, li = lane % S, base = lane - li;
  const int warp_t = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / S);
  if (warp_t >= tokens) return;
  const int t = min(warp_t + lane / S, tokens - 1);
  const bool real = warp_t + lane / S < tokens;   // lanes past the last token store nothing
  const T* row = logits + (int64_t)t * E;
  T* grow = grad_logits + (int64_t)t * E;
  const int ks = k + shared;
  int e = -1;
  float gw = 0.f, l = 0.f;
  if (li < k) {
    e = topk_idx[(int64_t)t * ks + li];
    gw = scale * grad_w[(int64_t)t * ks + li];
  }
  const bool live = e >= 0 && e < E;
  if (live) l = load_logit(row + e);
  else gw = 0.f;
  float top = 0.f, inv = 0.f, dot = 0.f;
  float p[NV > 0 ? NV : 1];
  if constexpr (kEvery && NV > 0) {
#pragma unroll
    for (int c = 0; c < NV; c += kW) {
      float v[kW];
      const int i = li * kW + c * S;
      if (i < E) load_vec<kW>(row + i, v);
#pragma unroll
      for (int b = 0; b < kW; ++b) p[c + b] = i < E ? v[b] : -INFINITY;
    }
    top = -INFINITY;
#pragma unroll
    for (int c = 0; c < NV; ++c) top = fmaxf(top, p[c]);
    top = sub_max<S>(top);
    float z = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      p[c] = grad_exp<T>(p[c] - top);   // 0 of slots without an expert
      z += p[c];
    }
    inv = 1.f / sub_sum<S>(z);
    dot = sub_sum<S>(live ? gw * (expf(l - top) * inv) : 0.f);
  } else if constexpr (kEvery) {
    // running maximum and sum in one pass, an element a load (E is of no wide one).
    // expf's elements wait for one rescaling together (1002 f32, one token / 32768:
    // 11 / 95 us, each by itself 17 / 103); quick ones do not gain (bf16 67, 64 us)
    constexpr int kEach = sizeof(T) == 4 ? 16 : 1;
    float m = -INFINITY, z = 0.f;
    for (int i = li; i < E; i += kEach * S) {
      float v[kEach];
#pragma unroll
      for (int b = 0; b < kEach; ++b) v[b] = i + b * S < E ? load_logit(row + i + b * S) : -INFINITY;
      float vm = v[0];
#pragma unroll
      for (int b = 1; b < kEach; ++b) vm = fmaxf(vm, v[b]);
      if (vm > m) {
        z *= grad_exp<T>(m - vm);
        m = vm;
      }
#pragma unroll
      for (int b = 0; b < kEach; ++b) z += v[b] == -INFINITY ? 0.f : grad_exp<T>(v[b] - m);
    }
    top = sub_max<S>(m);
    z = sub_sum<S>(z == 0.f ? 0.f : z * grad_exp<T>(m - top));
    inv = 1.f / z;
    dot = sub_sum<S>(live ? gw * (expf(l - top) * inv) : 0.f);
  }
  // what every expert gets
  if constexpr (kEvery && NV > 0) {
#pragma unroll
    for (int c = 0; c < NV; c += kW) {
      float v[kW];
#pragma unroll
      for (int b = 0; b < kW; ++b) v[b] = p[c + b] * inv * -dot;
      if (real && li * kW + c * S < E) store_vec<kW>(grow + li * kW + c * S, v);
    }
  } else if constexpr (kEvery) {
    if (real)
      for (int i = li; i < E; i += S) store_grad(grow + i, grad_exp<T>(load_logit(row + i) - top) * inv * -dot);
  } else if (real) {
    const float none[kW] = {};
    for (int i = li * kW; i < E; i += S * kW) store_vec<kW>(grow + i, none);
  }
  // and what the chosen ones get: d from slot li
  float d;
  if constexpr (kEvery) {
    d = gw;
  } else {
    float q = kRenorm ? renorm_term<kSigmoid, S>(l, live) : 1.f / (1.f + expf(-l));
    float gd = gw;
    if (kRenorm) {
      const float s = sub_sum<S>(q);
      q = s == 0.f ? 0.f : q / s;   // 0: no slot takes part
      gd -= sub_sum<S>(q * gw);
    }
    d = q * gd;
    if (kSigmoid) d *= 1.f / (1.f + expf(l));
  }
  // an expert named twice: every slot of it writes their sum, in slot order
  bool twice = false;
#pragma unroll 7
  for (int off = 1; off < S; ++off) {
    const int o = __shfl_xor_sync(kFull, live ? e : -1, off);
    twice |= live && o == e;
  }
  if (__any_sync(kFull, twice)) {
    float sum = 0.f;
    for (int j = 0; j < k; ++j) {
      const float dj = __shfl_sync(kFull, d, base + j);
      const int ej = __shfl_sync(kFull, live ? e : -1, base + j);
      if (ej == e) sum += dj;
    }
    d = sum;
  }
  if constexpr (kEvery) d = expf(l - top) * inv * (d - dot);
  __syncwarp();   // after the stores above
  if (real && live) store_grad(grow + e, d);
}

}  // namespace

cudaError_t launch_gate(const Ctx& c, const moe_gate_desc& g, const void* logits, const float* bias, int32_t* idx,
                        float* w) {
  const int T = (int)c.s.T, E = (int)c.routed_E, k = (int)c.routed_k;
  auto go = [&](auto kernel, auto* l, int S, int NV) {
    const int per = (E + S - 1) / S, tokens = kWarps * 32 / S;   // tokens of a block
    // a warp's scratch in doubles: a row, the tokens' rows in floats, the lanes' lists
    Groups gr{E / g.groups, 0, std::max(std::max(E, (32 / S * E + 1) / 2), 16 * (NV + 4)) + 1 & ~1};
    if (gr.n % per == 0 && ((gr.n / per) & (gr.n / per - 1)) == 0) gr.span = gr.n / per;
    kernel<<<(T + tokens - 1) / tokens, kWarps * 32, (size_t)kWarps * gr.scratch * sizeof(double), c.stream>>>(
        l, bias, T, E, per, k, c.shared, c.s.renorm, g, gr, idx, w, c.ws.hdr);
    return cudaGetLastError();
  };
  auto by_size = [&](auto* l, auto sig, auto close) {
    using L = std::remove_const_t<std::remove_pointer_t<decltype(l)>>;
    constexpr bool kSig = decltype(sig)::value, kClose = decltype(close)::value;
    // a lane for every slot and, where the keys are not exact, the best one left
    const int lanes = std::max(k + (sizeof(L) == 2 && !bias ? 0 : 1), (int)g.groups);
    // Fewer lanes a token once the SMs are full of warps anyway; later where the
    // choice needs scores, as a token in doubt keeps the others of its warp waiting,
    // longest for a softmax's sum. Measured, a warp / 8 lanes: 128 bf16, 4096 tokens
    // 3.2 / 3.1 us, 2048 2.6 / 2.9; 64 f32, 4096 3.9 / 2.9, 2048 3.2 / 3.3. With scores,
    // sigmoid: 64 f32, 4096 4.3 / 4.0; 128 f32, 8192 6.2 / 5.9, 4096 4.4 / 4.8; softmax:
    // 64 f32, 6000 5.4 / 5.1, 4096 4.3 / 5.0; 96 f32, 10240 7.9 / 8.0, 6000 5.8 / 7.0.
    // 16 lanes: 128 f32, 8192 5.5 / 5.0, 4096 4.2 / 4.4; sigmoid with a bias 8192 6.3 /
    // 5.7, and groups 12288 9.7 / 8.6, 8192 7.5 / 9.0.
    // Beyond 128 experts it is a matter of little: 16384 x 256 bf16 9.0 / 8.7, 12288
    // 7.3 / 7.3; 16384 x 160 bf16 with groups 12.3 / 11.5, 12288 9.7 / 9.4; with scores
    // 160 f32 and groups 16384 14.3 / 13.1, 12288 13.0 / 14.2; 256 never (32768, f32 and
    // groups 25.4 / 28.0)
    const bool scores = bias || (g.groups > 1 && g.group_best == 2);
    const int from8 = !scores ? 4096 : E <= 64 ? (kSig ? 4096 : 6000) : (kSig ? 8192 : 10240);
    if (lanes <= 8 && E <= 128 && T >= from8)
      return E <= 64 ? go(gate_kernel<L, kSig, 8, 8, false>, l, 8, 8) : go(gate_kernel<L, kSig, 16, 8, false>, l, 8, 16);
    if (lanes <= 16 && E <= 128 && T >= (scores && (!kSig || g.groups > 1) ? 10240 : 8192))
      return go(gate_kernel<L, kSig, 8, 16, false>, l, 16, 8);
    if (lanes <= 16 && E <= (scores ? 192 : 256) && T >= (scores ? 16384 : 12288))
      return go(gate_kernel<L, kSig, 16, 16, false>, l, 16, 16);
    if (E <= 128) return go(gate_kernel<L, kSig, 4, 32, kClose>, l, 32, 4);
    if (E <= 256) return go(gate_kernel<L, kSig, 8, 32, kClose>, l, 32, 8);
    if (E <= 512) return go(gate_kernel<L, kSig, 16, 32, kClose>, l, 32, 16);
    return go(gate_kernel<L, kSig, 32, 32, kClose>, l, 32, 32);
  };
  auto by_score = [&](auto* l) {
    std::true_type yes;
    std::false_type no;
    const bool close = g.groups > 1 && (bias || g.group_best == 2);
    if (g.score == MOE_SCORE_SIGMOID) return close ? by_size(l, yes, yes) : by_size(l, yes, no);
    return close ? by_size(l, no, yes) : by_size(l, no, no);
  };
  return g.logits_dtype == MOE_BF16 ? by_score((const __nv_bfloat16*)logits) : by_score((const float*)logits);
}

cudaError_t launch_gate_backward(const moe_shape& s, const moe_gate_desc& g, const void* logits, const int32_t* idx,
                                 const float* grad_w, void* grad_logits, cudaStream_t stream) {
  const int T = (int)s.T, E = (int)s.E, k = (int)s.topk, shared = (s.flags & MOE_FLAG_SHARED_EXPERT) ? 1 : 0;
  auto go = [&](auto kernel, auto* l, auto* d, int S) {
    const int tokens = kWarps * 32 / S;
    kernel<<<(T + tokens - 1) / tokens, kWarps * 32, 0, stream>>>(l, idx, grad_w, T, E, k, shared, g.scale, d);
    return cudaGetLastError();
  };
  auto by_size = [&](auto* l, auto* d, auto sig, auto ren) {
    using L = std::remove_pointer_t<decltype(d)>;
    constexpr bool kSig = decltype(sig)::value, kRen = decltype(ren)::value;
    constexpr int kV = 16 / sizeof(L);
    // the fewest lanes that hold the slots: 8 against 32 lanes 8192 x 256 f32
    // 3.5 / 6.3 us, one token 2.1 / 3.0. A plain softmax keeps its row in registers
    // (32768 x 128 bf16 4.9 us, 32768 x 1024 29; reading it twice 7.9 and 44)
    if constexpr (!kSig && !kRen) {
      if (E % kV == 0 && k <= 8 && E <= 128) return go(gate_backward_kernel<L, kSig, kRen, 8, kV, 16>, l, d, 8);
      if (E % kV == 0 && k <= 8 && E <= 256) return go(gate_backward_kernel<L, kSig, kRen, 8, kV, 32>, l, d, 8);
      if (E % kV == 0 && E <= 512) return go(gate_backward_kernel<L, kSig, kRen, 32, kV, 16>, l, d, 32);
      if (E % kV == 0) return go(gate_backward_kernel<L, kSig, kRen, 32, kV, 32>, l, d, 32);
    } else {
      if (E % kV == 0 && k <= 8) return go(gate_backward_kernel<L, kSig, kRen, 8, kV, 0>, l, d, 8);
      if (E % kV == 0) return go(gate_backward_kernel<L, kSig, kRen, 32, kV, 0>, l, d, 32);
    }
    return k <= 8 ? go(gate_backward_kernel<L, kSig, kRen, 8, 1, 0>, l, d, 8)
                  : go(gate_backward_kernel<L, kSig, kRen, 32, 1, 0>, l, d, 32);
  };
  auto by_form = [&](auto* l, auto* d) {
    std::true_type yes;
    std::false_type no;
    if (g.score == MOE_SCORE_SIGMOID) return s.renorm ? by_size(l, d, yes, yes) : by_size(l, d, yes, no);
    return s.renorm ? by_size(l, d, no, yes) : by_size(l, d, no, no);
  };
  return g.logits_dtype == MOE_BF16 ? by_form((const __nv_bfloat16*)logits, (__nv_bfloat16*)grad_logits)
                                    : by_form((const float*)logits, (float*)grad_logits);
}

}  // namespace moe
