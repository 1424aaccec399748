// The gate: routing with softmax or sigmoid scores, a balance bias, expert
// groups, top-k and renormalised, scaled weights; and its gradient.
//
// gate_kernel gives one warp a token. Lane i holds `per` = ceil(E / 32)
// consecutive experts from i * per on, so that for most groupings a group is a
// whole power-of-two set of lanes. Each lane sorts 32-bit keys that order like
// its choice values c, their low 7 to 10 bits given to the expert (a sorting
// network of min and max, two instructions a comparison), and each of the topk
// rounds takes the largest head with one warp reduction, which names the
// expert too, and pops it.
//
// What is chosen has to be what binary64 chooses. The keys drop low bits and
// c = s + bias carries binary32 roundings, so the chosen values (and the best
// one left) are compared once more with the bounds of both: a token with two
// neighbours closer than that, or with a group at the border of the open ones
// closer than that, is done over in binary64 (choose_exactly). Without a bias
// c is the logit itself; bf16 logits then lose nothing in the keys and need no
// second look.
//
// The row is read once, four elements at a time where its alignment allows.
// gate_backward_kernel also gives one warp a token, adds the chosen experts'
// derivatives into a row of shared memory in slot order and writes the row.
#include <algorithm>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kNoKey = 0u;   // below the key of every number

// 32-bit key that orders like the number
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);   // -0 and +0 are one value
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
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
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// The warp's best (value, index): larger value, lower index on a tie.
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const double ov = __shfl_xor_sync(kFull, v, off);
    const int oi = __shfl_xor_sync(kFull, i, off);
    if (ov > v || (ov == v && oi < i)) { v = ov; i = oi; }
  }
}

// Terms a_j of the chosen scores (lane j holds logit l of slot j, `live` if it
// takes part), equal to s_j up to a common factor, so that a_j / sum a is the
// renormalised score. The factor keeps the largest term near 1, where the
// scores themselves would underflow: exp(l - max) for softmax; for sigmoid,
// with m = min(0, max l), exp(-m) s = exp(l - m) / (1 + exp(l)).
template <bool kSigmoid>
__device__ __forceinline__ float renorm_term(float l, bool live) {
  const float top = warp_max(live ? l : -INFINITY);
  if (!live) return 0.f;
  if (!kSigmoid) return expf(l - top);
  const float m = fminf(top, 0.f);
  return l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
}

// The choice in binary64, lane j < k returning slot j's expert. c: E doubles
// of shared memory of this warp.
template <typename T, bool kSigmoid>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, int E, int k, moe_gate_desc g, float top,
                                           double* c) {
  const int lane = threadIdx.x & 31;
  double z = 1.0;
  if (!kSigmoid) {
    z = 0.0;
    for (int e = lane; e < E; e += 32) z += exp((double)load_logit(row + e) - (double)top);
    z = warp_sum(z);
  }
  auto score = [&](int e) -> double {
    const double l = load_logit(row + e);
    return kSigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / z;
  };
  for (int e = lane; e < E; e += 32) c[e] = bias ? score(e) + (double)bias[e] : (double)load_logit(row + e);
  __syncwarp();
  if (g.groups > 1) {
    const int n = E / g.groups;
    double rank = -INFINITY;
    if (lane < g.groups) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < n; ++i) {
        const int e = lane * n + i;
        const double v = (!bias && g.group_best == 2) ? score(e) : c[e];
        if (v > b1) { b2 = b1; b1 = v; }
        else if (v > b2) b2 = v;
      }
      rank = g.group_best == 2 ? b1 + b2 : b1;
    }
    uint32_t open = 0;
    for (int j = 0; j < g.topk_groups; ++j) {
      const bool free = lane < g.groups && !((open >> lane) & 1u);
      double v = free ? rank : -INFINITY;
      int i = free ? lane : 64;
      warp_best(v, i);
      open |= 1u << i;
    }
    __syncwarp();
    for (int e = lane; e < E; e += 32)
      if (!((open >> (e / n)) & 1u)) c[e] = -INFINITY;
    __syncwarp();
  }
  int sel = 0;
  for (int j = 0; j < k; ++j) {
    double v = -INFINITY;
    int i = INT32_MAX;
    for (int e = lane; e < E; e += 32)
      if (c[e] > v) { v = c[e]; i = e; }
    warp_best(v, i);
    if (lane == j) sel = i;
    if (lane == 0) c[i] = -INFINITY;
    __syncwarp();
  }
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
};

// s of one logit for the choice, within err0 (below) of its value.
template <bool kSigmoid>
__device__ __forceinline__ float quick_score(float l, float top, float inv_z) {
  return kSigmoid ? __fdividef(1.f, 1.f + __expf(-l)) : __expf(l - top) * inv_z;
}

// NV slots of a lane, the first `per` of them used.
template <typename T, bool kSigmoid, int NV>
__global__ void __launch_bounds__(kWarps * 32)
gate_kernel(const T* __restrict__ logits, const float* __restrict__ bias, int tokens, int E, int per, int k,
            int shared, int renorm, moe_gate_desc g, Groups gr, int32_t* __restrict__ topk_idx,
            float* __restrict__ topk_w, Header* hdr) {
  constexpr int kBits = NV <= 4 ? 7 : NV <= 8 ? 8 : NV <= 16 ? 9 : 10;   // 32 NV experts at most
  constexpr uint32_t kIdx = (1u << kBits) - 1u;
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31;
  double* scratch = smem + (threadIdx.x >> 5) * max(E, 16);
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T* row = logits + (int64_t)t * E;
  const int ks = k + shared;
  int32_t* idx = topk_idx + (int64_t)t * ks;
  float* out = topk_w + (int64_t)t * ks;
  const int e0 = lane * per;
  const int mine = max(0, min(per, E - e0));   // experts of this lane

  float l[NV], c[NV];   // logits, choice values
  // wide loads where every lane's part starts on a boundary and none is cut
  const bool wide = E == 32 * NV;
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
  float zero = 0.f;   // stays 0 unless a value is not finite
#pragma unroll
  for (int v = 0; v < NV; ++v) zero = __fmaf_rn(l[v], 0.f, __fmaf_rn(c[v], 0.f, zero));
  if (__any_sync(kFull, zero != 0.f)) {
    if (lane < ks) {
      idx[lane] = lane < k ? lane : E;
      out[lane] = lane < k ? __int_as_float(0x7fc00000) : 1.f;
    }
    if (lane == 0) latch_error(hdr, MOE_ERR_NONFINITE, (uint32_t)t);
    return;
  }
  const bool lossless = sizeof(T) == 2 && !bias;   // the keys tell all choice values apart
  const bool scores = bias || (g.groups > 1 && g.group_best == 2);
  float top = 0.f, z = 1.f, inv_z = 1.f;
  if (!kSigmoid) {
    top = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v < mine) top = fmaxf(top, l[v]);
    top = warp_max(top);
    if (scores || !renorm) {
      float part = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) part += v < mine ? __expf(l[v] - top) : 0.f;
      z = warp_sum(part);
      inv_z = 1.f / z;
    }
  }
  // err0 + err1 |c|: how far c can be from its binary64 value, with exp off by
  // (2 + 1.173 |x|) 2^-23 relative and the fast quotient by 2^-22.
  // Sigmoid: s (1 - s) times the former is below 2^-23, the sum adds 2^-24, the
  // quotient 2^-22. Softmax: x is itself off by |x| 2^-24; over z the errors of
  // exp average to at most 10.5 * 2^-23 (of 1024 terms), and the sum has a
  // depth of at most 37: below 2^-17 of the largest score 1 / z in all. The
  // sum with the bias: 2^-24 |c|.
  const float err0 = scores ? (kSigmoid ? 0x1p-21f : 0x1p-17f * inv_z) : 0.f;
  const float err1 = bias ? 0x1p-23f : 0.f;
  if (scores) {
#pragma unroll
    for (int v = 0; v < NV; ++v) c[v] += quick_score<kSigmoid>(l[v], top, inv_z);
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) c[v] = l[v];
  }

  // groups: which slots' groups are open, one bit each
  uint32_t open = ~0u;
  bool unsure = false;
  if (g.groups > 1) {
    float b1 = -INFINITY, b2 = -INFINITY;
    auto take = [&](float v) {
      b2 = fmaxf(b2, fminf(b1, v));
      b1 = fmaxf(b1, v);
    };
    int gi = lane;   // this lane's group
    if (gr.span) {   // a group is an aligned set of lanes, all of them full
      gi = lane >> (__ffs(gr.span) - 1);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine) take(c[v]);
      for (int off = 1; off < gr.span; off <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, b1, off), o2 = __shfl_xor_sync(kFull, b2, off);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
    } else {         // any other grouping: lane i looks at group i
      float* row_c = reinterpret_cast<float*>(scratch);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine) row_c[e0 + v] = c[v];
      __syncwarp();
      if (lane < g.groups)
        for (int i = 0; i < gr.n; ++i) take(row_c[lane * gr.n + i]);
      __syncwarp();
    }
    const bool two = g.group_best == 2;
    const float r = two ? b1 + b2 : b1;
    const float e = two ? 2.f * err0 + err1 * (fabsf(b1) + fabsf(b2)) + 0x1p-23f * fabsf(r)
                        : (scores ? err0 + err1 * fabsf(b1) : 0.f);
    const float lo = r - e, hi = r + e;
    // a group is open if fewer than topk_groups others may be above it
    const int step = gr.span ? gr.span : 1;
    int above = 0, may = 0;
    if (scores) {
      for (int h = 0; h < g.groups; ++h) {
        const float olo = __shfl_sync(kFull, lo, h * step), ohi = __shfl_sync(kFull, hi, h * step);
        above += olo > hi;       // not of itself
        may += !(ohi < lo);      // of itself too
      }
      --may;
    } else {   // exact: ties to the lowest group
      for (int h = 0; h < g.groups; ++h) {
        const float o = __shfl_sync(kFull, r, h * step);
        above += o > r || (o == r && h < gi);
      }
      may = above;
    }
    const bool in = gi < g.groups;
    unsure = in && may >= g.topk_groups && above < g.topk_groups;
    const uint32_t opens = __ballot_sync(kFull, in && may < g.topk_groups);
    if (gr.span) {
      open = may < g.topk_groups ? ~0u : 0u;
    } else {
      open = 0;
      int q = e0 / gr.n, at = e0 - q * gr.n;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (v < mine) open |= ((opens >> q) & 1u) << v;
        if (++at == gr.n) { at = 0; ++q; }
      }
    }
    if (!bias && scores) {
#pragma unroll
      for (int v = 0; v < NV; ++v) c[v] = l[v];   // the scores only ranked the groups
    }
  }

  uint32_t key[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v)
    key[v] = v < mine && ((open >> v) & 1u) ? (order_key(c[v]) & ~kIdx) | (kIdx - (uint32_t)(e0 + v)) : kNoKey;
  sort_descending<0, NV>(key);
  uint32_t won = kNoKey;   // lane j: slot j's key (lane k: that of the best one left)
  auto pop = [&](int j) {   // the largest head, into lane j
    const uint32_t m = __reduce_max_sync(kFull, key[0]);
    if (lane == j) won = m;
    if (key[0] == m) {
#pragma unroll
      for (int v = 0; v + 1 < NV; ++v) key[v] = key[v + 1];
      key[NV - 1] = kNoKey;
    }
  };
  const int rounds = lossless ? k : min(k + 1, 32);
#pragma unroll 1
  for (int j = 0; j < rounds; ++j) pop(j);
  int sel = won == kNoKey ? -1 : (int)(kIdx - (won & kIdx));
  float lj = sel >= 0 ? load_logit(row + sel) : 0.f;
  unsure = __any_sync(kFull, unsure);   // which groups are open
  if (!lossless && !unsure) {
    float v = -INFINITY;
    if (sel >= 0) v = bias ? __ldg(bias + sel) + quick_score<kSigmoid>(lj, top, inv_z) : lj;
    const float next = __shfl_down_sync(kFull, v, 1);
    const int nsel = __shfl_down_sync(kFull, sel, 1);
    const float mag = fmaxf(fmaxf(fabsf(v), sel >= 0 && nsel >= 0 ? fabsf(next) : 0.f), 0x1p-126f);
    const float near = 2.f * (err0 + err1 * mag);       // between two choice values
    const float cut = mag * (float)(1u << kBits) * 0x1p-23f;   // and what the keys drop
    bool doubt = false;   // between lanes j and j + 1
    if (lane + 1 < k) doubt = bias ? !(v - next > near) : !(v > next || (v == next && sel < nsel));
    if (lane == k - 1) doubt = k == 32 || (nsel >= 0 && !(v - next > near + cut));
    if (__any_sync(kFull, doubt)) {
      // pop whatever may reach the last slot
      const uint32_t lim = order_key(__shfl_sync(kFull, v - (near + cut), k - 1));
      int n = rounds;
      uint32_t m = __reduce_max_sync(kFull, key[0]);
      while (n < 32 && m != kNoKey && (m | kIdx) >= lim) {
        pop(n++);
        m = __reduce_max_sync(kFull, key[0]);
      }
      unsure = m != kNoKey && (m | kIdx) >= lim;   // more than a warp of them
      if (!unsure) {
        sel = won == kNoKey ? -1 : (int)(kIdx - (won & kIdx));
        double zd = 1.0;
        if (!kSigmoid && bias) {
          double part = 0.0;
#pragma unroll 1
          for (int i = 0; i < mine; ++i) part += exp((double)load_logit(row + e0 + i) - (double)top);
          zd = warp_sum(part);
        }
        double c64 = -INFINITY;
        if (sel >= 0) {
          const double x = load_logit(row + sel);
          c64 = !bias ? x
                      : (kSigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / zd) + (double)__ldg(bias + sel);
        }
        int rank = 0;
        for (int i = 0; i < n; ++i) {
          const double o = __shfl_sync(kFull, c64, i);
          const int os = __shfl_sync(kFull, sel, i);
          rank += o > c64 || (o == c64 && os < sel);
        }
        int* slots = reinterpret_cast<int*>(scratch);
        __syncwarp();
        if (sel >= 0 && rank < k) slots[rank] = sel;
        __syncwarp();
        if (lane < k) sel = slots[lane];
      }
    }
  }
  if (unsure) {
    __syncwarp();
    sel = choose_exactly<T, kSigmoid>(row, bias, E, k, g, top, scratch);
  }

  const bool live = lane < k;
  if (!lossless || unsure) lj = live ? load_logit(row + sel) : 0.f;
  float a;
  if (renorm) {
    a = renorm_term<kSigmoid>(lj, live);
    a /= warp_sum(a);
  } else {
    a = kSigmoid ? 1.f / (1.f + expf(-lj)) : expf(lj - top) / z;
  }
  if (lane < ks) {
    idx[lane] = live ? sel : E;
    out[lane] = live ? g.scale * a : 1.f;
  }
}

// Lane i holds elements (32 c + i) kW .. + kW - 1 of the row, c < NV / kW:
// kW = 4 where rows start on a boundary of four elements, else 1. The row is
// read only for a softmax that is not renormalised, where every logit has a
// gradient, and then once.
template <typename T, bool kSigmoid, bool kRenorm, int NV, int kW>
__global__ void __launch_bounds__(kWarps * 32)
gate_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                     const float* __restrict__ grad_w, int tokens, int E, int k, int shared, float scale,
                     T* __restrict__ grad_logits) {
  constexpr bool kEvery = !kSigmoid && !kRenorm;
  __shared__ float gsum[kWarps][32 * NV];
  const int lane = threadIdx.x & 31;
  float* acc = gsum[threadIdx.x >> 5];
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T* row = logits + (int64_t)t * E;
  T* grow = grad_logits + (int64_t)t * E;
  const int ks = k + shared;
  int e = -1;
  float gw = 0.f, l = 0.f;
  if (lane < k) {
    e = topk_idx[(int64_t)t * ks + lane];
    gw = scale * grad_w[(int64_t)t * ks + lane];
  }
  const bool live = e >= 0 && e < E;
  float p[kEvery ? NV : 1];
  if constexpr (kEvery) {
#pragma unroll
    for (int v = 0; v < NV; v += kW) {
      const int i = (32 * (v / kW) + lane) * kW;
      if constexpr (kW == 1) {
        p[v] = i < E ? load_logit(row + i) : -INFINITY;
      } else {
        float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i < E) load4(row + i, q);
#pragma unroll
        for (int b = 0; b < 4; ++b) p[v + b] = q[b];
      }
    }
  }
  if (live) l = load_logit(row + e);
  else gw = 0.f;
#pragma unroll
  for (int i = 0; i < NV; i += 4)
    *reinterpret_cast<float4*>(acc + 32 * i + 4 * lane) = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, z = 0.f, d;   // d: what slot `lane` adds to its expert
  if constexpr (kEvery) {
#pragma unroll
    for (int v = 0; v < NV; ++v) top = fmaxf(top, p[v]);
    top = warp_max(top);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      p[v] = p[v] == -INFINITY ? 0.f : expf(p[v] - top);
      z += p[v];
    }
    z = warp_sum(z);
    d = gw;
  } else {
    float q = kRenorm ? renorm_term<kSigmoid>(l, live) : 1.f / (1.f + expf(-l));
    float gd = gw;
    if (kRenorm) {
      const float s = warp_sum(q);
      q = s == 0.f ? 0.f : q / s;   // 0: no slot takes part
      gd -= warp_sum(q * gw);
    }
    d = q * gd;
    if (kSigmoid) d *= 1.f / (1.f + expf(l));
  }
  __syncwarp();
  // an expert named twice sums in slot order; nearly always none is
  const uint32_t same = __match_any_sync(kFull, live ? e : ~lane);
  if (!__any_sync(kFull, (same & (same - 1u)) != 0u)) {
    if (live) acc[e] = d;
  } else {
    for (int j = 0; j < k; ++j) {
      if (lane == j && live) acc[e] += d;
      __syncwarp();
    }
  }
  __syncwarp();
  const float inv = kEvery ? 1.f / z : 0.f;
  const float dot = kEvery ? warp_sum(live ? gw * (expf(l - top) * inv) : 0.f) : 0.f;
#pragma unroll
  for (int v = 0; v < NV; v += kW) {
    const int i = (32 * (v / kW) + lane) * kW;
    if (i >= E) break;
    if constexpr (kW == 1) {
      float r = acc[i];
      if constexpr (kEvery) r = p[v] * inv * (r - dot);
      store_grad(grow + i, r);
    } else {
      const float4 a = *reinterpret_cast<const float4*>(acc + i);
      float r[4] = {a.x, a.y, a.z, a.w};
      if constexpr (kEvery) {
#pragma unroll
        for (int b = 0; b < 4; ++b) r[b] = p[v + b] * inv * (r[b] - dot);
      }
      store4(grow + i, r);
    }
  }
}

}  // namespace

cudaError_t launch_gate(const Ctx& c, const moe_gate_desc& g, const void* logits, const float* bias, int32_t* idx,
                        float* w) {
  const int T = (int)c.s.T, E = (int)c.routed_E, k = (int)c.routed_k, per = (E + 31) / 32;
  const dim3 grid((T + kWarps - 1) / kWarps);
  const size_t smem = (size_t)kWarps * std::max(E, 16) * sizeof(double);   // a warp: a row, or 32 slots; <= 32 KB
  Groups gr{E / g.groups, 0};
  if (gr.n % per == 0 && ((gr.n / per) & (gr.n / per - 1)) == 0) gr.span = gr.n / per;
  auto go = [&](auto kernel, auto* l) {
    kernel<<<grid, kWarps * 32, smem, c.stream>>>(l, bias, T, E, per, k, c.shared, c.s.renorm, g, gr, idx, w, c.ws.hdr);
    return cudaGetLastError();
  };
  auto by_size = [&](auto* l, auto sig) {
    using L = std::remove_const_t<std::remove_pointer_t<decltype(l)>>;
    constexpr bool kSig = decltype(sig)::value;
    if (per <= 4) return go(gate_kernel<L, kSig, 4>, l);
    if (per <= 8) return go(gate_kernel<L, kSig, 8>, l);
    if (per <= 16) return go(gate_kernel<L, kSig, 16>, l);
    return go(gate_kernel<L, kSig, 32>, l);
  };
  auto by_score = [&](auto* l) {
    return g.score == MOE_SCORE_SIGMOID ? by_size(l, std::true_type()) : by_size(l, std::false_type());
  };
  return g.logits_dtype == MOE_BF16 ? by_score((const __nv_bfloat16*)logits) : by_score((const float*)logits);
}

cudaError_t launch_gate_backward(const moe_shape& s, const moe_gate_desc& g, const void* logits, const int32_t* idx,
                                 const float* grad_w, void* grad_logits, cudaStream_t stream) {
  const int T = (int)s.T, E = (int)s.E, k = (int)s.topk, shared = (s.flags & MOE_FLAG_SHARED_EXPERT) ? 1 : 0;
  const dim3 grid((T + kWarps - 1) / kWarps);
  auto go = [&](auto kernel, auto* l, auto* d) {
    kernel<<<grid, kWarps * 32, 0, stream>>>(l, idx, grad_w, T, E, k, shared, g.scale, d);
    return cudaGetLastError();
  };
  auto by_size = [&](auto* l, auto* d, auto sig, auto ren) {
    using L = std::remove_pointer_t<decltype(d)>;
    constexpr bool kSig = decltype(sig)::value, kRen = decltype(ren)::value;
    if (E % 4) return go(gate_backward_kernel<L, kSig, kRen, 32, 1>, l, d);
    if (E <= 128) return go(gate_backward_kernel<L, kSig, kRen, 4, 4>, l, d);
    if (E <= 256) return go(gate_backward_kernel<L, kSig, kRen, 8, 4>, l, d);
    if (E <= 512) return go(gate_backward_kernel<L, kSig, kRen, 16, 4>, l, d);
    return go(gate_backward_kernel<L, kSig, kRen, 32, 4>, l, d);
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
