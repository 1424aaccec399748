// The gate: routing with softmax or sigmoid scores, a balance bias, expert
// groups, top-k and renormalised, scaled weights; and its gradient.
//
// gate_kernel gives one warp a token. Lane i holds `per` = ceil(E / 32)
// consecutive experts from i * per on, so that lower lanes hold lower experts
// and, for most groupings, a group is a whole power-of-two set of lanes. Each lane
// sorts 32-bit keys that order like its choice values c, the low bits given
// to the place in the lane (a sorting network of min and max, two
// instructions a comparison), and each of the topk rounds takes the largest
// head with one warp reduction and pops it.
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

// NV slots of a lane, the first `per` of them used; kBits of the key hold the slot.
template <typename T, bool kSigmoid, int NV>
__global__ void __launch_bounds__(kWarps * 32)
gate_kernel(const T* __restrict__ logits, const float* __restrict__ bias, int tokens, int E, int per, int k,
            int shared, int renorm, moe_gate_desc g, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
            Header* hdr) {
  constexpr int kBits = NV <= 4 ? 2 : NV <= 8 ? 3 : NV <= 16 ? 4 : 5;
  constexpr uint32_t kSlot = (1u << kBits) - 1u;
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31;
  double* scratch = smem + (threadIdx.x >> 5) * E;
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
  if (per == NV && E == 32 * NV) {
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
  bool bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    bad |= !isfinite(l[v]);
    if (v < mine) top = fmaxf(top, l[v]);
  }
  const bool lossless = sizeof(T) == 2 && !bias;   // the keys tell all choice values apart
  const bool scores = bias || (g.groups > 1 && g.group_best == 2);
  float z = 1.f;
  if (!kSigmoid) {
    top = warp_max(top);
    if (scores || !renorm) {
      float part = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) part += v < mine ? expf(l[v] - top) : 0.f;
      z = warp_sum(part);
    }
  }
  // err0 + err1 |c|: bound of the difference between c (of one or of the sum of
  // a few) and its binary64 value. Sigmoid: exp 2^-22, the sum and the
  // quotient 2^-24 each, all at most 3 * 2^-24 of s <= 1, and the bias's sum
  // 2^-24 |c|. Softmax: exp's argument and value, and a sum of E terms in a
  // tree of depth <= 37: below 2^-18 of the largest score 1 / z.
  const float err0 = bias || scores ? (kSigmoid ? 0x1p-21f : 0x1p-18f / z) : 0.f;
  const float err1 = bias ? 0x1p-22f : 0.f;
  bool unsure = false;
  if (scores) {
#pragma unroll
    for (int v = 0; v < NV; ++v) c[v] = kSigmoid ? 1.f / (1.f + expf(-l[v])) : expf(l[v] - top) / z;
    if (bias) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine) {
          const float b = __ldg(bias + e0 + v);
          bad |= !isfinite(b);
          c[v] += b;
        }
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) c[v] = l[v];
  }
  if (__any_sync(kFull, bad)) {
    if (lane < ks) {
      idx[lane] = lane < k ? lane : E;
      out[lane] = lane < k ? __int_as_float(0x7fc00000) : 1.f;
    }
    if (lane == 0) latch_error(hdr, MOE_ERR_NONFINITE, (uint32_t)t);
    return;
  }

  // groups: `closed` has bit v where slot v's group is not open
  uint32_t closed = 0;
  if (g.groups > 1) {
    const int n = E / g.groups;
    float b1 = -INFINITY, b2 = -INFINITY;
    auto take = [&](float v) {
      b2 = fmaxf(b2, fminf(b1, v));
      b1 = fmaxf(b1, v);
    };
    const int span = n / per;   // lanes of a group
    const bool lanes = span * per == n && (span & (span - 1)) == 0;
    if (lanes) {   // a group is an aligned set of lanes (and all of them are full)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine) take(c[v]);
      for (int off = 1; off < span; off <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, b1, off), o2 = __shfl_xor_sync(kFull, b2, off);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
    } else {       // any other grouping: lane i looks at group i
      float* row_c = reinterpret_cast<float*>(scratch);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v < mine) row_c[e0 + v] = c[v];
      __syncwarp();
      if (lane < g.groups)
        for (int i = 0; i < n; ++i) take(row_c[lane * n + i]);
      __syncwarp();
    }
    const bool two = g.group_best == 2;
    const float r = two ? b1 + b2 : b1;
    const float e = two ? 2.f * err0 + err1 * (fabsf(b1) + fabsf(b2)) + 0x1p-23f * fabsf(r)
                        : err0 + err1 * fabsf(b1);
    const float lo = r - e, hi = r + e;
    // lane i: whether its group (lanes: the one it belongs to) is open: fewer
    // than topk_groups others may be above it
    const int gi = lanes ? lane / span : lane;
    int above = 0, may = 0;
    for (int h = 0; h < g.groups; ++h) {
      const int src = lanes ? h * span : h;
      const float olo = __shfl_sync(kFull, lo, src), ohi = __shfl_sync(kFull, hi, src);
      if (e == 0.f) {   // exact: ties to the lowest group
        above += olo > r || (olo == r && h < gi);
        may = above;
      } else if (h != gi) {
        above += olo > hi;
        may += !(ohi < lo);
      }
    }
    const bool open = may < g.topk_groups;
    unsure = gi < g.groups && !open && above < g.topk_groups;
    const uint32_t opens = __ballot_sync(kFull, gi < g.groups && open);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int src = lanes ? lane : (e0 + v < E ? (e0 + v) / n : 0);
      if (!((opens >> src) & 1u)) closed |= 1u << v;
    }
    if (!bias && scores) {
#pragma unroll
      for (int v = 0; v < NV; ++v) c[v] = l[v];   // the groups' scores only ranked the groups
    }
  }

  uint32_t key[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v)
    key[v] = v < mine && !((closed >> v) & 1u) ? (order_key(c[v]) & ~kSlot) | (kSlot - v) : kNoKey;
  // odd-even merge sort, descending
#pragma unroll
  for (int p = 1; p < NV; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < NV; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (j + i + q < NV && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
            const uint32_t a = key[j + i], b = key[j + i + q];
            key[j + i] = max(a, b);
            key[j + i + q] = min(a, b);
          }
  int sel = -1;   // lane j: slot j's expert (lane k: the best one left, or -1)
  auto pop = [&](int j) -> uint32_t {   // the largest head, into lane j
    const uint32_t head = key[0] & ~kSlot;
    const uint32_t m = __reduce_max_sync(kFull, head);
    const int who = __ffs(__ballot_sync(kFull, head == m)) - 1;   // lowest lane: lowest expert
    const int e = __shfl_sync(kFull, e0 + (int)(kSlot - (key[0] & kSlot)), who);
    if (lane == j && m != kNoKey) sel = e;
    if (lane == who) {
#pragma unroll
      for (int v = 0; v + 1 < NV; ++v) key[v] = key[v + 1];
      key[NV - 1] = kNoKey;
    }
    return m;
  };
  const int rounds = lossless ? k : min(k + 1, 32);
  for (int j = 0; j < rounds; ++j) pop(j);
  unsure = __any_sync(kFull, unsure);   // which groups are open
  if (!lossless && !unsure) {
    float v = sel >= 0 ? load_logit(row + sel) : -INFINITY;
    if (bias && sel >= 0) v = (kSigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / z) + __ldg(bias + sel);
    const float next = __shfl_down_sync(kFull, v, 1);
    const int nsel = __shfl_down_sync(kFull, sel, 1);
    const float mag = fmaxf(fmaxf(fabsf(v), sel >= 0 && nsel >= 0 ? fabsf(next) : 0.f), 0x1p-126f);
    const float cut = ldexpf(mag, kBits - 23);   // what the keys drop
    const float near = 2.f * (err0 + err1 * mag) + cut;
    bool doubt = false;   // between lanes j and j + 1
    if (lane + 1 < k) doubt = bias ? !(v - next > near) : !(v > next || (v == next && sel < nsel));
    if (lane == k - 1) doubt = k == 32 || (nsel >= 0 && !(v - next > near));
    if (__any_sync(kFull, doubt)) {
      // pop whatever may reach the last slot
      const uint32_t lim = order_key(__shfl_sync(kFull, v - near, k - 1));
      int n = rounds;
      uint32_t m = __reduce_max_sync(kFull, key[0]);
      while (n < 32 && m != kNoKey && (m | kSlot) >= lim) {
        pop(n++);
        m = __reduce_max_sync(kFull, key[0]);
      }
      unsure = m != kNoKey && (m | kSlot) >= lim;   // more than a warp of them
      if (!unsure) {
        double zd = 1.0;
        if (!kSigmoid && bias) {
          double part = 0.0;
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (i < mine) part += exp((double)l[i] - (double)top);
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
    top = warp_max(top);
    __syncwarp();
    sel = choose_exactly<T, kSigmoid>(row, bias, E, k, g, top, scratch);
  }

  const bool live = lane < k;
  const float lj = live ? load_logit(row + sel) : 0.f;
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
  const size_t smem = (size_t)kWarps * E * sizeof(double);   // <= 32 KB
  auto go = [&](auto kernel, auto* l) {
    kernel<<<grid, kWarps * 32, smem, c.stream>>>(l, bias, T, E, per, k, c.shared, c.s.renorm, g, idx, w, c.ws.hdr);
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
