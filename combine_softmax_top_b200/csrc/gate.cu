// The gate: routing with softmax or sigmoid scores, a balance bias, expert
// groups, top-k and renormalised, scaled weights; and its gradient.
//
// Both kernels give one warp a token and keep what belongs to its row in
// shared memory. The choice is made in binary64 throughout.
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kFull = 0xffffffffu;

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

template <typename T, bool kSigmoid>
__global__ void __launch_bounds__(kWarps * 32)
gate_kernel(const T* __restrict__ logits, const float* __restrict__ bias, int tokens, int E, int k, int shared,
            int renorm, moe_gate_desc g, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, Header* hdr) {
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 31;
  double* c = smem + (threadIdx.x >> 5) * E;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T* row = logits + (int64_t)t * E;
  const int ks = k + shared;
  int32_t* idx = topk_idx + (int64_t)t * ks;
  float* out = topk_w + (int64_t)t * ks;
  if (shared && lane == k) {
    idx[k] = E;
    out[k] = 1.f;
  }
  bool bad = false;
  float top = -INFINITY;
  for (int e = lane; e < E; e += 32) {
    const float l = load_logit(row + e);
    bad |= !isfinite(l) || (bias && !isfinite(bias[e]));
    top = fmaxf(top, l);
  }
  if (__any_sync(kFull, bad)) {
    if (lane < k) {
      idx[lane] = lane;
      out[lane] = __int_as_float(0x7fc00000);
    }
    if (lane == 0) latch_error(hdr, MOE_ERR_NONFINITE, (uint32_t)t);
    return;
  }
  top = warp_max(top);
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
      double v = ((open >> lane) & 1u) ? -INFINITY : rank;
      int i = lane < g.groups && !((open >> lane) & 1u) ? lane : 64;
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
  const bool live = lane < k;
  const float l = live ? load_logit(row + sel) : 0.f;
  float a;
  if (renorm) {
    a = renorm_term<kSigmoid>(l, live);
    a /= warp_sum(a);
  } else {
    a = kSigmoid ? 1.f / (1.f + expf(-l)) : expf(l - top) / (float)z;
  }
  if (live) {
    idx[lane] = sel;
    out[lane] = g.scale * a;
  }
}

template <typename T, bool kSigmoid>
__global__ void __launch_bounds__(kWarps * 32)
gate_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                     const float* __restrict__ grad_w, int tokens, int E, int k, int shared, int renorm, float scale,
                     T* __restrict__ grad_logits) {
  extern __shared__ float gsum[];
  const int lane = threadIdx.x & 31;
  float* acc = gsum + (threadIdx.x >> 5) * E;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T* row = logits + (int64_t)t * E;
  const int ks = k + shared;
  int e = -1;
  float gw = 0.f, l = 0.f;
  if (lane < k) {
    e = topk_idx[(int64_t)t * ks + lane];
    if (e >= 0 && e < E) {
      gw = scale * grad_w[(int64_t)t * ks + lane];
      l = load_logit(row + e);
    } else {
      e = -1;
    }
  }
  const bool live = e >= 0;
  float top = 0.f, z = 1.f, d;   // d: what slot `lane` adds to its expert
  const bool every = !kSigmoid && !renorm;
  if (every) {
    top = -INFINITY;
    for (int i = lane; i < E; i += 32) top = fmaxf(top, load_logit(row + i));
    top = warp_max(top);
    z = 0.f;
    for (int i = lane; i < E; i += 32) z += expf(load_logit(row + i) - top);
    z = warp_sum(z);
    d = gw;
  } else {
    float q = renorm ? renorm_term<kSigmoid>(l, live) : 1.f / (1.f + expf(-l));
    float gd = gw;
    if (renorm) {
      const float s = warp_sum(q);
      q = s > 0.f || s != s ? q / s : 0.f;   // no slot takes part: 0
      gd -= warp_sum(q * gw);
    }
    d = q * gd;
    if (kSigmoid) d *= 1.f / (1.f + expf(l));
  }
  for (int i = lane; i < E; i += 32) acc[i] = 0.f;
  __syncwarp();
  for (int j = 0; j < k; ++j) {   // slot order: an expert named twice sums in a fixed order
    if (lane == j && live) acc[e] += d;
    __syncwarp();
  }
  if (every) {
    const float dot = warp_sum(live ? gw * (expf(l - top) / z) : 0.f);
    for (int i = lane; i < E; i += 32)
      store_grad(grad_logits + (int64_t)t * E + i, expf(load_logit(row + i) - top) / z * (acc[i] - dot));
  } else {
    for (int i = lane; i < E; i += 32) store_grad(grad_logits + (int64_t)t * E + i, acc[i]);
  }
}

}  // namespace

cudaError_t launch_gate(const Ctx& c, const moe_gate_desc& g, const void* logits, const float* bias, int32_t* idx,
                        float* w) {
  const int T = (int)c.s.T, E = (int)c.routed_E, k = (int)c.routed_k;
  const dim3 grid((T + kWarps - 1) / kWarps);
  const size_t smem = (size_t)kWarps * E * sizeof(double);   // <= 32 KB
  auto go = [&](auto kernel, auto* l) {
    kernel<<<grid, kWarps * 32, smem, c.stream>>>(l, bias, T, E, k, c.shared, c.s.renorm, g, idx, w, c.ws.hdr);
    return cudaGetLastError();
  };
  const bool sig = g.score == MOE_SCORE_SIGMOID;
  if (g.logits_dtype == MOE_BF16) {
    const __nv_bfloat16* l = (const __nv_bfloat16*)logits;
    return sig ? go(gate_kernel<__nv_bfloat16, true>, l) : go(gate_kernel<__nv_bfloat16, false>, l);
  }
  const float* l = (const float*)logits;
  return sig ? go(gate_kernel<float, true>, l) : go(gate_kernel<float, false>, l);
}

cudaError_t launch_gate_backward(const moe_shape& s, const moe_gate_desc& g, const void* logits, const int32_t* idx,
                                 const float* grad_w, void* grad_logits, cudaStream_t stream) {
  const int T = (int)s.T, E = (int)s.E, k = (int)s.topk, shared = (s.flags & MOE_FLAG_SHARED_EXPERT) ? 1 : 0;
  const dim3 grid((T + kWarps - 1) / kWarps);
  const size_t smem = (size_t)kWarps * E * sizeof(float);
  auto go = [&](auto kernel, auto* l, auto* d) {
    kernel<<<grid, kWarps * 32, smem, stream>>>(l, idx, grad_w, T, E, k, shared, s.renorm, g.scale, d);
    return cudaGetLastError();
  };
  const bool sig = g.score == MOE_SCORE_SIGMOID;
  if (g.logits_dtype == MOE_BF16) {
    const __nv_bfloat16* l = (const __nv_bfloat16*)logits;
    __nv_bfloat16* d = (__nv_bfloat16*)grad_logits;
    return sig ? go(gate_backward_kernel<__nv_bfloat16, true>, l, d)
               : go(gate_backward_kernel<__nv_bfloat16, false>, l, d);
  }
  const float* l = (const float*)logits;
  float* d = (float*)grad_logits;
  return sig ? go(gate_backward_kernel<float, true>, l, d) : go(gate_backward_kernel<float, false>, l, d);
}

}  // namespace moe
