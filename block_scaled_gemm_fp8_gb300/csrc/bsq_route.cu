// bsq_route.cu -- the router of a mixture layer: the k experts of each token's highest scores and
// their weights, and the gradient of the logits.
//
//   score = logit, or logit + bias (softmax), sigmoid(logit) + bias (sigmoid gate);
//   softmax   w_j = f p_j, p the softmax over all logits, or renormalized over the chosen ones
//   sigmoid   w_j = f s_j, s = sigmoid(logit), or renormalized f s_j / sum_chosen s
//   softmax   dl_e = p_e (g_e - sum_chosen g p),           g = f grad_w at the chosen, else 0
//             (renormalized: the same over the chosen, all other gradients zero)
//   sigmoid   dl_j = g_j s_j (1 - s_j), renormalized (g_j - sum g s / sum s) s_j (1 - s_j) / sum s
//
// A warp per token: lane l holds experts l, l + 32, ... in registers.  Scores are compared as
// integers of the same order, so that one warp-wide integer maximum finds the best and a
// minimum over indices breaks ties; a chosen expert's key becomes zero, the key of an expert
// that cannot be chosen (a NaN or minus infinity).  All sums are float32.
#include <cuda_bf16.h>

#include "bsq_moe_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

constexpr int kWarpsR = 4;    // tokens a CTA
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// An unsigned integer of the same order as the score; 0 for a NaN and minus infinity.
__device__ __forceinline__ uint32_t order_of(float s) {
  const uint32_t u = __float_as_uint(s + 0.f);   // -0 becomes 0: they are equal
  const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return s > -INFINITY ? key : 0u;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// V: experts a lane.
template <typename T, int V>
__global__ void __launch_bounds__(kWarpsR * 32) route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int k,
                                                            int gate, bool renorm, const float* __restrict__ bias,
                                                            float factor, int32_t* __restrict__ ids,
                                                            float* __restrict__ weights) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsR + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  const T* row = logits + t * E;
  float l[V];
  uint32_t key[V];
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 32 * v + lane;
    l[v] = e < E ? load(row + e) : -INFINITY;
    nan |= l[v] != l[v];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 32 * v + lane;
    float s = l[v];
    if (bias && e < E) s = (gate == BSQ_GATE_SIGMOID ? sigmoid(s) : s) + __ldg(bias + e);
    key[v] = order_of(s);
  }
  nan = __any_sync(kFull, nan);
  int id = -1;             // lane j: slot j's expert and its logit
  float chosen = -INFINITY;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0, e = kFull;
    float at = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) best = key[v], e = 32 * v + lane, at = l[v];
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;   // the rest cannot be chosen
    const uint32_t winner = __reduce_min_sync(kFull, best == top ? e : kFull);
    const float logit = __shfl_sync(kFull, at, winner & 31);
    if (lane == j) id = static_cast<int>(winner), chosen = logit;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (winner == 32u * v + lane) key[v] = 0;
  }
  const bool have = id >= 0;
  float w;
  if (gate == BSQ_GATE_SOFTMAX) {
    float m = chosen, sum = 0.f;
    if (!renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);
    }
    m = warp_max(m);
    const float ex = have ? expf(chosen - m) : 0.f;
    if (renorm) {
      sum = ex;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) sum += 32 * v + lane < E ? expf(l[v] - m) : 0.f;
    }
    w = ex / warp_sum(sum);
  } else {
    w = have ? sigmoid(chosen) : 0.f;
    if (renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : sum;   // every sigmoid zero (or a NaN): nothing to divide by
    }
  }
  if (lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = !have ? 0.f : nan ? NAN : factor * w;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kWarpsR * 32) route_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E,
                                                                     int k, int gate, bool renorm, float factor,
                                                                     const int32_t* __restrict__ ids,
                                                                     const float* __restrict__ grad_weights,
                                                                     T* __restrict__ grad_logits) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsR + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  const T* row = logits + t * E;
  const int id = lane < k ? __ldg(ids + t * k + lane) : -1;
  const bool have = static_cast<unsigned>(id) < static_cast<unsigned>(E);
  const float g = have ? factor * __ldg(grad_weights + t * k + lane) : 0.f;
  const float chosen = have ? load(row + id) : -INFINITY;
  const bool any = __any_sync(kFull, have);
  const bool full = gate == BSQ_GATE_SOFTMAX && !renorm && any;   // every expert's gradient, not the chosen ones' alone
  float p[V], mean = 0.f, d = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = 0.f;
  if (gate == BSQ_GATE_SOFTMAX) {
    float m = chosen, sum = 0.f;
    if (full) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = 32 * v + lane < E ? load(row + 32 * v + lane) : -INFINITY;
        m = fmaxf(m, p[v]);
      }
    }
    m = warp_max(m);
    const float ex = have ? expf(chosen - m) : 0.f;
    if (full) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = 32 * v + lane < E ? expf(p[v] - m) : 0.f;
        sum += p[v];
      }
    } else {
      sum = ex;
    }
    sum = warp_sum(sum);
    const float q = have ? ex / sum : 0.f;
    mean = warp_sum(g * q);
    d = full ? g * q : q * (g - mean);
    if (full) {
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] = -(p[v] / sum) * mean;
    }
  } else {
    const float s = have ? sigmoid(chosen) : 0.f;
    d = g * s * (1.f - s);
    if (renorm) {
      const float sum = warp_sum(s), mass = warp_sum(g * s);
      d = sum != 0.f ? (g - mass / sum) / sum * s * (1.f - s) : 0.f;
    }
  }
  if (!have) d = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl_sync(kFull, id, j);
    const float add = __shfl_sync(kFull, d, j);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == 32 * v + lane) p[v] += add;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (32 * v + lane < E) store(grad_logits + t * E + 32 * v + lane, p[v]);
}

template <typename T, int V>
void launch_v(const RouteArgs& a, unsigned grid) {
  const T* logits = static_cast<const T*>(a.logits);
  if (a.grad_logits)
    route_backward_kernel<T, V><<<grid, kWarpsR * 32, 0, a.stream>>>(logits, a.T, a.E, a.k, a.gate, a.renormalize, a.factor,
                                                                     a.ids, a.grad_weights, static_cast<T*>(a.grad_logits));
  else
    route_kernel<T, V><<<grid, kWarpsR * 32, 0, a.stream>>>(logits, a.T, a.E, a.k, a.gate, a.renormalize, a.bias, a.factor,
                                                            a.ids, a.weights);
}

template <typename T>
int launch_typed(const RouteArgs& a, const char** msg) {
  const int64_t grid = (a.T + kWarpsR - 1) / kWarpsR;   // T < 2^31
  const unsigned g = static_cast<unsigned>(grid);
  if (a.E <= 32) launch_v<T, 1>(a, g);
  else if (a.E <= 64) launch_v<T, 2>(a, g);
  else if (a.E <= 128) launch_v<T, 4>(a, g);
  else if (a.E <= 256) launch_v<T, 8>(a, g);
  else if (a.E <= 512) launch_v<T, 16>(a, g);
  else launch_v<T, 32>(a, g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

int launch_any(const RouteArgs& a, const char** msg) {
  return a.dtype == BSQ_DT_BF16 ? launch_typed<__nv_bfloat16>(a, msg) : launch_typed<float>(a, msg);
}

}  // namespace

int launch_route(const RouteArgs& a, const char** msg) { return launch_any(a, msg); }
int launch_route_backward(const RouteArgs& a, const char** msg) { return launch_any(a, msg); }

}  // namespace bsq
