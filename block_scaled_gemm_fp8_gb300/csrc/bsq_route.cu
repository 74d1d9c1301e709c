// bsq_route.cu -- the router of a mixture layer: the k experts of each token's highest scores and
// their weights, and the gradient of the logits.
//
//   score = logit, or logit + bias (softmax), sigmoid(logit) + bias (sigmoid gate);
//   softmax   w_j = f p_j, p the softmax over all logits, or renormalized over the chosen ones
//   sigmoid   w_j = f s_j, s = sigmoid(logit), or renormalized f s_j / sum_chosen s
//   softmax   dl_e = p_e (g_e - sum_chosen g p),           g = f grad_w at the chosen, else 0
//             (renormalized: the same over the chosen, all other gradients zero)
//   sigmoid   dl_j = g_j s_j (1 - s_j), renormalized q_j (g_j - sum g q) (1 - s_j), q = s / sum s
//
// A warp per token, V = E / 32 experts a lane in registers.  Scores are compared as
// integers of the same order, so that one warp-wide integer maximum finds the best and the
// first lane that has it the lowest index; a chosen expert's key leaves, and the key of an expert
// that cannot be chosen (a NaN or minus infinity) is zero.  All sums are float32.  Bound by the
// instructions of the rounds, 0.75 of the issue slots (HBM's part is 1.4 us, of the gradient 2.6):
//   float32 logits, eight experts a token, us           16384 x 128   gradient   16384 x 256   gradient
//   softmax over all, without and with a bias             7.9   8.3        6.9    12.5  14.6        9.0
//   softmax over the chosen                               7.3   7.6        5.7    11.1  13.3        6.7
//   sigmoid, not renormalized                             6.9   9.0        5.0    11.1  16.1        6.1
//   sigmoid, renormalized                                 7.7   9.9        6.2    11.8  17.0        7.0
// 16 tokens on 64 experts, four each: 2.0 us.
#include <cuda_bf16.h>

#include "bsq_lanes.cuh"
#include "bsq_moe_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

constexpr int kWarpsR = 4;    // tokens a CTA
constexpr int log2_of(int v) { return v < 2 ? 0 : 1 + log2_of(v / 2); }

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
// {s, 1 - s} of the sigmoid, by e^-|x|, which does not overflow: each keeps its bits as far as float32 has numbers
// (|x| = 103).  One reciprocal for both (16384 x 128, the gradient of eight: 5.3 us with a
// division each, 5.0 so).
__device__ __forceinline__ float2 sigmoids(float x) {
  const float e = expf(-fabsf(x)), r = 1.f / (1.f + e), er = e * r;
  return x >= 0.f ? make_float2(r, er) : make_float2(er, r);
}
__device__ __forceinline__ float sigmoid(float x) { return sigmoids(x).x; }
// e^x for the softmax's x <= 0, as 2^(x log2 e).  The product's rounding and the constant's (0.23 2^-24 of it) add up to
// 1.23 |x| 2^-24 to the relative error: beside the rounding of x = l - m, |x| 2^-24, or alone where that
// difference is exact.  It is below 2^-19 for what counts, |x| <= 25 (with expf 16384 x 128 take 8.1 us, so 7.7).
__device__ __forceinline__ float exp_of(float x) { return exp2f(x * 1.4426950408889634f); }

// A lane's experts by falling score, equal ones by rising index: neighbours are exchanged in turn, and
// only for a higher score; V rounds put V in order.
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V], uint32_t (&e)[V]) {
#pragma unroll
  for (int n = 0; n < V; ++n) {
#pragma unroll
    for (int i = n & 1; i + 1 < V; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const uint32_t k0 = swap ? key[i + 1] : key[i], e0 = swap ? e[i + 1] : e[i];
      key[i + 1] = swap ? key[i] : key[i + 1];
      e[i + 1] = swap ? e[i] : e[i + 1];
      key[i] = k0;
      e[i] = e0;
    }
  }
}

// A lane's V logits; minus infinity past the last.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int lane, int E, float (&l)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = lane * V + v < E ? load(row + lane * V + v) : -INFINITY;
}

// V: experts a lane.  Up to eight, a lane puts its own in order first, so that each of the k rounds
// looks at one key a lane; with more, the order costs more than it saves.
template <typename T, int V, bool SOFTMAX, bool BIAS>
__global__ void __launch_bounds__(kWarpsR * 32) route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int k,
                                                            bool renorm, const float* __restrict__ bias,
                                                            float factor, int32_t* __restrict__ ids,
                                                            float* __restrict__ weights) {
  __shared__ int32_t taken[kWarpsR][32];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsR + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  int32_t* mine = taken[threadIdx.x >> 5];
  const T* row = logits + t * E;
  constexpr bool kOrdered = V <= 8;
  float l[V];
  uint32_t key[V], expert[V];
  bool nan = false;
  load_row(row, lane, E, l);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    float s = l[v];
    nan |= s != s;
    // a masked expert stays so: its sigmoid would be zero, above an expert's with a lower bias
    if (BIAS && e < E) s = (SOFTMAX || s == -INFINITY ? s : sigmoid(s)) + __ldg(bias + e);
    key[v] = order_of(s);
    expert[v] = e;
  }
  nan = __any_sync(kFull, nan);
  if (kOrdered) sort_keys(key, expert);
  int j = 0;
  for (; j < k; ++j) {
    uint32_t best = key[0], e = expert[0];
    if (!kOrdered) {
#pragma unroll
      for (int v = 1; v < V; ++v)
        if (key[v] > best) best = key[v], e = expert[v];
    }
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;   // the rest cannot be chosen
    // the first lane of equal ones holds the lowest index
    const uint32_t equal = __ballot_sync(kFull, best == top);
    if (lane == __ffs(equal) - 1) {
      mine[j] = static_cast<int32_t>(e);
      if (kOrdered) {
#pragma unroll
        for (int v = 0; v + 1 < V; ++v) key[v] = key[v + 1], expert[v] = expert[v + 1];
        key[V - 1] = 0;
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (expert[v] == e) key[v] = 0;
      }
    }
  }
  __syncwarp();
  const int id = lane < j ? mine[lane] : -1;     // lane j: slot j's expert
  const bool have = id >= 0;
  const float chosen = have ? load(row + id) : -INFINITY;
  float w;
  if (SOFTMAX) {
    float m = chosen, sum = 0.f;
    if (!renorm) {
#pragma unroll
      for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);
    }
    m = warp_max(m);
    const float ex = have ? exp_of(chosen - m) : 0.f;
    if (renorm) {
      sum = ex;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) sum += lane * V + v < E ? exp_of(l[v] - m) : 0.f;
    }
    w = __fdividef(ex, warp_sum(sum));     // the sum is between 1 and E
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

// The row's gradient that all experts share (-p mean, or zero) goes to shared memory, the lanes of
// the chosen add theirs, and the row is written once.
template <typename T, int V, bool SOFTMAX>
__global__ void __launch_bounds__(kWarpsR * 32) route_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E,
                                                                     int k, bool renorm, float factor,
                                                                     const int32_t* __restrict__ ids,
                                                                     const float* __restrict__ grad_weights,
                                                                     T* __restrict__ grad_logits) {
  __shared__ float grads[kWarpsR][32 * V];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarpsR + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= tokens) return;
  const T* row = logits + t * E;
  float* mine = grads[threadIdx.x >> 5];
  const bool every = SOFTMAX && !renorm;   // every expert's gradient, not the chosen ones' alone
  float p[V];
  if (every) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 32 * v + lane < E ? load(row + 32 * v + lane) : -INFINITY;
  }
  const int id = lane < k ? __ldg(ids + t * k + lane) : -1;
  const bool have = static_cast<unsigned>(id) < static_cast<unsigned>(E);
  const float g = have ? factor * __ldg(grad_weights + t * k + lane) : 0.f;
  const float chosen = have ? load(row + id) : -INFINITY;
  const bool full = every && __any_sync(kFull, have);
  float mean = 0.f, d = 0.f;
  if (SOFTMAX) {
    float m = chosen, sum = 0.f;
    if (full) {
#pragma unroll
      for (int v = 0; v < V; ++v) m = fmaxf(m, p[v]);
    }
    m = warp_max(m);
    const float ex = have ? exp_of(chosen - m) : 0.f;
    if (full) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = 32 * v + lane < E ? exp_of(p[v] - m) : 0.f;
        sum += p[v];
      }
    } else {
      sum = ex;
    }
    sum = warp_sum(sum);
    const float q = have ? __fdividef(ex, sum) : 0.f;     // the sum is between 1 and E
    mean = warp_sum(g * q);
    d = full ? g * q : q * (g - mean);
    const float share = full ? __fdividef(-mean, sum) : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = full ? p[v] * share : 0.f;
  } else {
    // 1 - s would lose its bits where s is near 1
    const float2 both = sigmoids(chosen);
    const float s = have ? both.x : 0.f, rest = both.y;
    d = g * s * rest;
    if (renorm) {
      // divided first: the quotients are at most 1 however small the sum is
      const float sum = warp_sum(s), q = sum != 0.f ? s / sum : 0.f;
      d = q * (g - warp_sum(g * q)) * rest;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 0.f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) mine[32 * v + lane] = p[v];
  __syncwarp();
  // one lane an expert adds; ids that are given twice take turns, the first lane first
  const uint32_t same = same_lanes(have ? id : 32 * V, 6 + log2_of(V));
  const int before = __popc(same & ((1u << lane) - 1u));
  const int turns = __reduce_max_sync(kFull, have ? before : 0);
  for (int n = 0; n <= turns; ++n) {
    if (have && before == n) mine[id] += d;
    __syncwarp();
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (32 * v + lane < E) store(grad_logits + t * E + 32 * v + lane, mine[32 * v + lane]);
}

template <typename T, int V>
void launch_v(const RouteArgs& a, unsigned grid) {
  const T* logits = static_cast<const T*>(a.logits);
  const bool softmax = a.gate == BSQ_GATE_SOFTMAX;
  const auto backward = [&](auto kernel) {
    kernel<<<grid, kWarpsR * 32, 0, a.stream>>>(logits, a.T, a.E, a.k, a.renormalize, a.factor, a.ids, a.grad_weights,
                                                static_cast<T*>(a.grad_logits));
  };
  const auto forward = [&](auto kernel) {
    kernel<<<grid, kWarpsR * 32, 0, a.stream>>>(logits, a.T, a.E, a.k, a.renormalize, a.bias, a.factor, a.ids, a.weights);
  };
  if (a.grad_logits && softmax) backward(route_backward_kernel<T, V, true>);
  else if (a.grad_logits) backward(route_backward_kernel<T, V, false>);
  else if (softmax && a.bias) forward(route_kernel<T, V, true, true>);
  else if (softmax) forward(route_kernel<T, V, true, false>);
  else if (a.bias) forward(route_kernel<T, V, false, true>);
  else forward(route_kernel<T, V, false, false>);
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

}  // namespace

int launch_route(const RouteArgs& a, const char** msg) {
  return a.dtype == BSQ_DT_BF16 ? launch_typed<__nv_bfloat16>(a, msg) : launch_typed<float>(a, msg);
}

}  // namespace bsq
