// bsq_tokens.cu -- tokens to their experts' rows and back.
//
//   sort      rows[i] = place of slot i (token i / k) when slots are sorted by expert, stable
//   dispatch  out[rows[t, j]] = w[t, j] x[t], as BF16 and as E4M3 codes of x[t] in blocks of 128
//             columns with the blocks' scales times w[t, j]
//   combine   out[t] = sum_j w[t, j] y[rows[t, j]], in the order of j, float32, rounded once
//   backward  grad_y[rows[t, j]] = w[t, j] g[t] (as dispatch), grad_w[t, j] = g[t] . y[rows[t, j]]
//
// All but the sort are bound by HBM: a token's columns are read once, whatever k is, and a
// token's codes are made once, since a weight only changes a block's scale.  Dispatch of 4096
// tokens of 2048 to four rows each, as BF16 and E4M3: 17.3 us, 6.8 TB/s; combine of eight rows of 7168
// for 8191 tokens 153 us, 6.9 TB/s; of four of 2816 for 4096 tokens 20.7, its gradients 40.0 (6.4).
#include <atomic>
#include <cuda_bf16.h>

#include "bsq_e4m3.cuh"
#include "bsq_internal.h"
#include "bsq_lanes.cuh"
#include "bsq_moe_internal.h"
#include "bsq_ptx.cuh"
#include "../../include/bsq.h"

namespace bsq {

namespace {

int last_error(const char** msg) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return 0;
  *msg = cudaGetErrorString(e);
  return static_cast<int>(e);
}

// ---------------------------------------------------------------- sort
constexpr int kSortWarps = 32;
constexpr int kMaxSortSmem = (kSortWarps + 2) * kMaxExperts * 4;
constexpr int kAheadS = 4;       // ids a lane loads before the first is counted, where it does not hold them all

// Counts a warp's 32 slots: the number of slots of the same expert before each, within the warp's run;
// `mine`: the warp's counters.  Lanes of one expert find one another by votes, so nothing is added
// atomically.  bits: of E.
__device__ __forceinline__ int32_t count_slots(int32_t* mine, int e, bool in, uint32_t below, int E, int bits) {
  const uint32_t same = same_lanes(in ? e : E, bits);
  const int32_t before = in ? mine[e] + __popc(same & below) : 0;
  __syncwarp();
  if (in && (same & below) == 0) mine[e] += __popc(same);
  __syncwarp();
  return before;
}

// A counting sort in one launch of one cluster.  Every warp counts its run of slots in
// counters of its own, the counts become first places (over warps, CTAs through distributed
// shared memory, then experts), and every slot's place is its expert's first plus its rank.
// HELD: slots a lane holds in registers, 32 HELD a warp's run; 0: any run, read and counted twice.
// Bound by latency: 64 slots on 64 experts 2.6 us, 16384 4.9, 32764 on 128 6.5; then by the
// scattered stores of `slots`, of which an SM does a sector a cycle (131072 on 128 experts 12.9 us).
template <int HELD>
__global__ void __launch_bounds__(kSortWarps * 32) sort_experts_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                                      int64_t run, int ctas, int32_t* __restrict__ offsets,
                                                                      int32_t* __restrict__ rows, int32_t* __restrict__ slots) {
  extern __shared__ int32_t counts[];      // [kSortWarps][E], total[E], base[E]
  int32_t* total = counts + kSortWarps * E;
  int32_t* base = total + E;
  __shared__ int32_t wsum[kSortWarps];
  __shared__ int32_t kept;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x);
  const int64_t begin = min(n, (static_cast<int64_t>(rank) * kSortWarps + warp) * run), end = min(n, begin + run);
  const uint32_t below = (1u << lane) - 1u;
  int held[HELD > 0 ? HELD : 1], rank_of[HELD > 0 ? HELD : 1];
#pragma unroll
  for (int u = 0; u < HELD; ++u) held[u] = begin + 32 * u + lane < end ? __ldg(ids + begin + 32 * u + lane) : -1;
  for (int i = tid; i < kSortWarps * E; i += kSortWarps * 32) counts[i] = 0;
  __syncthreads();
  int32_t* mine = counts + warp * E;
  const int bits = 32 - __clz(E);
  const auto known = [&](int e) { return static_cast<unsigned>(e) < static_cast<unsigned>(E); };

  if (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; ++u) rank_of[u] = count_slots(mine, held[u], known(held[u]), below, E, bits);
  } else {
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kAheadS) {
      int e[kAheadS];
#pragma unroll
      for (int u = 0; u < kAheadS; ++u) e[u] = i0 + 32 * u + lane < end ? __ldg(ids + i0 + 32 * u + lane) : -1;
#pragma unroll
      for (int u = 0; u < kAheadS; ++u) count_slots(mine, e[u], known(e[u]), below, E, bits);
    }
  }
  __syncthreads();
  int32_t sum = 0;                          // thread e: slots of expert e in this CTA
  if (tid < E) {
#pragma unroll
    for (int w0 = 0; w0 < kSortWarps; w0 += 8) {
      int32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = counts[(w0 + w) * E + tid];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        counts[(w0 + w) * E + tid] = sum;
        sum += c[w];
      }
    }
    total[tid] = sum;
  }
  int32_t before = 0, all = sum;
  if (ctas > 1) {
    cluster_sync();
    if (tid < E) {
      all = 0;
#pragma unroll 8
      for (int c = 0; c < ctas; ++c) {
        const int32_t v = static_cast<int32_t>(ld_shared_cluster_u32(map_to_rank(smem_u32(total + tid), c)));
        before += c < rank ? v : 0;
        all += v;
      }
    }
  }
  int32_t upto = tid < E ? all : 0;         // inclusive sum over experts (E <= 1024, one a thread)
  const int32_t own = upto;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t v = __shfl_up_sync(kFull, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  upto += __reduce_add_sync(kFull, lane < warp ? wsum[lane] : 0);
  if (tid < E) {
    base[tid] = upto - own + before;
    if (rank == 0) offsets[tid] = upto;
    if (tid == E - 1) kept = upto;
  }
  // No CTA leaves before the cluster has read its counts: said here, waited for at the end.
  if (ctas > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  __syncthreads();

  const auto place = [&](int64_t i, int e, int32_t at) {
    const int32_t row = known(e) ? base[e] + at : -1;
    if (i < end) rows[i] = row;
    if (known(e) && slots) slots[row] = static_cast<int32_t>(i);
  };
  if (HELD > 0) {
#pragma unroll
    for (int u = 0; u < HELD; ++u) place(begin + 32 * u + lane, held[u], rank_of[u] + (known(held[u]) ? mine[held[u]] : 0));
  } else {
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kAheadS) {
      int e[kAheadS];
#pragma unroll
      for (int u = 0; u < kAheadS; ++u) e[u] = i0 + 32 * u + lane < end ? __ldg(ids + i0 + 32 * u + lane) : -1;
#pragma unroll
      for (int u = 0; u < kAheadS; ++u) place(i0 + 32 * u + lane, e[u], count_slots(mine, e[u], known(e[u]), below, E, bits));
    }
  }
  if (slots)
    for (int64_t i = static_cast<int64_t>(kept) + rank * (kSortWarps * 32) + tid; i < n; i += static_cast<int64_t>(ctas) * (kSortWarps * 32))
      slots[i] = -1;
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---------------------------------------------------------------- rows of a token
// Lane j < k holds slot j's row (-1: none) and weight.
struct Slots {
  int32_t row;
  float weight;
  __device__ Slots(const int32_t* rows, const float* weights, int64_t t, int k, int64_t S, int lane) {
    row = lane < k ? __ldg(rows + t * k + lane) : -1;
    if (row >= S) row = -1;
    weight = weights && lane < k ? __ldg(weights + t * k + lane) : 1.f;
  }
};

__device__ __forceinline__ uint32_t scaled_pair(uint32_t v, float w) {
  return pack_bf16x2(__float_as_uint(__uint_as_float(v << 16) * w), __float_as_uint(__uint_as_float(v & 0xFFFF0000u) * w));
}
__device__ __forceinline__ uint4 scaled(const uint4& v, float w) {
  return make_uint4(scaled_pair(v.x, w), scaled_pair(v.y, w), scaled_pair(v.z, w), scaled_pair(v.w, w));
}
// Largest magnitude of the 128-column block that 16 lanes of eight columns hold.
__device__ __forceinline__ float block_amax16(const Eight<__nv_bfloat16>& v) {
  uint32_t m = v.amax();
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(kFull, m, d));
  return block_amax(m);
}

constexpr int kThreadsT = 128;
constexpr int kPieces = 2;       // pieces of 256 columns (eight a lane) per warp

template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(kThreadsT) dispatch_kernel(const __nv_bfloat16* __restrict__ x, int64_t tokens, int64_t S,
                                                            int cols, int segs, int nblocks, const int32_t* __restrict__ rows,
                                                            int k, const float* __restrict__ weights,
                                                            __nv_bfloat16* __restrict__ out, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scale) {
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreadsT / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = item / segs;
  if (t >= tokens) return;
  const Slots s(rows, weights, t, k, S, lane);
  // unsigned: a token may end within the last piece before 2^31
  const uint32_t c0 = static_cast<uint32_t>(item - t * segs) * (256 * kPieces) + lane * 8, end = cols;
  Eight<__nv_bfloat16> v[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (c0 + 256 * i < end) v[i].load(x + t * cols + c0 + 256 * i);
    else v[i].zero();
  }
  float sc[kPieces];
  uint2 code[kPieces];
  if (E4M3) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const float a = block_amax16(v[i]);
      code[i] = encode(v[i], __fdiv_rn(448.f, a));
      sc[i] = __fdiv_rn(a, 448.f);
    }
  }
  for (int j = 0; j < k; ++j) {
    const int64_t r = __shfl_sync(kFull, s.row, j);
    const float w = __shfl_sync(kFull, s.weight, j);
    if (r < 0) continue;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t c = c0 + 256 * i;
      if (c >= end) continue;
      if (BF16) *reinterpret_cast<uint4*>(out + r * cols + c) = weights ? scaled(v[i].v, w) : v[i].v;
      if (E4M3) {
        *reinterpret_cast<uint2*>(codes + r * cols + c) = code[i];
        if ((lane & 15) == 0) scale[r * nblocks + (c >> 7)] = sc[i] * w;
      }
    }
  }
}

// Slots whose rows are in flight together.
constexpr int kTogether = 4;

// U: pieces of 256 columns a warp sums, all their loads in flight at once.
template <int U>
__global__ void __launch_bounds__(kThreadsT) combine_kernel(const __nv_bfloat16* __restrict__ y, int64_t tokens, int64_t S,
                                                           int cols, int segs, const int32_t* __restrict__ rows, int k,
                                                           const float* __restrict__ weights, __nv_bfloat16* __restrict__ out) {
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreadsT / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = item / segs;
  if (t >= tokens) return;
  const Slots s(rows, weights, t, k, S, lane);
  // unsigned: a row may end within the last piece before 2^31
  const uint32_t c0 = static_cast<uint32_t>(item - t * segs) * (256 * U) + lane * 8, end = cols;
  float acc[U][8] = {};
  for (int j0 = 0; j0 < k; j0 += kTogether) {
    Eight<__nv_bfloat16> v[kTogether][U];
    float w[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const int64_t r = __shfl_sync(kFull, s.row, j0 + u);     // j0 + u < 32; lanes from k on hold -1
      w[u] = __shfl_sync(kFull, s.weight, j0 + u);
      if (r < 0) w[u] = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (r >= 0 && c0 + 256 * i < end) v[u][i].load(y + r * cols + c0 + 256 * i);
        else v[u][i].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = v[u][i].pair(q);
          acc[i][2 * q] = fmaf(w[u], f.x, acc[i][2 * q]);
          acc[i][2 * q + 1] = fmaf(w[u], f.y, acc[i][2 * q + 1]);
        }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (c0 + 256 * i >= end) continue;
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(__float_as_uint(acc[i][2 * q]), __float_as_uint(acc[i][2 * q + 1]));
    *reinterpret_cast<uint4*>(out + t * cols + c0 + 256 * i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Small CTAs, whose warps end at about the same time (4096 tokens of four rows of 2816, two warps a token: 42.5 us
// in CTAs of eight warps, 41.1 in CTAs of four; the weights' gradient alone 22.1 and 20.2).
constexpr int backward_warps(int wpt) { return wpt > kThreadsT / 32 ? wpt : kThreadsT / 32; }

// WPT warps of a CTA share a token: 2 with tokens enough to fill the GPU, else 8.
template <bool BF16, bool E4M3, bool DOT, int WPT>
__global__ void __launch_bounds__(backward_warps(WPT) * 32) combine_backward_kernel(
    const __nv_bfloat16* __restrict__ g, const __nv_bfloat16* __restrict__ y, int64_t tokens, int64_t S, int cols, int nblocks,
    const int32_t* __restrict__ rows, int k, const float* __restrict__ weights, __nv_bfloat16* __restrict__ out,
    uint8_t* __restrict__ codes, float* __restrict__ scale, float* __restrict__ grad_weights) {
  constexpr int kWarps = backward_warps(WPT), kTokens = kWarps / WPT, G = kTogether, U = 2;
  __shared__ float part[kWarps][G];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t own = static_cast<int64_t>(blockIdx.x) * kTokens + warp / WPT;
  const bool there = own < tokens;          // all warps of a CTA stay together for the barriers
  const int64_t t = there ? own : tokens - 1;
  Slots s(rows, weights, t, k, S, lane);
  if (!there) s.row = -1;
  for (int j0 = 0; j0 < k; j0 += G) {
    int64_t r[G];
    float w[G], dot[G];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      r[u] = __shfl_sync(kFull, s.row, j0 + u);
      w[u] = __shfl_sync(kFull, s.weight, j0 + u);
      dot[u] = 0.f;
    }
    for (uint32_t piece = static_cast<uint32_t>(warp % WPT) * (256 * U); piece < static_cast<uint32_t>(cols); piece += WPT * 256 * U) {
      Eight<__nv_bfloat16> a[U], b[G][U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = piece + 256 * i + lane * 8;
        const bool in = c < static_cast<uint32_t>(cols);
        if (in) a[i].load(g + t * cols + c);
        else a[i].zero();
        if (DOT) {
#pragma unroll
          for (int u = 0; u < G; ++u) {
            if (r[u] >= 0 && in) b[u][i].load(y + r[u] * cols + c);
            else b[u][i].zero();
          }
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t c = piece + 256 * i + lane * 8;
        const bool in = c < static_cast<uint32_t>(cols);
        uint2 code = make_uint2(0, 0);
        float sc = 0.f;
        if (E4M3) {
          const float m = block_amax16(a[i]);
          code = encode(a[i], __fdiv_rn(448.f, m));
          sc = __fdiv_rn(m, 448.f);
        }
#pragma unroll
        for (int u = 0; u < G; ++u) {
          if (r[u] < 0) continue;
          if (DOT) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 x = a[i].pair(q), z = b[u][i].pair(q);
              dot[u] = fmaf(x.x, z.x, fmaf(x.y, z.y, dot[u]));
            }
          }
          if (!in) continue;
          if (BF16) *reinterpret_cast<uint4*>(out + r[u] * cols + c) = weights ? scaled(a[i].v, w[u]) : a[i].v;
          if (E4M3) {
            *reinterpret_cast<uint2*>(codes + r[u] * cols + c) = code;
            if ((lane & 15) == 0) scale[r[u] * nblocks + (c >> 7)] = sc * w[u];
          }
        }
      }
    }
    if (DOT) {
#pragma unroll
      for (int u = 0; u < G; ++u) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot[u] += __shfl_xor_sync(kFull, dot[u], d);
      }
      if (lane == 0) {
#pragma unroll
        for (int u = 0; u < G; ++u) part[warp][u] = dot[u];
      }
      __syncthreads();
      if (there && warp % WPT == 0 && lane < G && j0 + lane < k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < WPT; ++i) sum += part[warp + i][lane];
        grad_weights[t * k + j0 + lane] = sum;
      }
      if (j0 + G < k) __syncthreads();
    }
  }
}

struct SortLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  SortLaunch(int ctas, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kSortWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
  }
};

// Whether a cluster of 16 such CTAs fits this device, which is asked once.
bool sixteen_fit() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  int k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    const auto kernel = sort_experts_kernel<16>;
    const SortLaunch l(16, kMaxSortSmem, nullptr);
    int clusters = 0;
    const bool asked = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSortSmem) == cudaSuccess &&
                       cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                       cudaOccupancyMaxActiveClusters(&clusters, kernel, &l.cfg) == cudaSuccess;
    if (!asked) cudaGetLastError();
    k = asked && clusters > 0 ? 1 : 2;
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 1;
}

}  // namespace

int launch_sort_experts(const SortArgs& a, const char** msg) {
  // One CTA while a warp of it has few slots, then eight (8192 on 64 experts: 4.6 us, with sixteen 4.9), then
  // sixteen, where the device has a place for such a cluster (16384: 5.8 us with eight, 4.9 with
  // sixteen; 131072 on 128: 21.6 and 12.9; 800000 on 256: 146 and 79).
  const int ctas = a.n <= 1024 ? 1 : a.n <= 8192 || !sixteen_fit() ? 8 : 16;
  // a warp's run, in whole warps of slots
  const int64_t run = ((a.n + ctas * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32;
  auto kernel = sort_experts_kernel<0>;
  if (run <= 32) kernel = sort_experts_kernel<1>;
  else if (run <= 64) kernel = sort_experts_kernel<2>;
  else if (run <= 128) kernel = sort_experts_kernel<4>;
  else if (run <= 256) kernel = sort_experts_kernel<8>;
  else if (run <= 512) kernel = sort_experts_kernel<16>;
  const size_t smem = static_cast<size_t>(kSortWarps + 2) * a.E * 4;
  // The limit is the function's, for all host threads: always the largest, so that no call lowers it
  // between another's setting and its launch.
  cudaError_t e = cudaSuccess;
  if (smem > 47 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSortSmem);
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) {
    SortLaunch l(ctas, smem, a.stream);
    e = cudaLaunchKernelEx(&l.cfg, kernel, a.ids, a.n, a.E, run, ctas, a.offsets, a.rows, a.slots);
  }
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

int launch_dispatch(const TokenArgs& a, const char** msg) {
  const int cols = static_cast<int>(a.cols), nb = static_cast<int>((a.cols + 127) / 128);
  const int segs = static_cast<int>((a.cols + 256 * kPieces - 1) / (256 * kPieces));
  const int64_t grid = (a.T * segs + kThreadsT / 32 - 1) / (kThreadsT / 32);
  if (grid > INT32_MAX) {
    *msg = "too many blocks";
    return -1;
  }
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kThreadsT, 0, a.stream>>>(
        static_cast<const __nv_bfloat16*>(a.x), a.T, a.S, cols, segs, nb, a.rows, a.k, a.weights,
        static_cast<__nv_bfloat16*>(a.out), static_cast<uint8_t*>(a.codes), a.scale);
  };
  if (a.out && a.codes) go(dispatch_kernel<true, true>);
  else if (a.out) go(dispatch_kernel<true, false>);
  else go(dispatch_kernel<false, true>);
  return last_error(msg);
}

int launch_combine(const TokenArgs& a, const char** msg) {
  // Two pieces a warp (8191 tokens of eight rows of 7168 153 us, with one 170), four where there are many
  // tokens whose last piece of 1024 columns is more than half full (4096 of four of 2816: 20.7 us,
  // with two 21.4; 1300 of eight of 4096: 18.5, with two 17.0; 16 of four of 2816: 2.6, with two 2.3).
  const bool four = a.T >= 16ll * a.num_sms && (a.cols - 1) % 1024 >= 512;
  const int segs = static_cast<int>(four ? (a.cols + 1023) / 1024 : (a.cols + 511) / 512);
  const int64_t grid = (a.T * segs + kThreadsT / 32 - 1) / (kThreadsT / 32);
  if (grid > INT32_MAX) {
    *msg = "too many blocks";
    return -1;
  }
  const auto kernel = four ? combine_kernel<4> : combine_kernel<2>;
  kernel<<<static_cast<unsigned>(grid), kThreadsT, 0, a.stream>>>(
      static_cast<const __nv_bfloat16*>(a.y), a.T, a.S, static_cast<int>(a.cols), segs, a.rows, a.k, a.weights,
      static_cast<__nv_bfloat16*>(a.out));
  return last_error(msg);
}

int launch_combine_backward(const TokenArgs& a, const char** msg) {
  const int cols = static_cast<int>(a.cols), nb = static_cast<int>((a.cols + 127) / 128);
  // four rows of 2816: 450 tokens 5.0 us with eight warps a token, 6.2 with two; 700: 7.5 and 7.2; 4096: 44.7 and 41.1
  // (with four 41.7; with one 44.1)
  const int wpt = a.T >= 4ll * a.num_sms ? 2 : 8;
  const int warps = backward_warps(wpt);
  const int64_t grid = (a.T * wpt + warps - 1) / warps;
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), warps * 32, 0, a.stream>>>(
        static_cast<const __nv_bfloat16*>(a.x), static_cast<const __nv_bfloat16*>(a.y), a.T, a.S, cols, nb, a.rows, a.k,
        a.weights, static_cast<__nv_bfloat16*>(a.out), static_cast<uint8_t*>(a.codes), a.scale, a.grad_weights);
  };
  const int what = (a.out ? 4 : 0) | (a.codes ? 2 : 0) | (a.grad_weights ? 1 : 0);
  const auto pick = [&](auto wpt) {
    constexpr int W = decltype(wpt)::value;
    switch (what) {
      case 1: go(combine_backward_kernel<false, false, true, W>); break;
      case 2: go(combine_backward_kernel<false, true, false, W>); break;
      case 3: go(combine_backward_kernel<false, true, true, W>); break;
      case 4: go(combine_backward_kernel<true, false, false, W>); break;
      case 5: go(combine_backward_kernel<true, false, true, W>); break;
      case 6: go(combine_backward_kernel<true, true, false, W>); break;
      case 7: go(combine_backward_kernel<true, true, true, W>); break;
    }
  };
  if (wpt == 8) pick(std::integral_constant<int, 8>{});
  else pick(std::integral_constant<int, 2>{});
  return last_error(msg);
}

}  // namespace bsq
