// bsq_fp4_smallm.cu -- products of a few BF16 token rows with 4-bit weights (decode), dense and
// per expert:  y[m, n] = sum_k x[m, k] deq(W)[n, k],  deq = RNE_bf16(code * RNE_bf16(scale)).
//
// Bound by reading W once, half a byte and a scale's share per element, and beside that by the
// instructions that decode it.  A CTA owns 16 MT columns of y (rows of W) and the whole
// contraction; its warps take pieces of it in turn, each thread streaming W straight into the
// register fragments of mma.m16n8k16.  The order of k inside a piece is free as long as both
// operands share it: a thread takes 16 bytes (32 codes) of a row, whose 8-code words decode to
// the pairs (c0, c4), (c1, c5), ... without a permutation (bsq_decode.cuh); the tokens' values
// are brought to that order instead, once for all rows of W.  The warps' accumulators are added
// in warp order through shared memory, so results do not depend on timing.
#include <cuda_bf16.h>

#include "bsq_decode.cuh"
#include "bsq_moe_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kOnex2 = 0x3F803F80u;     // BF16 pair (1, 1)

struct Fp4SmallParams {
  const __nv_bfloat16* x;
  const uint8_t* w;
  const uint8_t* ws;
  const float* ts;
  __nv_bfloat16* y;
  const int32_t* offsets;
  int32_t* err;
  int32_t S, N, K, E;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// W is read once: kept out of L1 so that the tokens stay there.
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Factors of a scale: the decoded pair times `first`, and where any of them is not fast, times
// `second` too (1 for a fast one).
struct Factors {
  uint32_t first, second;
  __device__ __forceinline__ bool set(const ScaleBf16& s) {
    first = s.fast ? s.c2 : kPow2_126x2;
    second = s.fast ? kOnex2 : s.s2;
    return s.fast;
  }
};

// MT: 16-row groups of W a CTA; NT: groups of 8 tokens per pass over W; H: pieces of 128 k a
// warp loads at once; WARPS of a CTA; CTAS an SM shall hold.
template <int FMT, int MT, int NT, int H, int WARPS, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS) fp4_smallm_kernel(const Fp4SmallParams p) {
  constexpr int kRows = 16 * MT, kPad = kRows + 4;   // the pitch keeps fragment writes free of bank conflicts
  constexpr int kScales = FMT == BSQ_NVFP4 ? 2 : 1;  // scales of a thread's 32 codes
  __shared__ float red[WARPS][8][kPad];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int e = blockIdx.y;
  int r0 = 0, r1 = p.S, bad = 0;
  if (p.offsets) {
    r0 = e > 0 ? __ldg(p.offsets + e - 1) : 0;
    r1 = __ldg(p.offsets + e);
    for (int i = tid; i < p.E; i += WARPS * 32) {
      const int a = i > 0 ? __ldg(p.offsets + i - 1) : 0, b = __ldg(p.offsets + i);
      bad |= a < 0 || b < a || b > p.S;
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0 && blockIdx.x == 0 && e == 0) atomicCAS(p.err, 0, BSQ_DEVERR_BAD_OFFSETS);
    if (bad || r0 == r1) return;
  }
  const int n0 = blockIdx.x * kRows;
  // Rows past N: any row, not stored.  Offsets of a CTA's rows fit 32 bits (K <= 2^24).
  const int rows_left = p.N - 1 - n0;
  const int64_t row0 = static_cast<int64_t>(e) * p.N + n0;
  const uint32_t wpitch = static_cast<uint32_t>(p.K) >> 1, spitch = static_cast<uint32_t>(p.K) >> (FMT == BSQ_NVFP4 ? 4 : 5);
  const uint8_t* wbase = p.w + row0 * wpitch + 16 * t;
  const uint8_t* sbase = p.ws + row0 * spitch + kScales * t;
  const float ts = FMT == BSQ_NVFP4 ? __ldg(p.ts + e) : 0.f;

  for (int m0 = r0; m0 < r1; m0 += 8 * NT) {
    const int left = r1 - m0;
    const __nv_bfloat16* xbase = p.x + static_cast<int64_t>(m0) * p.K + 32 * t;
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = 0.f;

#pragma unroll 1
    for (int k0 = warp * (128 * H); k0 < p.K; k0 += WARPS * (128 * H)) {
      uint4 wv[H][MT][2];
      uint32_t sv[H][MT][2];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int k = k0 + 128 * h;
        const bool in = k + 32 * t < p.K;     // K % 32 == 0: whole pieces of 32 codes
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t row = static_cast<uint32_t>(min(16 * i + 8 * q + g, rows_left));
            wv[h][i][q] = in ? ldg_stream(wbase + (row * wpitch + (k >> 1))) : make_uint4(0, 0, 0, 0);
            const uint8_t* s = sbase + (row * spitch + (k >> (FMT == BSQ_NVFP4 ? 4 : 5)));
            if (FMT == BSQ_NVFP4) sv[h][i][q] = in ? __ldg(reinterpret_cast<const uint16_t*>(s)) : 0u;
            else sv[h][i][q] = in ? __ldg(s) : 127u;
          }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int k = k0 + 128 * h;
        const bool in = k + 32 * t < p.K;
        // the tokens' values in the order of the decoded pairs: [word of 8][pair]
        uint32_t xp[NT][4][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int m = 8 * j + g;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in && m < left) v = __ldg(reinterpret_cast<const uint4*>(xbase + (static_cast<int64_t>(m) * p.K + k + 8 * q)));
            unzip_pairs(v.x, v.z, xp[j][q][0], xp[j][q][1]);
            unzip_pairs(v.y, v.w, xp[j][q][2], xp[j][q][3]);
          }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          Factors f[2][kScales];
          bool fast = true;
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int s = 0; s < kScales; ++s)
              fast &= f[q][s].set(FMT == BSQ_NVFP4 ? make_scale_nvfp4(sv[h][i][q] >> (8 * s), ts) : make_scale_e8m0(sv[h][i][q]));
          const bool slow = __any_sync(kFull, !fast);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t a[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const Factors& m = f[q][kScales == 2 ? c >> 1 : 0];
              spread_e2m1x8(word(wv[h][i][q], c), a[q]);
#pragma unroll
              for (int u = 0; u < 4; ++u) a[q][u] = bf16x2_mul(a[q][u], m.first);
              if (slow) {
#pragma unroll
                for (int u = 0; u < 4; ++u) a[q][u] = bf16x2_mul(a[q][u], m.second);
              }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma_bf16(acc[i][j], a[0][0], a[1][0], a[0][1], a[1][1], xp[j][c][0], xp[j][c][1]);
              mma_bf16(acc[i][j], a[0][2], a[1][2], a[0][3], a[1][3], xp[j][c][2], xp[j][c][3]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (8 * j >= left) break;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        red[warp][2 * t][16 * i + g] = acc[i][j][0];
        red[warp][2 * t + 1][16 * i + g] = acc[i][j][1];
        red[warp][2 * t][16 * i + 8 + g] = acc[i][j][2];
        red[warp][2 * t + 1][16 * i + 8 + g] = acc[i][j][3];
      }
      __syncthreads();
      for (int o = tid; o < 8 * kRows; o += WARPS * 32) {
        const int m = o / kRows, n = o % kRows;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += red[w][m][n];
        if (8 * j + m < left && n <= rows_left) p.y[static_cast<int64_t>(m0 + 8 * j + m) * p.N + n0 + n] = __float2bfloat16_rn(s);
      }
      __syncthreads();
    }
  }
}

template <int FMT, int MT, int NT, int H, int WARPS, int CTAS>
int launch_typed(const Fp4SmallParams& p, const Fp4Args& a, const char** msg) {
  const dim3 grid(static_cast<unsigned>((a.N + 16 * MT - 1) / (16 * MT)), static_cast<unsigned>(a.offsets ? a.E : 1));
  fp4_smallm_kernel<FMT, MT, NT, H, WARPS, CTAS><<<grid, WARPS * 32, 0, a.stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

template <int FMT>
int launch_fmt(const Fp4SmallParams& p, const Fp4Args& a, const char** msg) {
  const int64_t rows = a.offsets ? (a.S + a.E - 1) / a.E : a.S;
  if (rows <= 8) return launch_typed<FMT, 2, 1, 2, 8, 2>(p, a, msg);
  if (rows <= 16) return launch_typed<FMT, 2, 2, 1, 8, 2>(p, a, msg);
  return launch_typed<FMT, 2, 4, 1, 8, 2>(p, a, msg);
}

}  // namespace

bool fp4_takes_smallm(const Fp4Args& a) { return a.S <= 64; }

int launch_fp4_smallm(const Fp4Args& a, const char** msg) {
  Fp4SmallParams p;
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.w = static_cast<const uint8_t*>(a.w);
  p.ws = static_cast<const uint8_t*>(a.w_scale);
  p.ts = a.tensor_scale;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.offsets = a.offsets;
  p.err = a.err;
  p.S = static_cast<int32_t>(a.S);
  p.N = static_cast<int32_t>(a.N);
  p.K = static_cast<int32_t>(a.K);
  p.E = static_cast<int32_t>(a.E);
  return a.fmt == BSQ_MXFP4 ? launch_fmt<BSQ_MXFP4>(p, a, msg) : launch_fmt<BSQ_NVFP4>(p, a, msg);
}

}  // namespace bsq
