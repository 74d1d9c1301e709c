// bsq_fp8_smallm.cu -- the forward of E4M3 operands for a few token rows (decode), dense and
// per expert:  y[m, n] = sum_b xs[m, b] ws[n/128, b] sum_{k in b} xc[m, k] wc[n, k].
//
// Bound by reading W once.  A CTA owns 32 columns of y (rows of W) and the whole
// contraction; its warps take the 128-deep blocks in turn, each thread streaming W
// straight into the register fragments of mma.m16n8k32 (no shared memory, no barrier
// between the load and its use).  A fragment wants 4-byte pieces 16 k apart; the order of k
// inside a block is free as long as both operands share it, so each thread instead takes
// 16 consecutive bytes of its row for two MMAs, and the token codes are read the same way.
// Every block's partial sum is scaled into FP32 accumulators; the warps' accumulators are
// added in warp order through shared memory, so results do not depend on timing.
//
// Measured: 64 experts of 2816 x 2048, 64 skewed rows, 30.7 us, 5.3 TB/s; 4096 x 4096, 16 rows,
// 7.2 us on the device, 2.3 TB/s (too short a kernel to fill the memory's pipe).
#include <cuda_bf16.h>

#include "bsq_fp8_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

constexpr int kColsS = 32;              // columns of y per CTA
constexpr int kPadS = kColsS + 4;       // row pitch of the reduction buffer: conflict-free fragment writes

struct Fp8SmallParams {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  __nv_bfloat16* y;
  const int32_t* offsets;
  int32_t* err;
  int32_t S, N, K, E, kblocks;
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// W is read once: kept out of L1 so that the token codes stay there.
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// NT: groups of 8 tokens per pass over W.  WARPS of a CTA; AHEAD: a block's W is loaded while
// the one before it is multiplied; CTAS an SM shall hold.
template <int NT, int WARPS, bool AHEAD, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS) fp8_smallm_kernel(const Fp8SmallParams p) {
  __shared__ float red[WARPS][8 * NT][kPadS];
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
  const int n0 = blockIdx.x * kColsS;
  // One pointer each for W and the tokens; a fragment's rows are 32-bit offsets from them
  // (8 rows of W, 8 tokens apart).  Rows past N: any row, not stored.
  const int rows_left = p.N - 1 - n0;
  const uint8_t* wbase = p.w + (static_cast<int64_t>(e) * p.N + n0) * p.K + 16 * t;
  uint32_t woff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) woff[i] = static_cast<uint32_t>(min(8 * i + g, rows_left)) * static_cast<uint32_t>(p.K);
  const float* ws = p.ws + (static_cast<int64_t>(e) * ((p.N + 127) >> 7) + (n0 >> 7)) * p.kblocks;

  for (int m0 = r0; m0 < r1; m0 += 8 * NT) {
    // tokens past the last: any token, not stored
    const int last = r1 - 1 - m0;
    const uint8_t* xbase = p.x + static_cast<int64_t>(m0) * p.K + 16 * t;
    const float* sbase = p.xs + static_cast<int64_t>(m0) * p.kblocks;
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = 0.f;

    // the codes of one block: [half of 64 k][row of the fragment]
    auto load_w = [&](int kb, uint4 (&v)[2][4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kb * 128 + 64 * h;
        const bool in = k + 16 * t < p.K;   // K % 16 == 0: whole 16-byte pieces
#pragma unroll
        for (int i = 0; i < 4; ++i) v[h][i] = in ? ldg_stream(wbase + (woff[i] + k)) : make_uint4(0, 0, 0, 0);
      }
    };
    uint4 next[2][4];
    if (AHEAD && warp < p.kblocks) load_w(warp, next);
#pragma unroll 1
    for (int kb = warp; kb < p.kblocks; kb += WARPS) {
      uint4 cur[2][4];
      if (AHEAD) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) cur[h][i] = next[h][i];
      } else {
        load_w(kb, cur);
      }
      uint4 xv[NT][2];
      float sx[NT][2];
      const float sw = __ldg(ws + kb);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kb * 128 + 64 * h;
          const uint32_t off = static_cast<uint32_t>(min(8 * j + g, last)) * static_cast<uint32_t>(p.K) + k;
          xv[j][h] = k + 16 * t < p.K ? __ldg(reinterpret_cast<const uint4*>(xbase + off)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) sx[j][i] = __ldg(sbase + (min(8 * j + 2 * t + i, last) * p.kblocks + kb));
      }
      if (AHEAD && kb + WARPS < p.kblocks) load_w(kb + WARPS, next);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 &lo = cur[h][2 * i], &hi = cur[h][2 * i + 1], &x = xv[j][h];
            mma_e4m3(c, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
            mma_e4m3(c, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
          }
          const float s0 = sx[j][0] * sw, s1 = sx[j][1] * sw;
          acc[i][j][0] += c[0] * s0;
          acc[i][j][1] += c[1] * s1;
          acc[i][j][2] += c[2] * s0;
          acc[i][j][3] += c[3] * s1;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        red[warp][8 * j + 2 * t][16 * i + g] = acc[i][j][0];
        red[warp][8 * j + 2 * t + 1][16 * i + g] = acc[i][j][1];
        red[warp][8 * j + 2 * t][16 * i + 8 + g] = acc[i][j][2];
        red[warp][8 * j + 2 * t + 1][16 * i + 8 + g] = acc[i][j][3];
      }
    __syncthreads();
    for (int m = warp; m < 8 * NT; m += WARPS) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += red[w][m][lane];
      if (m0 + m < r1 && n0 + lane < p.N) p.y[static_cast<int64_t>(m0 + m) * p.N + n0 + lane] = __float2bfloat16_rn(s);
    }
    __syncthreads();
  }
}

template <int NT, int WARPS, bool AHEAD, int CTAS>
int launch_typed(const Fp8SmallParams& p, const Fp8Args& a, const char** msg) {
  const dim3 grid(static_cast<unsigned>((a.N + kColsS - 1) / kColsS), static_cast<unsigned>(a.E));
  fp8_smallm_kernel<NT, WARPS, AHEAD, CTAS><<<grid, WARPS * 32, 0, a.stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

}  // namespace

// Dense, up to 16 rows: one pass over W.  Up to 32: two, the second from L2, while W is small
// enough to stay there beside what else runs (4096 x 4096, 32 rows: 11.2 us against 13.4 of the
// tensor-core kernel; 14336 x 5120: 36.8 against 24.9).  Per expert: up to 64 rows and
// one an expert on average (64 experts of 2816 x 2048: 64 skewed rows 30.7 us against 39.4, 64
// even ones 40.6 against 42.9; of 2048 x 2048: 28.9 against 28.8 and 47.2 against 51.2; but 128
// skewed rows 45.7 against 32.8, and 256 on 256 experts 73 against 65), up to 32 rows two (16
// experts of 4096 x 4096, 32 rows: 36.6 against 47.1).  An expert's rows past the eighth cost a
// pass over its W each eight: were all 64 rows one expert's, 38.5 us against 14.0, which
// routing to more than one expert a token does not do.  32-bit offsets within 32 rows bound K.
bool fp8_takes_smallm(const Fp8Args& a) {
  if (a.dgrad || a.K > (1 << 26)) return false;
  if (a.offsets) return a.S <= 32 ? a.S <= 2 * a.E : a.S <= 64 && a.S <= a.E;
  return a.S <= 16 || (a.S <= 32 && a.N * a.K <= (1 << 25));
}

int launch_fp8_smallm(const Fp8Args& a, const char** msg) {
  Fp8SmallParams p;
  p.x = static_cast<const uint8_t*>(a.x);
  p.xs = a.x_scale;
  p.w = static_cast<const uint8_t*>(a.w);
  p.ws = a.w_scale;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.offsets = a.offsets;
  p.err = a.err;
  p.S = static_cast<int32_t>(a.S);
  p.N = static_cast<int32_t>(a.N);
  p.K = static_cast<int32_t>(a.K);
  p.E = static_cast<int32_t>(a.E);
  p.kblocks = static_cast<int32_t>((a.K + 127) / 128);
  // With CTAs enough to fill every SM several times over, small CTAs side by side keep more bytes
  // in flight than one that loads ahead, and one's reduction hides behind another's loads
  // (14336 x 5120, 8 rows: 15.2 us against 19.5).  With fewer, one CTA of 16 warps an SM (4096
  // x 4096: 5.8 us for 8 rows, 7.2 for 16).  An expert here rarely has more than 8 rows.  Warps
  // that would have two or three blocks of a short contraction each spend more on the
  // reduction than on loads: half as many, six CTAs an SM, if there are CTAs for it (64 experts
  // of 2816 x 2048: 64 skewed rows 30.7 us against 35.0, 64 even ones 40.6 against 45.5; of
  // 7168 x 1024: 50.8 against 65.7; but of 2048 x 4096: 60.8 against 57.8; 448 CTAs of a dense
  // 14336 x 5120: 18.2 against 14.7).
  const int64_t ctas = (a.N + kColsS - 1) / kColsS * (a.offsets ? a.E : 1);
  const bool many = a.offsets || ctas >= 2 * a.num_sms;
  if (a.offsets || a.S <= 8) {
    if (p.kblocks <= 24 && ctas >= 5 * a.num_sms) return launch_typed<1, 4, false, 6>(p, a, msg);
    return many ? launch_typed<1, 8, false, 3>(p, a, msg) : launch_typed<1, 16, true, 1>(p, a, msg);
  }
  return many ? launch_typed<2, 8, false, 2>(p, a, msg) : launch_typed<2, 16, false, 1>(p, a, msg);
}

}  // namespace bsq
