// bsq_fp4_smallm.cu -- products of a few BF16 token rows with 4-bit weights (decode), dense and
// per expert:  y[m, n] = sum_k x[m, k] deq(W)[n, k],  deq = RNE_bf16(code * RNE_bf16(scale)).
//
// Bound by the instructions that decode W (about 100 for 1024 codes of a warp, where the codes and
// their scales are half a byte each), and for few columns by latency.  A CTA owns 16 MT columns of
// y (rows of W) and the whole contraction; its warps take steps of 128 k in turn, each with a
// ring of its own in shared memory that asynchronous copies fill some steps ahead.  A thread copies
// 16 bytes (32 codes) of a row and reads them back as register fragments of mma.m16n8k16: the
// order of k inside a step is free as long as both operands share it, so the 8-code words decode
// to the pairs (c0, c4), (c1, c5), ... without a permutation (bsq_decode.cuh), and the tokens'
// values are brought to that order instead, once for all rows of W.  CTAs begin at different
// steps: when all asked for the same tokens' values at once, the cache line's slice held them up
// (14336 x 5120, 8 rows: 24 us against 19).  The warps' accumulators are added in warp order
// through shared memory, so results do not depend on timing.
//
// Measured (graph of calls on rotated weights): 4096 x 4096 MXFP4, one row 5.7 us; 14336 x 5120 NVFP4,
// 1 / 8 / 16 rows 17 / 19 / 23 us; 64 rows by 128 MXFP4 experts of 2048 x 7168 83 us, 3.7 TB/s.
// Without the multiplication those 14336 x 5120 take 12 us, without the loads 11.
#include <cuda_bf16.h>

#include "bsq_decode.cuh"
#include "bsq_moe_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

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

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// 16 bytes from global to shared memory, past L1 and without a register; a group per step.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The scales of a thread's 32 codes of one row, from their bytes: BF16 pairs (s, s) * 2^126, the
// factor of spread_e2m1x8's pairs, when that is finite; else `slow` is set, and the pairs are
// multiplied by 2^126 and by (s, s) one after the other (the same result, see bsq_decode.cuh).
template <int FMT>
struct Scales;
template <>
struct Scales<BSQ_MXFP4> {
  static constexpr int kCount = 1;
  static constexpr uint32_t kOne = 127;      // a scale of 1, for codes that are not there
  uint32_t c[1];
  __device__ __forceinline__ bool set(uint32_t bytes, float) {
    c[0] = bytes * 0x00800080u + 126u * 0x00800080u;   // (b + 126) << 7 in both halves
    return bytes > 128u;
  }
  static __device__ __forceinline__ uint32_t plain(uint32_t bytes, int, float) { return make_scale_e8m0(bytes).s2; }
};
template <>
struct Scales<BSQ_NVFP4> {
  static constexpr int kCount = 2;
  static constexpr uint32_t kOne = 0;
  uint32_t c[2];
  __device__ __forceinline__ bool set(uint32_t bytes, float ts) {
    const uint32_t s2 = pack_bf16x2(__float_as_uint(__fmul_rn(e4m3_to_f32(bytes), ts)), __float_as_uint(__fmul_rn(e4m3_to_f32(bytes >> 8), ts)));
    const uint32_t c2 = bf16x2_mul(s2, kPow2_126x2);
    c[0] = prmt(c2, c2, 0x1010u);
    c[1] = prmt(c2, c2, 0x3232u);
    const uint32_t m = c2 & 0x7FFF7FFFu;
    return __vmaxu2(m, 0x7F7F7F7Fu) != 0x7F7F7F7Fu;    // an infinity or a NaN
  }
  static __device__ __forceinline__ uint32_t plain(uint32_t bytes, int i, float ts) { return make_scale_nvfp4(bytes >> (8 * i), ts).s2; }
};

// MT: 16-row groups of W a CTA; NT: groups of 8 tokens per pass over W; STAGES: steps of 128 k
// that a warp has in flight; WARPS of a CTA; CTAS an SM shall hold.  ALIGNED: K % 128 == 0 and
// aligned scales, which then come by copies of a row's bytes of a step.
template <int FMT, int MT, int NT, int STAGES, int WARPS, int CTAS, bool ALIGNED>
__global__ void __launch_bounds__(WARPS * 32, CTAS) fp4_smallm_kernel(const Fp4SmallParams p) {
  constexpr int kRows = 16 * MT, kPad = kRows + 4;   // the pitch keeps fragment writes free of bank conflicts
  constexpr int kCount = Scales<FMT>::kCount;
  constexpr int kShift = FMT == BSQ_NVFP4 ? 4 : 5;   // log2 of the elements of a scale
  // a warp's step in shared memory: W (read back by the thread that copied it), the tokens' values, the
  // rows' scales
  constexpr int kX = 2 * MT * 512, kS = kX + NT * 2048, kStage = kS + (kRows * 4 * kCount + 15) / 16 * 16;
  extern __shared__ __align__(16) uint8_t smem[];    // [WARPS][STAGES][kStage]; the partial sums in its place
  float (*red)[8][kPad] = reinterpret_cast<float (*)[8][kPad]>(smem);
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
  const uint32_t wpitch = static_cast<uint32_t>(p.K) >> 1, spitch = static_cast<uint32_t>(p.K) >> kShift;
  const uint8_t* wbase = p.w + row0 * wpitch + 16 * t;
  const uint8_t* sbase = p.ws + row0 * spitch;
  const float ts = FMT == BSQ_NVFP4 ? __ldg(p.ts + e) : 0.f;
  const uint8_t* ring = smem + warp * STAGES * kStage;
  const uint32_t ring_at = smem_u32(ring);
  const int steps = (p.K + 127) >> 7;
  // CTAs begin at different steps, so that they do not all ask for the same tokens' values at once
  const int turned = static_cast<int>(blockIdx.x * 5u) % steps;

  for (int m0 = r0; m0 < r1; m0 += 8 * NT) {
    const int left = r1 - m0;
    const __nv_bfloat16* xbase = p.x + static_cast<int64_t>(m0) * p.K;
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = 0.f;

    const auto fetch = [&](int turn, int slot) {
      const uint32_t to = ring_at + slot * kStage;
      if (turn < steps) {
        const int step = turn + turned < steps ? turn + turned : turn + turned - steps;
        if (ALIGNED || 128 * step + 32 * t < p.K) {     // K % 32 == 0: whole pieces of 32 codes
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i)
            copy_async<16>(to + i * 512 + lane * 16, wbase + (static_cast<uint32_t>(min(8 * i + g, rows_left)) * wpitch + 64u * step));
        }
        // sixteen lanes a token: one's 16 eights of the step, to where the lanes that need them read
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) {
          const int m = 2 * i + (lane >> 4), q = (lane >> 2) & 3, c = lane & 3;
          if (m < left && (ALIGNED || 128 * step + 32 * q < p.K))
            copy_async<16>(to + kX + ((m >> 3) * 4 + c) * 512 + ((m & 7) * 4 + q) * 16,
                           reinterpret_cast<const uint8_t*>(xbase + (static_cast<int64_t>(m) * p.K + 128 * step + 8 * (lane & 15))));
        }
        if (ALIGNED) {
#pragma unroll
          for (int i = 0; i < kRows; i += 32)
            if (i + lane < kRows)
              copy_async<4 * kCount>(to + kS + (i + lane) * 4 * kCount, sbase + (static_cast<uint32_t>(min(i + lane, rows_left)) * spitch + 4u * kCount * step));
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) fetch(warp + s * WARPS, s);
    int slot = 0;
#pragma unroll 1
    for (int turn = warp; turn < steps; turn += WARPS) {
      const int step = turn + turned < steps ? turn + turned : turn + turned - steps;
      const bool in = ALIGNED || 128 * step + 32 * t < p.K;
      const uint8_t* from = ring + slot * kStage;
      uint32_t sv[MT][2];
      if (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          const uint8_t* s = sbase + (static_cast<uint32_t>(min(8 * i + g, rows_left)) * spitch + kCount * (4 * step + t));
          sv[i >> 1][i & 1] = Scales<FMT>::kOne;
          if (in) sv[i >> 1][i & 1] = FMT == BSQ_NVFP4 ? __ldg(reinterpret_cast<const uint16_t*>(s)) : __ldg(s);
        }
      }
      copy_wait<STAGES - 2>();
      __syncwarp();          // tokens and scales were copied by other lanes
      if (ALIGNED) {
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          const uint8_t* s = from + kS + (8 * i + g) * 4 * kCount + kCount * t;
          sv[i >> 1][i & 1] = FMT == BSQ_NVFP4 ? *reinterpret_cast<const uint16_t*>(s) : *s;
        }
      }
      Scales<FMT> f[MT][2];
      bool slow = false;
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) slow |= f[i >> 1][i & 1].set(sv[i >> 1][i & 1], ts);
      slow = __any_sync(kFull, slow);
      uint4 wv[MT][2];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        wv[i >> 1][i & 1] = *reinterpret_cast<const uint4*>(from + i * 512 + lane * 16);
        if (!in) wv[i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
      }
      const auto multiply = [&](auto is_slow) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t xp[NT][4];      // in the order of the decoded pairs
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint4 v = *reinterpret_cast<const uint4*>(from + kX + (j * 4 + c) * 512 + lane * 16);
            if (!in) v = make_uint4(0, 0, 0, 0);
            unzip_pairs(v.x, v.z, xp[j][0], xp[j][1]);
            unzip_pairs(v.y, v.w, xp[j][2], xp[j][3]);
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t a[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              spread_e2m1x8(word(wv[i][q], c), a[q]);
              const int s = kCount == 2 ? c >> 1 : 0;
              if (decltype(is_slow)::value) {
                const uint32_t plain = Scales<FMT>::plain(sv[i][q], s, ts);
#pragma unroll
                for (int u = 0; u < 4; ++u) a[q][u] = bf16x2_mul(bf16x2_mul(a[q][u], kPow2_126x2), plain);
              } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) a[q][u] = bf16x2_mul(a[q][u], f[i][q].c[s]);
              }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma_bf16(acc[i][j], a[0][0], a[1][0], a[0][1], a[1][1], xp[j][0], xp[j][1]);
              mma_bf16(acc[i][j], a[0][2], a[1][2], a[0][3], a[1][3], xp[j][2], xp[j][3]);
            }
          }
        }
      };
      if (!slow) multiply(std::false_type{});
      else multiply(std::true_type{});
      __syncwarp();          // every lane has read the step before
      fetch(turn + (STAGES - 1) * WARPS, slot == 0 ? STAGES - 1 : slot - 1);
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    copy_wait<0>();
    __syncthreads();     // the partial sums take the place of what every warp has read
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

template <int FMT, int MT, int NT, int STAGES, int WARPS, int CTAS>
int launch_typed(const Fp4SmallParams& p, const Fp4Args& a, const char** msg) {
  const dim3 grid(static_cast<unsigned>((a.N + 16 * MT - 1) / (16 * MT)), static_cast<unsigned>(a.offsets ? a.E : 1));
  constexpr int kStage = 2 * MT * 512 + NT * 2048 + (16 * MT * 4 * Scales<FMT>::kCount + 15) / 16 * 16;
  constexpr int kRing = WARPS * STAGES * kStage, kRed = WARPS * 8 * (16 * MT + 4) * 4;
  constexpr int kSmem = kRing > kRed ? kRing : kRed;
  const bool aligned = a.K % 128 == 0 && (reinterpret_cast<uintptr_t>(a.w_scale) & 7u) == 0;
  const auto kernel = aligned ? fp4_smallm_kernel<FMT, MT, NT, STAGES, WARPS, CTAS, true> : fp4_smallm_kernel<FMT, MT, NT, STAGES, WARPS, CTAS, false>;
  cudaError_t e = cudaSuccess;
  if (kSmem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) {
    kernel<<<grid, WARPS * 32, kSmem, a.stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

template <int FMT>
int launch_fmt(const Fp4SmallParams& p, const Fp4Args& a, const char** msg) {
  if (a.offsets) {
    // an expert's rows on average: more than one pass over its W for the few that have more
    if (a.S <= 2 * a.E) return launch_typed<FMT, 4, 1, 3, 4, 2>(p, a, msg);
    return launch_typed<FMT, 4, 2, 2, 4, 2>(p, a, msg);
  }
  const bool narrow = a.N <= 32 * a.num_sms;
  if (a.S <= 8) return narrow ? launch_typed<FMT, 2, 1, 3, 8, 2>(p, a, msg) : launch_typed<FMT, 6, 1, 3, 8, 1>(p, a, msg);
  if (narrow && a.S > 16) return launch_typed<FMT, 2, 4, 2, 8, 1>(p, a, msg);
  return narrow ? launch_typed<FMT, 2, 2, 2, 8, 2>(p, a, msg) : launch_typed<FMT, 6, 2, 2, 8, 1>(p, a, msg);
}

}  // namespace

bool fp4_takes_smallm(const Fp4Args& a) { return a.S <= 16 || (a.S <= 64 && a.N <= 32 * a.num_sms); }

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
