// bsq_fp4_smallm.cu -- products of a few BF16 token rows with 4-bit weights (decode), dense and
// per expert:  y[m, n] = sum_k x[m, k] deq(W)[n, k],  deq = RNE_bf16(code * RNE_bf16(scale)).
//
// No unit is at its limit: with one or two rows an expert issue is at 0.64, the pipe of masks, permutes and shifts
// at 0.60, HBM at 0.48 of its peak.  Most of the instructions decode W: 99 in all for 1024 MXFP4 codes
// of a warp with 8 tokens, 126 for NVFP4 with 16.  A CTA owns some rows of W (columns of y) and the
// whole contraction; RW warps beside one another in N and KW in k, whose groups take steps of
// 256 k in turn, each with a ring of steps in shared memory that asynchronous copies fill.  256 k
// are 128 bytes of a row: copies of whole cache lines, for which the load unit pays by the line
// (steps of 128 k and four bytes of scales a row and step took 4 us to ask for what a CTA holds;
// the scales come once for the whole tile now, as they lie in memory).
// The fragments of mma.m16n8k16 come from those rows without a permutation: the order of k inside
// a step is free as long as both operands share it, so a thread takes 16 bytes (32 codes) of a row,
// whose 8-code words decode to the pairs (c0, c4), (c1, c5), ... (bsq_decode.cuh), and the tokens'
// values are brought to that order.  Chunks of 16 bytes lie exchanged within their line, by
// the row, so that a fragment's reads fall in different banks.  CTAs begin at different steps:
// when all asked for the same tokens' values at once, that held them up (14336 x 5120, 8 rows: 24
// us against 19 at the time).  The groups' accumulators are added in their order through
// shared memory, so results do not depend on timing.
//
// Measured (a graph of calls on rotated weights beyond L2): 4096 x 4096 MXFP4, one row 5.8 us; 14336 x 5120 NVFP4,
// 1 / 8 / 16 / 32 / 64 rows 13.8 / 13.9 / 17.0 / 22.3 / 39.6 us (MXFP4 12.9 / 13.4 / 15.5 / 21.5 / 38.3); 64 rows
// by 128 MXFP4 experts of 2048 x 7168 82.5 us, 3.7 TB/s; 509 by 64 NVFP4 experts of 2816 x 2048 76.6 us; 64 by 128
// MXFP4 experts of 2880 x 2880, whose scales do not come in whole copies, 58.7 us (2816 x 2816: 54.9, 2 % less a byte).
// Of those 14336 x 5120 a warp spends its time so: 1.7 us to the first copies' end of asking, 1.5
// until the first step is there, then the instructions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bsq_decode.cuh"
#include "bsq_internal.h"
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

// Bytes from global to shared memory without a register, past L1 where they are 16; zeros if not `there`.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src, bool there) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
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
  static __device__ __forceinline__ uint32_t plain(uint32_t bytes, int, float) { return make_scale_e8m0(bytes & 0xFFu).s2; }
};
template <>
struct Scales<BSQ_NVFP4> {
  static constexpr int kCount = 2;
  static constexpr uint32_t kOne = 0;
  uint32_t c[2];
  // A tensor scale for which no scale times 2^126 is infinite and every scale is zero, a NaN or a normal
  // number: the product and its rounding may then take the 2^126 with them (64 experts of
  // 2816 x 2048, 512 rows: 79.7 us against 81.4; 14336 x 5120, 13 rows: 17.5 against 17.8).
  static __device__ __forceinline__ bool ordinary(float ts) { return fabsf(ts) <= 0x1p-7f && fabsf(ts) >= 0x1p-110f; }
  __device__ __forceinline__ void set_ordinary(uint32_t bytes, float ts) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(bytes)));
    const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    const float t = ts * 0x1p126f;
    c[0] = pack_bf16x2(__float_as_uint(__fmul_rn(s.x, t)), __float_as_uint(__fmul_rn(s.x, t)));
    c[1] = pack_bf16x2(__float_as_uint(__fmul_rn(s.y, t)), __float_as_uint(__fmul_rn(s.y, t)));
  }
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

// The warps that share a k: RW of them, one after the other in the CTA.
template <int RW>
__device__ __forceinline__ void group_sync(int group) {
  if (RW == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(RW * 32) : "memory");
}

constexpr int kStepK = 256;             // k of a step: 128 bytes of a row of W, a whole cache line
constexpr int kRoutedWords = kMaxExperts / 32;
// Dynamic shared memory a CTA can ask for: what the kernel declares itself counts against the same 227 KB.
constexpr int kMaxSmem = 227 * 1024 - kRoutedWords * 4;

// MT: 16-row groups of W a warp; RW: warps beside one another in N; KW: in k; NT: groups of 8 tokens
// per pass over W; STAGES: steps in flight; CTAS an SM shall hold.  ALIGNED: K % 256 == 0 and
// scales to match, which are then copied once for the whole tile.
template <int FMT, int MT, int RW, int KW, int NT, int STAGES, int CTAS, bool ALIGNED>
__global__ void __launch_bounds__(RW * KW * 32, CTAS) fp4_smallm_kernel(const Fp4SmallParams p) {
  constexpr int kThreads = RW * KW * 32;
  constexpr int kWarpRows = 16 * MT, kRows = kWarpRows * RW, kPad = kRows + 4;   // the pitch keeps fragment writes free of bank conflicts
  constexpr int kCount = Scales<FMT>::kCount;
  constexpr int kShift = FMT == BSQ_NVFP4 ? 4 : 5;   // log2 of the elements of a scale
  constexpr int kX = kRows * 128, kStage = kX + NT * 8 * 512;   // a group's step: rows of W, tokens
  extern __shared__ __align__(128) uint8_t smem[];   // [KW][STAGES][kStage], the tile's scales; the partial sums in the place of the first
  float (*red)[8][kPad] = reinterpret_cast<float (*)[8][kPad]>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = warp / RW, rw = warp % RW;
  const int g = lane >> 2, t = lane & 3;
  int e = static_cast<int>(blockIdx.y), r0 = 0, r1 = p.S;
  if (p.offsets) {
    r0 = e > 0 ? __ldg(p.offsets + e - 1) : 0;
    r1 = __ldg(p.offsets + e);
    // With fewer rows than experts blockIdx.y counts the experts that have any, so that few CTAs find
    // nothing to do (8 rows on 512 experts of 2816 x 2048: 11 us against 29).
    const bool sparse = gridDim.y < static_cast<unsigned>(p.E);
    __shared__ uint32_t routed[kRoutedWords];
    bool bad = false;
    for (int i0 = 0; i0 < p.E; i0 += kThreads) {
      const int i = i0 + tid;
      const int a = i > 0 && i < p.E ? __ldg(p.offsets + i - 1) : 0, b = i < p.E ? __ldg(p.offsets + i) : a;
      bad |= i < p.E && (a < 0 || b < a || b > p.S);
      if (sparse) {
        const uint32_t votes = __ballot_sync(kFull, b > a);
        if (lane == 0 && i < p.E) routed[i >> 5] = votes;
      }
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicCAS(p.err, 0, BSQ_DEVERR_BAD_OFFSETS);
    if (bad) return;
    if (sparse) {
      int skip = e, word = 0;
      const int words = (p.E + 31) >> 5;
      while (word < words && skip >= __popc(routed[word])) skip -= __popc(routed[word++]);
      if (word == words) return;          // fewer experts have rows
      uint32_t votes = routed[word];
      for (; skip > 0; --skip) votes &= votes - 1;
      e = 32 * word + __ffs(votes) - 1;
      r0 = e > 0 ? __ldg(p.offsets + e - 1) : 0;
      r1 = __ldg(p.offsets + e);
    }
    if (r0 == r1) return;
  }
  const int n0 = blockIdx.x * kRows;
  // Rows past N: any row, not stored.  Offsets of a CTA's rows fit 32 bits (K <= 2^24).
  const int rows_left = p.N - 1 - n0;
  const int64_t row0 = static_cast<int64_t>(e) * p.N + n0;
  const uint32_t wpitch = static_cast<uint32_t>(p.K) >> 1, spitch = static_cast<uint32_t>(p.K) >> kShift;
  const uint32_t tpitch = spitch + 16;               // of the scales in shared memory: rows fall in different banks
  const uint8_t* sbase = p.ws + row0 * spitch;
  const float ts = FMT == BSQ_NVFP4 ? __ldg(p.ts + e) : 0.f;
  bool ordinary = false;
  if constexpr (FMT == BSQ_NVFP4) ordinary = Scales<FMT>::ordinary(ts);
  uint8_t* tile = smem + KW * STAGES * kStage;
  const uint32_t ring = smem_u32(smem) + group * (STAGES * kStage);
  const uint8_t* ring_ptr = smem + group * (STAGES * kStage);
  const int steps = (p.K + kStepK - 1) / kStepK;
  // CTAs begin at different steps, so that they do not all ask for the same tokens' values at once
  const int turned = static_cast<int>(blockIdx.x * 5u) % steps;

  // W is copied by the warp whose rows they are, eight lanes a row of a step, to the place of its
  // chunk under the rows' exchange of chunks; the tokens' by all warps of the group.
  const int wl = lane >> 3, wc = lane & 7;
  const uint8_t* wsrc = p.w + row0 * wpitch + 16 * wc;
  const uint32_t wdst = static_cast<uint32_t>(rw * kWarpRows + wl) * 128;

  for (int m0 = r0; m0 < r1; m0 += 8 * NT) {
    const int left = min(r1 - m0, 8 * NT);
    const __nv_bfloat16* xsrc = p.x + static_cast<int64_t>(m0) * p.K + 8 * lane;
    const auto fetch = [&](int turn, int slot) {
      if (turn < steps) {
        const int step = turn + turned < steps ? turn + turned : turn + turned - steps;
        const uint32_t to = ring + slot * kStage;
        const bool win = ALIGNED || kStepK * step + 32 * wc < p.K, xin = ALIGNED || kStepK * step + 8 * lane < p.K;
#pragma unroll
        for (int j = 0; j < 4 * MT; ++j) {
          const int r = rw * kWarpRows + 4 * j + wl;
          copy_async<16>(to + wdst + j * 512 + ((wc ^ (r & 7)) << 4), win ? wsrc + (static_cast<uint32_t>(min(r, rows_left)) * wpitch + 128u * step) : p.w, win);
        }
        for (int m = rw; m < left; m += RW)
          copy_async<16>(to + kX + m * 512 + (lane >> 3) * 128 + (((lane & 7) ^ (2 * (lane >> 3) + (m & 1))) << 4),
                         reinterpret_cast<const uint8_t*>(xin ? xsrc + (static_cast<int64_t>(m) * p.K + kStepK * step) : p.x), xin);
      }
      copy_commit();
    };
    if (ALIGNED && m0 == r0) {
      // the tile's scales, in pieces of 16 or 8 bytes; a power of two of lanes a row
      const int size = spitch & 15u ? 8 : 16, pieces = static_cast<int>(spitch) / size;
      const int shift = pieces <= 4 ? 2 : pieces <= 8 ? 3 : pieces <= 16 ? 4 : 5;
      for (int r = tid >> shift; r < kRows; r += kThreads >> shift) {
        const uint8_t* src = sbase + static_cast<uint32_t>(min(r, rows_left)) * spitch;
        const uint32_t dst = smem_u32(tile) + r * tpitch;
        for (int i = tid & ((1 << shift) - 1); i < pieces; i += 1 << shift) {
          if (size == 16) copy_async<16>(dst + 16 * i, src + 16 * i, true);
          else copy_async<8>(dst + 8 * i, src + 8 * i, true);
        }
      }
      copy_commit();
    }
#pragma unroll
    for (int s = 0; s < STAGES; ++s) fetch(group + s * KW, s);
    if (ALIGNED && m0 == r0) {
      copy_wait<STAGES>();
      __syncthreads();
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = 0.f;

    // Thread (g, t) takes the chunks 2 t and 2 t + 1 of a row: k = 64 t + 32 h of the step.
    const uint32_t wat = static_cast<uint32_t>(rw * kWarpRows + g) * 128 + (((2 * t) ^ g) << 4);
    uint32_t xat[NT];          // columns past the last token: any token, not stored
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int m = min(8 * j + g, left - 1);
      xat[j] = kX + m * 512 + t * 128 + ((2 * t + (m & 1)) << 4);
    }
    int slot = 0;
#pragma unroll 1
    for (int turn = group; turn < steps; turn += KW) {
      const int step = turn + turned < steps ? turn + turned : turn + turned - steps;
      // the scales of both halves: byte (or pair) 2 t, 2 t + 1 of the row's
      uint32_t sv[MT][2];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        uint32_t& v = sv[i >> 1][i & 1];
        const int r = rw * kWarpRows + 8 * i + g;
        const uint32_t at = static_cast<uint32_t>(8 * step + 2 * t) * kCount;
        if (ALIGNED) {
          const uint8_t* s = tile + r * tpitch + at;
          v = FMT == BSQ_NVFP4 ? *reinterpret_cast<const uint32_t*>(s) : *reinterpret_cast<const uint16_t*>(s);
        } else {
          const uint8_t* s = sbase + (static_cast<uint32_t>(min(r, rows_left)) * spitch + at);
          v = Scales<FMT>::kOne * 0x01010101u;
#pragma unroll
          for (int b = 0; b < 2 * kCount; ++b)
            if (at + b < spitch) v = (v & ~(0xFFu << (8 * b))) | (static_cast<uint32_t>(__ldg(s + b)) << (8 * b));
        }
      }
      copy_wait<STAGES - 1>();
      group_sync<RW>(group);         // what other lanes and warps copied is there
      const uint8_t* from = ring_ptr + slot * kStage;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Scales<FMT> f[MT][2];
        // codes that are not there stay zeros when the tensor's scale is infinite
        const float tsh = ALIGNED || kStepK * step + 64 * t + 32 * h < p.K ? ts : 0.f;
        const auto scale_bytes = [&](int i) { return sv[i >> 1][i & 1] >> (8 * kCount * h) & (kCount == 2 ? 0xFFFFu : 0xFFu); };
        bool slow = false;
        if constexpr (FMT == BSQ_NVFP4) {
          if (ordinary) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) f[i >> 1][i & 1].set_ordinary(scale_bytes(i), tsh);
          }
        }
        if (!ordinary) {
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) slow |= f[i >> 1][i & 1].set(scale_bytes(i), tsh);
          slow = __any_sync(kFull, slow);
        }
        uint4 wv[MT][2];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) wv[i >> 1][i & 1] = *reinterpret_cast<const uint4*>(from + ((wat ^ (h << 4)) + i * 1024));
        const auto multiply = [&](auto is_slow) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t xp[NT][4];      // in the order of the decoded pairs
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint4 v = *reinterpret_cast<const uint4*>(from + (xat[j] ^ ((4 * h + c) << 4)));
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
                  const uint32_t plain = Scales<FMT>::plain(sv[i][q] >> (8 * kCount * h), s, tsh);
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
      }
      group_sync<RW>(group);         // every lane has read the step
      fetch(turn + STAGES * KW, slot);
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    copy_wait<0>();
    __syncthreads();     // the partial sums take the place of what every warp has read
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (8 * j >= left) break;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int n = rw * kWarpRows + 16 * i + g;
        red[group][2 * t][n] = acc[i][j][0];
        red[group][2 * t + 1][n] = acc[i][j][1];
        red[group][2 * t][n + 8] = acc[i][j][2];
        red[group][2 * t + 1][n + 8] = acc[i][j][3];
      }
      __syncthreads();
      for (int o = tid; o < 8 * kRows; o += kThreads) {
        const int m = o / kRows, n = o % kRows;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) s += red[w][m][n];
        if (8 * j + m < left && n <= rows_left) p.y[static_cast<int64_t>(m0 + 8 * j + m) * p.N + n0 + n] = __float2bfloat16_rn(s);
      }
      __syncthreads();
    }
  }
}

template <int FMT, int MT, int RW, int KW, int NT, int STAGES, int CTAS>
int launch_typed(const Fp4SmallParams& p, const Fp4Args& a, const char** msg) {
  constexpr int kRows = 16 * MT * RW;
  const dim3 grid(static_cast<unsigned>((a.N + kRows - 1) / kRows), static_cast<unsigned>(a.offsets ? (a.S < a.E ? a.S : a.E) : 1));
  constexpr int kRing = KW * STAGES * (kRows * 128 + NT * 8 * 512), kRed = KW * 8 * (kRows + 4) * 4;
  static_assert(kRed <= kRing && kRing <= kMaxSmem, "shared memory");
  const int64_t spitch = a.K / (FMT == BSQ_NVFP4 ? 16 : 32);
  const int64_t with = kRing + kRows * (spitch + 16);
  const bool aligned = a.K % kStepK == 0 && (reinterpret_cast<uintptr_t>(a.w_scale) & (spitch % 16 ? 7u : 15u)) == 0 && with <= kMaxSmem;
  const int smem = aligned ? static_cast<int>(with) : kRing;
  const auto kernel = aligned ? fp4_smallm_kernel<FMT, MT, RW, KW, NT, STAGES, CTAS, true> : fp4_smallm_kernel<FMT, MT, RW, KW, NT, STAGES, CTAS, false>;
  // The limit is the function's, for all host threads: always the largest, so that no call lowers it
  // between another's setting and its launch.
  cudaError_t e = cudaSuccess;
  if (smem > 47 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess) {
    kernel<<<grid, RW * KW * 32, smem, a.stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *msg = cudaGetErrorString(e);
    return static_cast<int>(e);
  }
  return 0;
}

// The tile and the tokens of a pass by the number of rows; every limit with both sides measured, in
// us.  Per expert the limits are on the average, since the counts are the device's:
//   (rows on experts of falling popularity, r^-0.7; tokens a pass are 8, 16 or 32, 16 in tiles of 64 or 48 rows of W)
//   64 experts of 2816 x 2048 NVFP4   320 rows 68.3 with 8, 67.5 and 69.7 with 16; 384: 75.0, 69.3 and 72.1; 512: 87.8, 76.4 and
//                                     78.6; 1024: 101.7 and 98.2 with 16, 118 with 32; 2048: 173 and 162 with 16, 152 with 32
//   32 experts of 2048 x 7168 MXFP4   160 rows 78.4 with 8, 85.2 and 78.3 with 16; 384: 129, 105 and 99.5
//   128 experts of 2880 x 2880 MXFP4  64 rows 58.7 with 8, 61.6 and 63.8 with 16; 640: 201, 193 and 195
//   (128 experts of 1024 x 2048 would take 16 from 4 rows an expert: MXFP4 640 rows 66.9 with 8, 58.4 and 57.6 with 16)
// Dense, tiles of 32 rows while that gives an SM one at most: 4096 x 4096 MXFP4, 32 rows 8.8 with 32
// tokens a pass, 10.2 with 16; then 14336 x 5120 NVFP4, 8 rows 13.9 in 32-row tiles, 14.6 in
// 96-row ones; 13 rows 22.2 in 32-row tiles, 17.1 in 96-row ones; 32 rows 22.2 in 48-row tiles, 24.4 in 96-row ones.
// Of the registers 24 bytes a thread go to local memory in the 64-row tiles (16 MXFP4 and 32 NVFP4 where the scales stay in
// global memory), 24 MXFP4 and 20 NVFP4 in the 96-row ones, up to 24 in NVFP4's 48-row ones.
template <int FMT>
int launch_fmt(const Fp4SmallParams& p, const Fp4Args& a, const char** msg) {
  if (a.offsets) {
    if (a.S <= 5 * a.E) return launch_typed<FMT, 3, 1, 4, 1, 1, 3>(p, a, msg);
    if (a.S <= 8 * a.E) return launch_typed<FMT, 4, 1, 4, 2, 1, 3>(p, a, msg);
    return a.S <= 16 * a.E ? launch_typed<FMT, 3, 1, 4, 2, 1, 3>(p, a, msg) : launch_typed<FMT, 3, 1, 4, 4, 1, 2>(p, a, msg);
  }
  if (a.N <= 32 * a.num_sms) {
    if (a.S <= 8) return launch_typed<FMT, 2, 1, 8, 1, 2, 1>(p, a, msg);
    return a.S <= 16 ? launch_typed<FMT, 2, 1, 8, 2, 2, 1>(p, a, msg) : launch_typed<FMT, 2, 1, 8, 4, 1, 1>(p, a, msg);
  }
  if (a.S <= 8) return launch_typed<FMT, 2, 1, 4, 1, 2, 3>(p, a, msg);
  return a.S <= 16 ? launch_typed<FMT, 2, 3, 4, 2, 2, 1>(p, a, msg) : launch_typed<FMT, 3, 1, 4, 4, 1, 2>(p, a, msg);
}

}  // namespace

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
