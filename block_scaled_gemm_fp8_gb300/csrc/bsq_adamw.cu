// bsq_adamw.cu -- one AdamW step (decoupled weight decay, Loshchilov and Hutter 2019) over many
// tensors in one launch per 400 of them, FP32 parameters, states in 32 or in 8 bits:
//
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2        r = sqrt(v)
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (r / sqrt(1 - b2^t) + eps)
//
// 8-bit states hold m and r as E4M3 codes with one float32 scale per 128 elements of the
// tensor (a / 448, a the block's largest magnitude, the quantizer's rule).  With b2 near 1 a
// step moves r by less than half a code, and rounding to nearest would never move it; so
// the codes are rounded at random, up with the probability of the part cut off, from a
// hash of (seed, step, element): results repeat, and the states are right on average.  An
// r above zero keeps at least the smallest code above zero, so that a later step does not
// divide a remembered m by eps alone.
//
// Every operation of the states is rounded by itself (no contraction), so that the codes
// follow from the formula; the update's quotient, which no state sees, is within 2 ulp.
//
// Bound by HBM: 28 or 30 bytes per element with 32-bit states and a BF16 copy; 16.1 or 18.1
// with 8-bit ones, where the instructions of the rounding weigh as much.  A thread owns 8
// consecutive elements (32-byte accesses), 16 lanes a scale block, a CTA a chunk of one
// tensor, found by bisection in the launch's table.
#include <cmath>

#include <cuda_bf16.h>

#include "bsq_fp8_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

// Small CTAs with 8-bit states: an SM's place is refilled when two warps are done, not eight,
// which keeps loads in flight beside the rounding's instructions (146 M elements: 396 us; 413
// with 128 threads, 441 with 256, 402 with 32; with the instructions saved since, 382 us, 6.1
// TB/s).  With 32-bit states large tensors take 583 us with either, 300 small ones 29.4 us with
// 256 threads and 30.4 with 64, whose CTAs look up their tensor more often.
template <bool S8>
constexpr int kThreadsA = S8 ? 64 : 256;
template <bool S8>
constexpr int kStepA = kThreadsA<S8> * 8;      // elements of one sweep of a CTA
// Sweeps of a CTA: with 8-bit states, enough to pay for finding its tensor (384 us on the
// device; 388 of six sweeps, 383 of twelve); with 32-bit ones, where instructions do not count,
// one (300 small tensors: 29.4 us against 37.3 of two).
template <bool S8>
constexpr int kSweeps = S8 ? 8 : 1;
// Tensors of one launch: the table travels as a kernel parameter, so there are a small one
// (2.4 KB) and the largest that fits the 32764 bytes of parameters.
constexpr int kFewA = 32, kManyA = 400;

struct AdamwEntry {
  float* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  __nv_bfloat16* copy;
  int64_t n;
  float decay;           // 1 - lr * weight_decay
  uint32_t counter;      // of the tensor's first element
  int32_t chunk0;        // chunks of the tensors before it
  int32_t wide;          // every pointer allows the vector accesses
};

template <int N>
struct AdamwTable {
  AdamwEntry e[N];
  int32_t count;
  float b1, c1m, b2, c2m;   // betas and 1 - betas
  float lr1, rc2, eps;      // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float one;
  uint32_t salt;            // seed and step
  const float* grad_scale;
};
static_assert(sizeof(AdamwTable<kManyA>) <= 32764, "kernel parameter space");

__device__ __forceinline__ void ld8(const float* p, float (&x)[8]) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}
__device__ __forceinline__ void st8(float* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
               "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two E4M3 codes (low 16 bits) as floats: exact.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Products and sums of two floats an instruction, each rounded by itself.  A packed product
// and the packed sum it goes to are fused by the assembler, rounding modes notwithstanding;
// so the sum is a fused multiply-add itself, by a one that only the host knows.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b, float one) { return __ffma2_rn(a, make_float2(one, one), b); }

// 1 / x within 1 ulp; an x below 2^-126 counts as zero.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 32 random bits of an element: a Weyl step and MurmurHash3's finalizer (Appleby).
__device__ __forceinline__ uint32_t element_bits(uint32_t i, uint32_t salt) {
  uint32_t x = i * 0x9E3779B1u + salt;
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

// E4M3 value next to a, away from zero with the probability of the part cut off: 16 random bits
// against the mantissa bits below E4M3's three.  For magnitudes from 2^-6 to 448 and a little
// above; what comes out above 448 the conversion takes back to it.
__device__ __forceinline__ float round_normal(float a, uint32_t bits) {
  return __uint_as_float((__float_as_uint(a) + (bits << 4)) & 0xFFF00000u);
}
// The same for every a >= 0 (NaN stays): below 2^-6, against the part below the subnormal
// step of 2^-9.  x + 2^23 rounded down, less 2^23, is the floor of an x below 2^22.
__device__ __forceinline__ float round_any(float a, uint32_t bits) {
  if (a >= 0.015625f) return round_normal(a, bits);
  const float u = __uint_as_float(0x43000000u | bits) - 128.f;   // bits / 65536
  const float x = __fadd_rn(__fmul_rn(a, 512.f), u);
  return __fmul_rn(__fadd_rd(x, 8388608.f) - 8388608.f, 1.953125e-3f);
}

__device__ __forceinline__ float block_amax(float a) {
  return a == 0.f ? 448.f : a < 7.888609052210118e-31f ? 7.888609052210118e-31f : a;   // 2^-100; NaN stays
}

// Largest and smallest of three; the largest is NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Scale block of 16 lanes x 8 values: the block's a from each lane's largest magnitude (bit
// patterns between lanes: NaN is above infinity).
__device__ __forceinline__ float lane16_amax(const float (&x)[8]) {
  float f = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) f = max3_nan(f, fabsf(x[i]), fabsf(x[i + 1]));
  uint32_t m = __float_as_uint(f);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return block_amax(__uint_as_float(m));
}

template <bool G16, bool S8, int N>
__global__ void __launch_bounds__(kThreadsA<S8>, 1024 / kThreadsA<S8>) adamw_kernel(const __grid_constant__ AdamwTable<N> t) {
  int lo = 0, hi = t.count - 1;
  const int chunk = blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  const AdamwEntry& e = t.e[lo];
  const float gs = t.grad_scale ? __ldg(t.grad_scale) : 1.f;
  const int64_t first = static_cast<int64_t>(chunk - e.chunk0) * (kSweeps<S8> * kStepA<S8>) + threadIdx.x * 8;
#pragma unroll 1
  for (int sweep = 0; sweep < kSweeps<S8>; ++sweep) {
    const int64_t i0 = first + sweep * kStepA<S8>;
    const int64_t left = e.n - i0;
    const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;   // elements of this thread
    const bool wide = e.wide && n == 8;
    if (!S8 && n == 0) return;
    // as stored; an operand in fewer bits stays packed until its pair is used
    float g[8], p[8], m[8], v[8];
    uint32_t gw[4] = {}, mw[2] = {}, vw[2] = {};
    float ms = 0.f, vs = 0.f;
    if (S8 && n > 0) {
      ms = e.ms[i0 >> 7];
      vs = e.vs[i0 >> 7];
    }
    if (wide) {
      ld8(e.p + i0, p);
      if (G16) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.g) + i0));
        gw[0] = w.x, gw[1] = w.y, gw[2] = w.z, gw[3] = w.w;
      } else {
        ld8(static_cast<const float*>(e.g) + i0, g);
      }
      if (S8) {
        const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(e.m) + i0);
        const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(e.v) + i0);
        mw[0] = cm.x, mw[1] = cm.y;
        vw[0] = cv.x, vw[1] = cv.y;
      } else {
        ld8(static_cast<const float*>(e.m) + i0, m);
        ld8(static_cast<const float*>(e.v) + i0, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = g[j] = m[j] = v[j] = 0.f;
        if (j < n) {
          p[j] = e.p[i0 + j];
          if (G16) gw[j / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(e.g)[i0 + j]) << (16 * (j & 1));
          else g[j] = static_cast<const float*>(e.g)[i0 + j];
          if (S8) {
            mw[j / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(e.m)[i0 + j]) << (8 * (j & 3));
            vw[j / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(e.v)[i0 + j]) << (8 * (j & 3));
          } else {
            m[j] = static_cast<const float*>(e.m)[i0 + j];
            v[j] = static_cast<const float*>(e.v)[i0 + j];
          }
        }
      }
    }
    float r[8];
    // two elements an instruction: each operation still rounded by itself
    auto two = [](float x) { return make_float2(x, x); };
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 gj = make_float2(g[j], g[j + 1]), mj = make_float2(m[j], m[j + 1]), vj = make_float2(v[j], v[j + 1]);
      if (G16) gj = make_float2(__uint_as_float(gw[j / 2] << 16), __uint_as_float(gw[j / 2] & 0xFFFF0000u));
      gj = mul2(gj, two(gs));
      if (S8) {
        mj = mul2(from_e4m3x2(mw[j / 4] >> (8 * (j & 3)) & 0xFFFFu), two(ms));
        vj = mul2(from_e4m3x2(vw[j / 4] >> (8 * (j & 3)) & 0xFFFFu), two(vs));
        vj = mul2(vj, vj);
      }
      mj = add2(mul2(mj, two(t.b1)), mul2(gj, two(t.c1m)), t.one);
      vj = add2(mul2(vj, two(t.b2)), mul2(mul2(gj, gj), two(t.c2m)), t.one);
      const float2 rj = make_float2(__fsqrt_rn(vj.x), __fsqrt_rn(vj.y));
      const float2 den = add2(mul2(rj, two(t.rc2)), two(t.eps), t.one);
      const float2 u = mul2(mul2(mj, two(t.lr1)), make_float2(reciprocal(den.x), reciprocal(den.y)));
      const float2 pj = add2(mul2(make_float2(p[j], p[j + 1]), two(e.decay)), make_float2(-u.x, -u.y), t.one);
      p[j] = pj.x, p[j + 1] = pj.y;
      m[j] = mj.x, m[j + 1] = mj.y;
      v[j] = vj.x, v[j + 1] = vj.y;
      r[j] = rj.x, r[j + 1] = rj.y;
    }
    // the parameters are stored before the states are rounded, which wants their registers
    if (wide) {
      st8(e.p + i0, p);
      if (e.copy) {
        uint4 w;
        w.x = bf16x2(p[0], p[1]);
        w.y = bf16x2(p[2], p[3]);
        w.z = bf16x2(p[4], p[5]);
        w.w = bf16x2(p[6], p[7]);
        *reinterpret_cast<uint4*>(e.copy + i0) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          e.p[i0 + j] = p[j];
          if (e.copy) e.copy[i0 + j] = __float2bfloat16_rn(p[j]);
        }
      }
    }
    if (S8 && n < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= n) m[j] = r[j] = 0.f;   // past the end: no part of the block's maximum
    }
    uint32_t cm[4], cv[4];   // codes, two a word
    if (S8) {
      // One division each for 448 / a and a / 448 of both states: m's by the lower half of the
      // block's 16 lanes, r's by the upper.
      const int lane = threadIdx.x & 31;
      const bool upper = (lane & 8) != 0;
      const float am = lane16_amax(m), ar = lane16_amax(r);
      const float a = upper ? ar : am;
      const float inv = __fdiv_rn(448.f, a);
      const float im = __shfl_sync(0xffffffffu, inv, lane & 16), ir = __shfl_sync(0xffffffffu, inv, (lane & 16) | 8);
      const float scale = __fdiv_rn(a, 448.f);
      // lane 0 of the block has its first element; lane 8 may be past the tensor's end
      const int64_t block = (i0 - (upper ? 64 : 0)) >> 7;
      if ((lane & 7) == 0 && (block << 7) < e.n) (upper ? e.vs : e.ms)[block] = scale;
      const uint32_t at = e.counter + static_cast<uint32_t>(i0);
      float least = 1.f;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 mj = mul2(make_float2(m[j], m[j + 1]), two(im)), rj = mul2(make_float2(r[j], r[j + 1]), two(ir));
        const uint32_t b0 = element_bits(at + j, t.salt), b1 = element_bits(at + j + 1, t.salt);
        m[j] = mj.x, m[j + 1] = mj.y;
        r[j] = rj.x, r[j + 1] = rj.y;
        least = min3(min3(least, fabsf(mj.x), rj.x), fabsf(mj.y), rj.y);
        cm[j / 2] = e4m3x2(round_normal(mj.x, b0 & 0xFFFFu), round_normal(mj.y, b1 & 0xFFFFu));
        cv[j / 2] = e4m3x2(round_normal(rj.x, b0 >> 16), round_normal(rj.y, b1 >> 16));
      }
      // Below 2^-6 (2^-15 of the block's largest: rare), or NaN, which only a NaN or infinite
      // scale of either state leaves (`least` passes over NaN): once more in full.
      if (!(least >= 0.015625f) || !(im > 0.f) || !(ir > 0.f)) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float qm[2], qr[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t bits = element_bits(at + j + h, t.salt);
            qm[h] = copysignf(round_any(fabsf(m[j + h]), bits & 0xFFFFu), m[j + h]);
            const float q = round_any(r[j + h], bits >> 16);
            qr[h] = r[j + h] > 0.f && q == 0.f ? 1.953125e-3f : q;
          }
          cm[j / 2] = e4m3x2(qm[0], qm[1]);
          cv[j / 2] = e4m3x2(qr[0], qr[1]);
        }
      }
    }
    if (wide) {
      if (S8) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.m) + i0) = make_uint2(cm[0] | (cm[1] << 16), cm[2] | (cm[3] << 16));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.v) + i0) = make_uint2(cv[0] | (cv[1] << 16), cv[2] | (cv[3] << 16));
      } else {
        st8(static_cast<float*>(e.m) + i0, m);
        st8(static_cast<float*>(e.v) + i0, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          if (S8) {
            static_cast<uint8_t*>(e.m)[i0 + j] = static_cast<uint8_t>(cm[j >> 1] >> (8 * (j & 1)));
            static_cast<uint8_t*>(e.v)[i0 + j] = static_cast<uint8_t>(cv[j >> 1] >> (8 * (j & 1)));
          } else {
            static_cast<float*>(e.m)[i0 + j] = m[j];
            static_cast<float*>(e.v)[i0 + j] = v[j];
          }
        }
      }
    }
  }
}

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <int N>
int launch_tables(const AdamwArgs& a, const char** msg) {
  const bsq_adamw_tensor* ts = static_cast<const bsq_adamw_tensor*>(a.tensors);
  const bool g16 = a.grad_dtype == BSQ_DT_BF16, s8 = a.state_bits == 8;
  AdamwTable<N> t;
  t.b1 = static_cast<float>(a.beta1);
  t.c1m = static_cast<float>(1.0 - a.beta1);
  t.b2 = static_cast<float>(a.beta2);
  t.c2m = static_cast<float>(1.0 - a.beta2);
  t.lr1 = static_cast<float>(a.lr / (1.0 - std::pow(a.beta1, static_cast<double>(a.step))));
  t.rc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a.beta2, static_cast<double>(a.step))));
  t.eps = static_cast<float>(a.eps);
  t.one = 1.f;
  t.salt = a.seed + static_cast<uint32_t>(a.step) * 0x7F4A7C15u;
  t.grad_scale = a.grad_scale;
  int i = 0;
  while (i < a.count) {
    t.count = 0;
    int64_t chunks = 0;
    for (; i < a.count && t.count < N; ++i) {
      const bsq_adamw_tensor& s = ts[i];
      if (s.n == 0) continue;
      const int64_t chunk = s8 ? kSweeps<true> * kStepA<true> : kSweeps<false> * kStepA<false>;
      const int64_t c = (s.n + chunk - 1) / chunk;
      if (chunks + c > INT32_MAX) break;   // the next launch takes it
      AdamwEntry& e = t.e[t.count++];
      e.p = static_cast<float*>(s.param);
      e.g = s.grad;
      e.m = s.m;
      e.v = s.v;
      e.ms = s.m_scale;
      e.vs = s.v_scale;
      e.copy = static_cast<__nv_bfloat16*>(s.copy);
      e.n = s.n;
      e.decay = static_cast<float>(1.0 - a.lr * static_cast<double>(s.weight_decay));
      e.counter = s.counter;
      e.chunk0 = static_cast<int32_t>(chunks);
      e.wide = on(e.p, 32) && on(e.g, g16 ? 16 : 32) && on(e.m, s8 ? 8 : 32) && on(e.v, s8 ? 8 : 32) && on(e.copy, 16);
      chunks += c;
    }
    if (t.count == 0) break;
    const dim3 grid(static_cast<unsigned>(chunks));
    if (g16 && s8) adamw_kernel<true, true, N><<<grid, kThreadsA<true>, 0, a.stream>>>(t);
    else if (g16) adamw_kernel<true, false, N><<<grid, kThreadsA<false>, 0, a.stream>>>(t);
    else if (s8) adamw_kernel<false, true, N><<<grid, kThreadsA<true>, 0, a.stream>>>(t);
    else adamw_kernel<false, false, N><<<grid, kThreadsA<false>, 0, a.stream>>>(t);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
      *msg = cudaGetErrorString(e);
      return static_cast<int>(e);
    }
  }
  return 0;
}

}  // namespace

int launch_adamw(const AdamwArgs& a, const char** msg) {
  return a.count <= kFewA ? launch_tables<kFewA>(a, msg) : launch_tables<kManyA>(a, msg);
}

}  // namespace bsq
