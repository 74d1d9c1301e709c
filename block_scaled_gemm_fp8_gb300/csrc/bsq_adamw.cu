// bsq_adamw.cu -- one AdamW step (decoupled weight decay, Loshchilov and Hutter 2019) over many
// tensors in one launch per 256 of them, FP32 parameters, states in 32 or in 8 bits:
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
// Every operation is rounded by itself (no contraction), so the step equals the same
// formula in float32 tensor operations bit for bit.
//
// Bound by HBM: 28 or 30 bytes per element with 32-bit states and a BF16 copy (14.1 to 16.1
// with 8-bit ones).  A thread owns 8 consecutive elements (32-byte accesses), 16 lanes a
// scale block, a CTA a chunk of one tensor, found by bisection in the launch's table.
#include <cmath>

#include <cuda_bf16.h>

#include "bsq_internal.h"
#include "../../include/bsq.h"

namespace bsq {

namespace {

constexpr int kThreadsA = 256;
constexpr int kStepA = kThreadsA * 8;      // elements of one sweep of a CTA
constexpr int kSweeps = 2;
constexpr int kChunkA = kStepA * kSweeps;
constexpr int kTableA = 256;               // tensors of one launch

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

struct AdamwTable {
  AdamwEntry e[kTableA];
  int32_t count;
  float b1, c1m, b2, c2m;   // betas and 1 - betas
  float lr1, rc2, eps;      // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t salt;            // seed and step
  const float* grad_scale;
};
static_assert(sizeof(AdamwTable) <= 32764, "kernel parameter space");

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

// 32 random bits of an element: a Weyl step and MurmurHash3's finalizer (Appleby).
__device__ __forceinline__ uint32_t element_bits(uint32_t i, uint32_t salt) {
  uint32_t x = i * 0x9E3779B1u + salt;
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

// E4M3 magnitude next to a (0 <= a, about 448 at most), up with the probability of the part
// cut off: 16 random bits against the mantissa bits below E4M3's three, or against the
// part below its subnormal step of 2^-9.  NaN stays.
__device__ __forceinline__ float round_at_random(float a, uint32_t bits) {
  const float big = __uint_as_float((__float_as_uint(a) + (bits << 4)) & 0xFFF00000u);
  const float small = __fmul_rn(floorf(__fadd_rn(__fmul_rn(a, 512.f), __fmul_rn(static_cast<float>(bits), 1.52587890625e-5f))),
                                1.953125e-3f);
  const float r = a >= 0.015625f ? big : small;
  return r > 448.f ? 448.f : r;
}

__device__ __forceinline__ float block_amax(float a) {
  return a == 0.f ? 448.f : a < 7.888609052210118e-31f ? 7.888609052210118e-31f : a;   // 2^-100; NaN stays
}

// Scale block of 16 lanes x 8 values: the block's a from each lane's largest magnitude
// (bit patterns: NaN is above infinity).
__device__ __forceinline__ float lane16_amax(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return block_amax(__uint_as_float(m));
}

template <bool G16, bool S8>
__global__ void __launch_bounds__(kThreadsA) adamw_kernel(const __grid_constant__ AdamwTable t) {
  int lo = 0, hi = t.count - 1;
  const int chunk = blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  const AdamwEntry& e = t.e[lo];
  const float gs = t.grad_scale ? __ldg(t.grad_scale) : 1.f;
  const int64_t first = static_cast<int64_t>(chunk - e.chunk0) * kChunkA + threadIdx.x * 8;
#pragma unroll
  for (int sweep = 0; sweep < kSweeps; ++sweep) {
    const int64_t i0 = first + sweep * kStepA;
    const int64_t left = e.n - i0;
    const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;   // elements of this thread
    const bool wide = e.wide && n == 8;
    if (!S8 && n == 0) continue;
    float g[8], p[8], m[8], v[8];
    float ms = 0.f, vs = 0.f;
    if (S8 && n > 0) {
      ms = e.ms[i0 >> 7];
      vs = e.vs[i0 >> 7];
    }
    if (wide) {
      ld8(e.p + i0, p);
      if (G16) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.g) + i0));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[2 * j] = __uint_as_float(u[j] << 16);
          g[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
      } else {
        ld8(static_cast<const float*>(e.g) + i0, g);
      }
      if (S8) {
        const uint2 cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(e.m) + i0);
        const uint2 cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(e.v) + i0);
        const uint32_t um[4] = {cm.x & 0xFFFFu, cm.x >> 16, cm.y & 0xFFFFu, cm.y >> 16};
        const uint32_t uv[4] = {cv.x & 0xFFFFu, cv.x >> 16, cv.y & 0xFFFFu, cv.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 fm = from_e4m3x2(um[j]), fv = from_e4m3x2(uv[j]);
          m[2 * j] = fm.x;
          m[2 * j + 1] = fm.y;
          v[2 * j] = fv.x;
          v[2 * j + 1] = fv.y;
        }
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
          g[j] = G16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.g)[i0 + j]) : static_cast<const float*>(e.g)[i0 + j];
          if (S8) {
            m[j] = from_e4m3x2(static_cast<const uint8_t*>(e.m)[i0 + j]).x;
            v[j] = from_e4m3x2(static_cast<const uint8_t*>(e.v)[i0 + j]).x;
          } else {
            m[j] = static_cast<const float*>(e.m)[i0 + j];
            v[j] = static_cast<const float*>(e.v)[i0 + j];
          }
        }
      }
    }
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = __fmul_rn(g[j], gs);
      if (S8) {
        m[j] = __fmul_rn(m[j], ms);
        v[j] = __fmul_rn(v[j], vs);
        v[j] = __fmul_rn(v[j], v[j]);
      }
      m[j] = __fadd_rn(__fmul_rn(m[j], t.b1), __fmul_rn(gj, t.c1m));
      v[j] = __fadd_rn(__fmul_rn(v[j], t.b2), __fmul_rn(__fmul_rn(gj, gj), t.c2m));
      r[j] = __fsqrt_rn(v[j]);
      const float u = __fdiv_rn(__fmul_rn(m[j], t.lr1), __fadd_rn(__fmul_rn(r[j], t.rc2), t.eps));
      p[j] = __fsub_rn(__fmul_rn(p[j], e.decay), u);
      if (S8 && j >= n) m[j] = r[j] = 0.f;   // past the end: no part of the block's maximum
    }
    uint32_t cm[8], cv[8];
    if (S8) {
      const float am = lane16_amax(m), ar = lane16_amax(r);
      const float im = __fdiv_rn(448.f, am), ir = __fdiv_rn(448.f, ar);
      if (n > 0 && (threadIdx.x & 15) == 0) {
        e.ms[i0 >> 7] = __fdiv_rn(am, 448.f);
        e.vs[i0 >> 7] = __fdiv_rn(ar, 448.f);
      }
      const uint32_t at = e.counter + static_cast<uint32_t>(i0);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float qm[2], qv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t bits = element_bits(at + j + k, t.salt);
          const float xm = __fmul_rn(m[j + k], im), xr = __fmul_rn(r[j + k], ir);
          qm[k] = copysignf(round_at_random(fabsf(xm), bits & 0xFFFFu), xm);
          const float q = round_at_random(xr, bits >> 16);
          qv[k] = xr > 0.f && q == 0.f ? 1.953125e-3f : q;
        }
        const uint32_t c2m = e4m3x2(qm[0], qm[1]), c2v = e4m3x2(qv[0], qv[1]);
        cm[j] = c2m & 0xFFu;
        cm[j + 1] = c2m >> 8;
        cv[j] = c2v & 0xFFu;
        cv[j + 1] = c2v >> 8;
      }
    }
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
      if (S8) {
        auto four = [](const uint32_t* c) { return c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24); };
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.m) + i0) = make_uint2(four(cm), four(cm + 4));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.v) + i0) = make_uint2(four(cv), four(cv + 4));
      } else {
        st8(static_cast<float*>(e.m) + i0, m);
        st8(static_cast<float*>(e.v) + i0, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          e.p[i0 + j] = p[j];
          if (e.copy) e.copy[i0 + j] = __float2bfloat16_rn(p[j]);
          if (S8) {
            static_cast<uint8_t*>(e.m)[i0 + j] = static_cast<uint8_t>(cm[j]);
            static_cast<uint8_t*>(e.v)[i0 + j] = static_cast<uint8_t>(cv[j]);
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

}  // namespace

int launch_adamw(const AdamwArgs& a, const char** msg) {
  const bsq_adamw_tensor* ts = static_cast<const bsq_adamw_tensor*>(a.tensors);
  const bool g16 = a.grad_dtype == BSQ_DT_BF16, s8 = a.state_bits == 8;
  AdamwTable t;
  t.b1 = static_cast<float>(a.beta1);
  t.c1m = static_cast<float>(1.0 - a.beta1);
  t.b2 = static_cast<float>(a.beta2);
  t.c2m = static_cast<float>(1.0 - a.beta2);
  t.lr1 = static_cast<float>(a.lr / (1.0 - std::pow(a.beta1, static_cast<double>(a.step))));
  t.rc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a.beta2, static_cast<double>(a.step))));
  t.eps = static_cast<float>(a.eps);
  t.salt = a.seed + static_cast<uint32_t>(a.step) * 0x7F4A7C15u;
  t.grad_scale = a.grad_scale;
  int i = 0;
  while (i < a.count) {
    t.count = 0;
    int64_t chunks = 0;
    for (; i < a.count && t.count < kTableA; ++i) {
      const bsq_adamw_tensor& s = ts[i];
      if (s.n == 0) continue;
      const int64_t c = (s.n + kChunkA - 1) / kChunkA;
      if (c > INT32_MAX) {
        *msg = "a tensor is too long";
        return -1;
      }
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
    if (g16 && s8) adamw_kernel<true, true><<<grid, kThreadsA, 0, a.stream>>>(t);
    else if (g16) adamw_kernel<true, false><<<grid, kThreadsA, 0, a.stream>>>(t);
    else if (s8) adamw_kernel<false, true><<<grid, kThreadsA, 0, a.stream>>>(t);
    else adamw_kernel<false, false><<<grid, kThreadsA, 0, a.stream>>>(t);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
      *msg = cudaGetErrorString(e);
      return static_cast<int>(e);
    }
  }
  return 0;
}

}  // namespace bsq
