// bsq_e4m3.cuh -- register-level encoding of blocks to E4M3 codes, shared by the kernels that
// quantize (bsq_quant_e4m3.cu, bsq_tokens.cu):
//   a = max |x| over the block (a zero block takes 448, a smaller one than 2^-100 takes 2^-100)
//   scale = a / 448,   code = E4M3(x * (448 / a)), nearest even, saturating at +-448
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace bsq {

// Eight consecutive elements of either input type, as loaded.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  // bit pattern of the largest magnitude, as a float32's
  __device__ uint32_t amax() const {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(a << 16, a & 0xFFFF0000u);
  }
  __device__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ uint32_t amax() const {
    auto m = [](float x) { return __float_as_uint(x) & 0x7FFFFFFFu; };
    return max(max(max(m(a.x), m(a.y)), max(m(a.z), m(a.w))), max(max(m(b.x), m(b.y)), max(m(b.z), m(b.w))));
  }
  __device__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w) : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// a of the definition from the block's largest magnitude.
__device__ __forceinline__ float block_amax(uint32_t bits) {
  const float a = __uint_as_float(bits);
  return bits == 0 ? 448.f : a < 7.888609052210118e-31f ? 7.888609052210118e-31f : a;   // 2^-100; NaN stays
}

template <typename T>
__device__ __forceinline__ uint2 encode(const Eight<T>& v, float inv) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = v.pair(i);
    c[i] = e4m3x2(f.x * inv, f.y * inv);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace bsq
