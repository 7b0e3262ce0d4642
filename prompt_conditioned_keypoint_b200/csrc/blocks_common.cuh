// What the transformer-block kernels share: 16-byte loads and stores of fp32 and
// bf16 rows as fp32 values, and the activations of gkd_linear's epilogue.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gkd_internal.h"
#include "ptx.cuh"

namespace gkd {

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Four consecutive elements (16 bytes of fp32, 8 bytes of bf16) as fp32.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}
__device__ __forceinline__ void store4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// The factor on the scores of a row whose largest is m, and what m comes to with it (no key yet: every weight is 0).
__device__ __forceinline__ float score_factor(const ScoreScale& s, float m) { return fabsf(m) < s.far ? s.c : s.pow2; }
__device__ __forceinline__ float score_offset(const ScoreScale& s, float m) {
  return m == -INFINITY ? 0.f : m * score_factor(s, m);
}

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActQuickGelu = 3 };

__device__ __forceinline__ float ex2_approx(float x) {   // 2^x, about 2^-22 relative
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {   // 1 / x, within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {   // NaN if one of them is
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// y Phi(y) = max(y, 0) - |y| erfc(|y| / sqrt 2) / 2, with erfc(x) e^(x^2) as a
// polynomial of degree 7 in 1 / (1 + 0.49 x): the form of Hastings' rational
// approximations, its coefficients fitted for this file by reweighted least squares
// on 0 <= x <= 9.5 (erfc within 4e-7 as evaluated in fp32, within 7e-6 of its value
// up to x = 6). Two values share their operations; with erff (and one value at a time)
// the epilogue of a 128 x 256 tile outlasted its products: 36864 x 1280 -> 5120 took
// 1311 us.
__device__ __forceinline__ float2 gelu2(float2 y) {
  auto both = [](float c) { return make_float2(c, c); };
  const float2 z = make_float2(fminf(fabsf(y.x), 20.f), fminf(fabsf(y.y), 20.f));   // erfc is 0 from there on; keeps inf * 0 out
  float2 t = fma2(z, both(0.34648232f), both(1.f));
  t = make_float2(rcp_approx(t.x), rcp_approx(t.y));
  float2 q = fma2(t, both(0.0901875049f), both(-0.3830944f));
  q = fma2(q, t, both(0.462687463f));
  q = fma2(q, t, both(-0.0114476597f));
  q = fma2(q, t, both(0.295998424f));
  q = fma2(q, t, both(0.268764943f));
  q = fma2(q, t, both(0.276903629f));
  const float2 x = mul2(mul2(z, z), both(-0.72134752f));
  const float2 e = mul2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), t);
  // NaN stays NaN
  return fma2(mul2(z, both(-0.5f)), mul2(q, e), make_float2(y.x < 0.f ? 0.f : y.x, y.y < 0.f ? 0.f : y.y));
}

__device__ __forceinline__ float quick_gelu(float y) {   // y / (1 + exp(-1.702 y))
  return y * rcp_approx(1.f + ex2_approx(-2.45546696f * y));
}

// The activation of a few values at once: one branch for all of them.
template <int N>
__device__ __forceinline__ void activate(float (&y)[N], int act) {
  if (act == kActRelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = y[e] < 0.f ? 0.f : y[e];
  } else if (act == kActGelu) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 g = gelu2(make_float2(y[e], y[e + 1]));
      y[e] = g.x;
      y[e + 1] = g.y;
    }
  } else if (act == kActQuickGelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = quick_gelu(y[e]);
  }
}

}  // namespace gkd
