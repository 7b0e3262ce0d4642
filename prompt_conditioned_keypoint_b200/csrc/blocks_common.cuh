// What the transformer-block kernels share: 16-byte loads and stores of fp32 and
// bf16 rows as fp32 values, and the activations of gkd_linear's epilogue.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace gkd {

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

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

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActQuickGelu = 3 };

__device__ __forceinline__ float activate(float y, int act) {
  switch (act) {
    case kActRelu:
      return y < 0.f ? 0.f : y;                                   // NaN stays NaN
    case kActGelu:
      return 0.5f * y * (1.f + erff(y * 0.70710678f));
    case kActQuickGelu:
      return y / (1.f + expf(-1.702f * y));
    default:
      return y;
  }
}

}  // namespace gkd
