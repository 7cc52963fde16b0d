// e4m3.cuh -- the scales of the E4M3 cache, shared by its append and its two
// attention kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace nvfp4kv {
namespace dev {

constexpr float kMinScale = 0x1p-64f, kMaxScale = 0x1p64f;

// the scale, or the nearer end of the range (the lower for a NaN)
__device__ __forceinline__ float clamped_scale(float s) {
  return fminf(fmaxf(s, kMinScale), kMaxScale);
}
// log2 of a positive normal float, exact for a power of two
__device__ __forceinline__ float log2_scale(float s) {
  const uint32_t u = __float_as_uint(s);
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float((u & 0x7FFFFFu) | 0x3F800000u)));
  return static_cast<float>(static_cast<int>(u >> 23) - 127) + r;
}

}  // namespace dev
}  // namespace nvfp4kv
