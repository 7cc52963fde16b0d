// rope.cuh -- what the rotary kernels (rope.cu, norm_rope.cu) share: the rows of
// a token's heads, its angles, and the columns that a head is cut into.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "internal.h"

namespace nvfp4kv {
namespace dev {

constexpr int kMaxPairs = 256;  // rotary_dim / 2

// columns of two 16-byte chunks that make up a head (rope_kernel)
__host__ __device__ __forceinline__ int rope_columns(const RopeParams& p) {
  return p.interleaved ? (p.head_dim + 15) / 16
                       : p.rotary_dim / 16 + (p.head_dim - p.rotary_dim + 15) / 16;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
struct Row {
  const uint16_t* in;
  uint16_t* out;
};

__device__ __forceinline__ Row row_of(const RopeParams& p, int64_t t, int h) {
  if (h < p.num_qo_heads)
    return {p.q + t * p.q_st + h * p.q_sh, p.q_out + t * p.qo_st + h * p.qo_sh};
  const int k = h - p.num_qo_heads;
  return {p.k + t * p.k_st + k * p.k_sh, p.k_out + t * p.ko_st + k * p.ko_sh};
}

// sines and cosines of token t, scaled, into sc[0 .. R/2)
__device__ __forceinline__ void angles(const RopeParams& p, int64_t t, float2* sc, int lane) {
  const int64_t pos = p.positions[t];
  for (int i = lane; i < p.rotary_dim / 2; i += 32) {
    const uint64_t turns = static_cast<uint64_t>(pos) * p.freq[i];
    const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    sc[i] = make_float2(c * p.attention_factor, s * p.attention_factor);
  }
  __syncwarp();
}

}  // namespace dev
}  // namespace nvfp4kv
