// rope.cu -- rotary positions of the query and key heads, sm_103a.
//
// Dim pair i of a head at position t turns by the angle 2 pi t F_i:
//   y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin),
// the pair being dims (i, i + R/2) or (2i, 2i + 1) of the first R dims; the
// others pass through.  Angles: t F_i turns is taken as an exact product of
// the 32-bit position and F_i in units of 2^-64, modulo 2^64, so whole turns
// drop out without a rounding whatever the position; the signed top 32 bits,
// rounded to float32, are the turn in [-1/2, 1/2) to 2^-26, and sincospif of
// twice that gives sine and cosine to float32's accuracy.  Products and sums
// are float32, rounded once to the tensor's type.
//
// Bound by HBM for prompts (each element is read and written once) and by
// latency for a decode step.  A warp takes one token: its lanes compute the
// R/2 sines and cosines once (into shared memory), and every lane then keeps
// the eight (half layout) or four (interleaved) pairs of its 16-byte column in
// registers and walks the heads, so the angles cost a few percent of a
// 40-head token.  With few tokens the heads are spread over several warps.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace nvfp4kv {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxPairs = 256;  // rotary_dim / 2

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
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
template <bool F16>
__device__ __forceinline__ float one(uint16_t x) {
  return unpack2<F16>(x).x;
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

// 16-byte columns.  Half layout: R % 16 == 0, a column holds pairs 8c .. 8c+7
// (the elements at 8c and R/2 + 8c).  Interleaved: a column holds pairs
// 4c .. 4c+3.  Columns past the rotary dims are copied.
template <bool F16, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeParams p, int splits) {
  __shared__ __align__(16) float2 s_sc[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = unit / splits;
  const int part = static_cast<int>(unit % splits);
  if (t >= p.num_tokens) return;
  float2* sc = s_sc[warp];
  angles(p, t, sc, lane);
  const int heads = p.num_qo_heads + p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int rcols = INTER ? (half + 3) / 4 : half / 8;  // columns with pairs
  const int c0 = INTER ? rcols : half / 4;              // first passing 16-byte column
  const int cols = rcols + p.head_dim / 8 - c0;         // work columns of a head
  // lanes: column x head; a column keeps its pairs over the heads it walks
  const int wide = min(32, cols);
  const int hl = 32 / wide;                             // heads side by side
  const int my_h = lane / wide;
  if (my_h >= hl) return;
  for (int c = lane % wide; c < cols; c += wide) {
    if (c >= rcols) {  // passing dims
      const int d = 8 * (c - rcols + c0);
      for (int h = part * hl + my_h; h < heads; h += splits * hl) {
        const Row r = row_of(p, t, h);
        if (r.in != r.out)
          *reinterpret_cast<uint4*>(r.out + d) = *reinterpret_cast<const uint4*>(r.in + d);
      }
      continue;
    }
    constexpr int NP = INTER ? 4 : 8;
    float cs[NP], sn[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool in = !INTER || NP * c + j < half;
      cs[j] = in ? sc[NP * c + j].x : 1.f;
      sn[j] = in ? sc[NP * c + j].y : 0.f;
    }
    if constexpr (INTER) {
      const int live = min(NP, half - NP * c);  // below 4 where the rotary dims end
#pragma unroll 4
      for (int h = part * hl + my_h; h < heads; h += splits * hl) {
        const Row r = row_of(p, t, h);
        const uint4 v = *reinterpret_cast<const uint4*>(r.in + 8 * c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<F16>(w[j]);
          const uint32_t y = pack2<F16>(x.x * cs[j] - x.y * sn[j], x.y * cs[j] + x.x * sn[j]);
          o[j] = j < live ? y : w[j];
        }
        *reinterpret_cast<uint4*>(r.out + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
#pragma unroll 4
      for (int h = part * hl + my_h; h < heads; h += splits * hl) {
        const Row r = row_of(p, t, h);
        const uint4 va = *reinterpret_cast<const uint4*>(r.in + 8 * c);
        const uint4 vb = *reinterpret_cast<const uint4*>(r.in + half + 8 * c);
        const uint32_t a[4] = {va.x, va.y, va.z, va.w}, b[4] = {vb.x, vb.y, vb.z, vb.w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<F16>(a[j]), y = unpack2<F16>(b[j]);
          const float c0f = cs[2 * j], c1f = cs[2 * j + 1], s0f = sn[2 * j], s1f = sn[2 * j + 1];
          oa[j] = pack2<F16>(x.x * c0f - y.x * s0f, x.y * c1f - y.y * s1f);
          ob[j] = pack2<F16>(y.x * c0f + x.x * s0f, y.y * c1f + x.y * s1f);
        }
        *reinterpret_cast<uint4*>(r.out + 8 * c) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        *reinterpret_cast<uint4*>(r.out + half + 8 * c) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
      }
    }
  }
}

// The half layout where R/2 is not a multiple of 8: its pairs do not lie in
// 16-byte columns, so single elements are loaded.
template <bool F16>
__global__ void __launch_bounds__(kWarps * 32) rope_odd_kernel(const RopeParams p, int splits) {
  __shared__ __align__(16) float2 s_sc[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = unit / splits;
  const int part = static_cast<int>(unit % splits);
  if (t >= p.num_tokens) return;
  float2* sc = s_sc[warp];
  angles(p, t, sc, lane);
  const int heads = p.num_qo_heads + p.num_kv_heads, half = p.rotary_dim / 2;
  for (int h = part; h < heads; h += splits) {
    const Row r = row_of(p, t, h);
    for (int i = lane; i < half; i += 32) {
      const float x = one<F16>(r.in[i]), y = one<F16>(r.in[half + i]);
      const float2 a = sc[i];
      const uint32_t o = pack2<F16>(x * a.x - y * a.y, y * a.x + x * a.y);
      r.out[i] = static_cast<uint16_t>(o);
      r.out[half + i] = static_cast<uint16_t>(o >> 16);
    }
    if (r.in != r.out)
      for (int d = p.rotary_dim + lane; d < p.head_dim; d += 32) r.out[d] = r.in[d];
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  const int heads = p.num_qo_heads + p.num_kv_heads;
  if (p.num_tokens == 0 || heads == 0) return cudaSuccess;
  const bool odd = !p.interleaved && p.rotary_dim % 16 != 0;
  // Heads over several warps while the tokens alone leave SMs without one; a
  // warp has `side` heads side by side (the columns of rope_kernel).
  const int half = p.rotary_dim / 2;
  const int cols = p.interleaved ? p.head_dim / 8 : half / 8 + (p.head_dim - p.rotary_dim) / 8;
  const int side = odd || cols >= 32 ? 1 : 32 / cols;
  const int most = (heads + side - 1) / side;
  int splits = (152 * kWarps * 2 + p.num_tokens - 1) / p.num_tokens;
  if (splits > most) splits = most;
  const int64_t units = static_cast<int64_t>(p.num_tokens) * splits;
  const unsigned blocks = static_cast<unsigned>((units + kWarps - 1) / kWarps);
  if (odd)
    (p.f16 ? rope_odd_kernel<true> : rope_odd_kernel<false>)<<<blocks, kWarps * 32, 0, stream>>>(
        p, splits);
  else if (p.interleaved)
    (p.f16 ? rope_kernel<true, true> : rope_kernel<false, true>)<<<blocks, kWarps * 32, 0,
                                                                  stream>>>(p, splits);
  else
    (p.f16 ? rope_kernel<true, false> : rope_kernel<false, false>)<<<blocks, kWarps * 32, 0,
                                                                    stream>>>(p, splits);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
