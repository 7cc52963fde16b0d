// rope.cu -- rotary positions of the query and key heads, sm_103a.
//
// Dim pair i of a head at position t turns by the angle 2 pi t F_i:
//   y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin),
// the pair being dims (i, i + R/2) or (2i, 2i + 1) of the first R dims; the
// others pass through.  Angles: t F_i turns is taken as an exact product of
// the 32-bit position and F_i in units of 2^-64, modulo 2^64, so whole turns
// drop out without a rounding whatever the position; the signed top 32 bits,
// rounded to float32, are the turn in [-1/2, 1/2): off by 2^-26 for the rounding,
// 2^-32 for the bits below and 2^-34 for the table's half unit at position 2^31.
// sincospif of twice that gives sine and cosine to float32's accuracy.  Products and sums
// are float32, rounded once to the tensor's type.
//
// Bound by HBM for prompts (each element is read and written once) and by
// latency for a decode step.  A warp takes one token: its lanes compute the
// R/2 sines and cosines once (into shared memory), and every lane then keeps
// the eight pairs of its column in registers and walks the heads, so the
// angles cost a few percent of a 40-head token.  With few tokens the heads are
// spread over several warps.  Measured (replayed, three sets of tensors in turn):
// 16384 tokens x 40 heads of 128, bf16, 56 us, 6.0 TB/s (0.90 of a plain copy);
// 8191 x 18 heads of 256, a quarter rotating, f16, 30 us, 5.1 TB/s; 16 tokens
// 5.5 us, a launch and its dependent loads.  CTAs of one warp (65 and 32 us with
// two, 72 and 41 with eight: the warps that an SM runs then follow the token
// order, and the rows they stream stay neighbours), two heads in flight (four: 64
// and 34), four waves of CTAs at least (one: 58.5 and 31.5, sixteen: 61 and 45).
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"
#include "rope.cuh"

namespace nvfp4kv {
namespace {

using dev::angles;
using dev::kMaxPairs;
using dev::pack2;
using dev::rope_columns;
using dev::row_of;
using dev::unpack2;

constexpr int kBatch = 2;       // heads whose loads a lane has in flight
constexpr int kFewest = 152 * 128;  // warps a launch should have: four waves of CTAs

template <bool F16>
__device__ __forceinline__ float one(uint16_t x) {
  return unpack2<F16>(x).x;
}

// A lane's item is two 16-byte chunks of a head: in the half layout (R % 16 ==
// 0) the elements 8c .. 8c+7 and R/2 + 8c .., eight pairs, or two neighbouring
// chunks of the passing dims; interleaved, the elements 16c .. 16c+15, whose
// pairs past the rotary dims keep their bits.  A lane keeps its column and
// walks the heads in batches of kBatch: the loads of a batch are issued before
// its stores (which might alias them for all the compiler knows), and those of
// the first batch before the angles.
template <bool F16, bool INTER>
__global__ void __launch_bounds__(32) rope_kernel(const RopeParams p, int splits) {
  __shared__ __align__(16) float2 sc[kMaxPairs];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x / splits;
  const int part = static_cast<int>(blockIdx.x % splits);
  const int heads = p.num_qo_heads + p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int rcols = INTER ? 0 : half / 8;  // half layout: columns of pairs, then passing ones
  const int cols = rope_columns(p);
  const int side = 32 / cols;  // heads side by side (512 dims have 32 columns)
  const int step = splits * side, h0 = part * side + lane / cols, c = lane % cols;
  const bool idle = lane / cols >= side;
  uint4 va[kBatch], vb[kBatch];
  // the column's two chunks: elements d0 .., d1 .. (d1 may lie past the head)
  const int d0 = INTER ? 16 * c : c < rcols ? 8 * c : 2 * half + 16 * (c - rcols);
  const int d1 = !INTER && c < rcols ? half + 8 * c : d0 + 8;
  auto load = [&](int h1) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h1 + k * step;
      if (h < heads) {
        const uint16_t* in = row_of(p, t, h).in;
        va[k] = *reinterpret_cast<const uint4*>(in + d0);
        vb[k] = d1 < p.head_dim ? *reinterpret_cast<const uint4*>(in + d1)
                                : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  if (!idle) load(h0);
  angles(p, t, sc, lane);
  if (idle) return;
  // pairs of this column that turn (8 unless the rotary dims end in it)
  const int live = INTER ? min(8, max(0, half - 8 * c)) : c < rcols ? 8 : 0;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 x = j < live ? sc[8 * c + j] : make_float2(1.f, 0.f);
    cs[j] = x.x;
    sn[j] = x.y;
  }
  for (int h1 = h0; h1 < heads; h1 += kBatch * step) {
    if (h1 > h0) load(h1);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h1 + k * step;
      if (h >= heads) break;
      uint32_t a[4] = {va[k].x, va[k].y, va[k].z, va[k].w};
      uint32_t b[4] = {vb[k].x, vb[k].y, vb[k].z, vb[k].w};
      if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<F16>(a[j]), y = unpack2<F16>(b[j]);
          const uint32_t oa = pack2<F16>(x.x * cs[j] - x.y * sn[j], x.y * cs[j] + x.x * sn[j]);
          const uint32_t ob = pack2<F16>(y.x * cs[j + 4] - y.y * sn[j + 4],
                                         y.y * cs[j + 4] + y.x * sn[j + 4]);
          a[j] = j < live ? oa : a[j];
          b[j] = j + 4 < live ? ob : b[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<F16>(a[j]), y = unpack2<F16>(b[j]);
          const float c0 = cs[2 * j], c1 = cs[2 * j + 1], s0 = sn[2 * j], s1 = sn[2 * j + 1];
          const uint32_t oa = pack2<F16>(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
          const uint32_t ob = pack2<F16>(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
          a[j] = live ? oa : a[j];
          b[j] = live ? ob : b[j];
        }
      }
      uint16_t* out = row_of(p, t, h).out;
      *reinterpret_cast<uint4*>(out + d0) = make_uint4(a[0], a[1], a[2], a[3]);
      if (d1 < p.head_dim)
        *reinterpret_cast<uint4*>(out + d1) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
}

// The half layout where R/2 is not a multiple of 8: the pairs of a 16-byte column
// do not lie in another one.  A lane still loads, turns and stores whole columns
// (CP of them), and takes the other halves of its pairs from shared memory, where
// the warp lays the heads of a step.  8192 tokens x 48 heads of 128, 66 dims
// turning: 45 us, 4.5 TB/s (element by element 115 us).
template <bool F16, int CP>
__global__ void __launch_bounds__(32) rope_odd_kernel(const RopeParams p, int splits) {
  __shared__ __align__(16) float2 sc[kMaxPairs];
  __shared__ __align__(16) uint16_t rows[kBatch][256 * CP];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x / splits;
  const int part = static_cast<int>(blockIdx.x % splits);
  angles(p, t, sc, lane);
  const int heads = p.num_qo_heads + p.num_kv_heads, half = p.rotary_dim / 2;
  const int cols = p.head_dim / 8, wide = min(32, cols), side = 32 / wide, step = splits * side;
  const int hs = lane / wide, col = lane % wide;  // this lane's head of a step, its column
  float cs[CP][8], sn[CP][8];  // y = x cs + (the other of the pair) sn
#pragma unroll
  for (int c = 0; c < CP; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = 8 * (col + 32 * c) + j;
      const float2 a = d < 2 * half ? sc[d < half ? d : d - half] : make_float2(1.f, 0.f);
      cs[c][j] = a.x;
      sn[c][j] = d < half ? -a.y : a.y;
    }
  for (int b = part * side; b < heads; b += kBatch * step) {  // (the whole warp together)
    uint4 v[kBatch][CP];
    auto mine = [&](int k, int c) {
      return hs < side && b + hs + k * step < heads && col + 32 * c < cols;
    };
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int c = 0; c < CP; ++c)
        if (mine(k, c))
          v[k][c] = reinterpret_cast<const uint4*>(row_of(p, t, b + hs + k * step).in)[col + 32 * c];
    __syncwarp();  // the last step's rows have been read
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int c = 0; c < CP; ++c)
        if (mine(k, c))
          *reinterpret_cast<uint4*>(rows[k] + hs * p.head_dim + 8 * (col + 32 * c)) = v[k][c];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        if (!mine(k, c)) continue;
        const uint16_t* row = rows[k] + hs * p.head_dim;
        uint32_t w[4] = {v[k][c].x, v[k][c].y, v[k][c].z, v[k][c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d = 8 * (col + 32 * c) + 2 * j;
          const float2 x = unpack2<F16>(w[j]);
          float y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int o = d + e < half ? d + e + half : d + e - half;  // the other of the pair
            const float z = d + e < 2 * half ? one<F16>(row[o]) : 0.f;
            y[e] = (e ? x.y : x.x) * cs[c][2 * j + e] + z * sn[c][2 * j + e];
          }
          // (dims that pass keep their bits; rotary_dim is even)
          if (d < 2 * half) w[j] = pack2<F16>(y[0], y[1]);
        }
        reinterpret_cast<uint4*>(row_of(p, t, b + hs + k * step).out)[col + 32 * c] =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  const int heads = p.num_qo_heads + p.num_kv_heads;
  if (p.num_tokens == 0 || heads == 0) return cudaSuccess;
  const bool odd = !p.interleaved && p.rotary_dim % 16 != 0;
  // Heads over several warps while the tokens alone are few; a warp has `side`
  // heads side by side (the columns of rope_kernel).
  const int cols = odd ? p.head_dim / 8 : rope_columns(p);
  const int side = cols >= 32 ? 1 : 32 / cols;
  const int most = (heads + side - 1) / side;
  const int64_t want = ((int64_t)kFewest + p.num_tokens - 1) / p.num_tokens;
  const int splits = want < most ? static_cast<int>(want) : most;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.num_tokens) * splits);
  if (odd && cols > 32)
    (p.f16 ? rope_odd_kernel<true, 2> : rope_odd_kernel<false, 2>)<<<blocks, 32, 0, stream>>>(
        p, splits);
  else if (odd)
    (p.f16 ? rope_odd_kernel<true, 1> : rope_odd_kernel<false, 1>)<<<blocks, 32, 0, stream>>>(
        p, splits);
  else if (p.interleaved)
    (p.f16 ? rope_kernel<true, true> : rope_kernel<false, true>)<<<blocks, 32, 0,
                                                                  stream>>>(p, splits);
  else
    (p.f16 ? rope_kernel<true, false> : rope_kernel<false, false>)<<<blocks, 32, 0,
                                                                    stream>>>(p, splits);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
