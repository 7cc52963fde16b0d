// norm_rope.cu -- norms of the query and key heads and their rotary positions
// in one pass, sm_103a.
//
// A head x of D dims at position t becomes
//   n = x / sqrt(sum_d x_d^2 / D + eps) * (w + offset),
// w the learned weights of the queries' or the keys' norm, and the first R dims of
// n turn as in rope.cu (angles, pairs and their accuracy are those of rope.cuh);
// the others are n as it is.  With r = 1 / sqrt(...) a pair is
//   y1 = (r x1) (w1 c) - (r x2) (w2 s),  y2 = (r x2) (w2 c) + (r x1) (w1 s),
// c and s the pair's cosine and sine: the four products of a weight are the same for
// all heads of a token, so they are formed once and kept.  Sums, r and products
// are float32, rounded once to the tensor's type.
//
// A sum of squares of bf16 values may pass float32's range where its root does
// not: such a head is scaled by 2^-70 first (exact; the elements that it loses end
// below the type's smallest value).  eps is at least 1e-20, so squares that
// underflow do not count.
//
// Bound by HBM for prompts (each element is read and written once), by latency for
// a few tokens.  As in rope.cu a warp takes a token (with few tokens, some of its
// heads) and a lane keeps a column of two 16-byte chunks; the column's sum goes
// over the lanes of its head by shuffles, a power of two of them.  Loads, sum, root and
// stores of a head are one dependent chain, so a lane keeps three heads' loads in a ring:
// a head's place is taken by the load three on as soon as it is unpacked.  Measured
// (replayed, three sets of tensors in turn): 16384 tokens x 40 heads of 128, bf16, 60 us,
// 5.6 TB/s (0.84 of a plain copy); 211 tokens x 18 heads of 256, a quarter in pairs, f16,
// 3.8 us.  Loads in batches of three 66 us, of two 73 (and 85 with a token's heads on two
// warps: the angles and weights are then formed twice); two or four heads in the ring 63
// and 64; chunks of 8 bytes, half the registers and more warps, 66; loads that stay out of L1
// 62, streaming stores 60.2.
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

constexpr int kBatch = 3;          // heads whose loads a lane has in flight
constexpr int kFewest = 152 * 64;  // warps a launch should have

__host__ __device__ __forceinline__ int lanes_for(int columns) {  // a power of two, at most 32
  int w = 32;
  while (w / 2 >= columns) w /= 2;
  return w;
}

template <bool F16>
__device__ __forceinline__ float weight(const NormRopeParams& p, bool k, int d) {
  const void* w = k ? p.k_weight : p.q_weight;
  const float x = p.weight_f32 ? static_cast<const float*>(w)[d]
                               : unpack2<F16>(static_cast<const uint16_t*>(w)[d]).x;
  return x + p.weight_offset;
}

// 8 elements of 16 bits
struct Chunk {
  uint32_t w[4];
};
__device__ __forceinline__ Chunk load_chunk(const uint16_t* at) {
  const uint4 v = *reinterpret_cast<const uint4*>(at);
  return {{v.x, v.y, v.z, v.w}};
}
template <bool F16>
__device__ __forceinline__ void store_chunk(uint16_t* at, const float* y) {
  *reinterpret_cast<uint4*>(at) = make_uint4(pack2<F16>(y[0], y[1]), pack2<F16>(y[2], y[3]),
                                             pack2<F16>(y[4], y[5]), pack2<F16>(y[6], y[7]));
}
template <bool F16>
__device__ __forceinline__ void unpack_chunk(const Chunk& c, float* x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2<F16>(c.w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}

// the weights of a chunk of dims
template <bool F16>
__device__ __forceinline__ void weight_chunk(const NormRopeParams& p, bool k, int d,
                                             float (&w)[8]) {
  const void* at = k ? p.k_weight : p.q_weight;
  if (p.weight_f32) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(at) + d + j);
      w[j] = a.x; w[j + 1] = a.y; w[j + 2] = a.z; w[j + 3] = a.w;
    }
  } else {
    unpack_chunk<F16>(load_chunk(static_cast<const uint16_t*>(at) + d), w);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] += p.weight_offset;
}

template <bool F16, int N>
__device__ __forceinline__ float head_sum(const float (&x)[N], int lanes) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) ss = fmaf(x[j], x[j], ss);
  for (int o = lanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return ss;
}

// r of the head that this lane's values belong to (a head has `lanes` neighbouring
// lanes); values whose squares leave float32's range are scaled in place
template <bool F16, int N>
__device__ __forceinline__ float head_factor(const NormRopeParams& p, float (&x)[N], int lanes,
                                             float inv_dim) {
  float ss = head_sum<F16>(x, lanes), eps = p.eps;
  if (!F16 && __any_sync(0xffffffffu, isinf(ss))) {  // (f16 squares stay below 2^42)
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) most = fmaxf(most, fabsf(x[j]));
    for (int o = lanes / 2; o > 0; o >>= 1)
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    // (an infinite element stays: r is 0, and the element NaN, as the formula has it)
    const bool scaled = isinf(ss) && !isinf(most);
    const float s = scaled ? 0x1p-70f : 1.f;  // (512 squares of at most 2^58)
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] *= s;
    ss = head_sum<F16>(x, lanes);
    eps *= s * s;
  }
  return rsqrtf(fmaf(ss, inv_dim, eps));
}

// Columns as in rope_kernel: in the half layout (R % 16 == 0) the elements 8c .. 8c+7 and
// R/2 + 8c .., eight pairs, or two neighbouring chunks of the dims behind; interleaved, the
// elements 16c .. 16c+15.
template <bool F16, bool INTER>
__global__ void __launch_bounds__(32, 20) norm_rope_kernel(const NormRopeParams np, int splits) {
  __shared__ __align__(16) float2 sc[kMaxPairs];
  const RopeParams& p = np.rope;
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x / splits;
  const int part = static_cast<int>(blockIdx.x % splits);
  const int heads = p.num_qo_heads + p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int rcols = INTER ? 0 : half / 8;
  const int cols = rope_columns(p), wide = lanes_for(cols);
  const int side = 32 / wide, step = splits * side;  // heads side by side, heads a step passes
  const int hs = lane / wide, c = lane % wide;
  // (a lane without a head of its own: there may be no weights for it either)
  const bool idle = c >= cols || part * side + hs >= heads;
  const float inv_dim = 1.f / static_cast<float>(p.head_dim);
  // the column's two chunks: elements d0 .., d1 .. (d1 may lie past the head)
  const int d0 = INTER ? 16 * c : c < rcols ? 8 * c : 2 * half + 16 * (c - rcols);
  const int d1 = !INTER && c < rcols ? half + 8 * c : d0 + 8;
  const bool two = !idle && d1 < p.head_dim;
  Chunk va[kBatch], vb[kBatch];
  auto load = [&](int h, Chunk& a, Chunk& b) {
    a = b = Chunk{};
    if (h < heads && !idle) {
      const uint16_t* in = row_of(p, t, h).in;
      a = load_chunk(in + d0);
      if (two) b = load_chunk(in + d1);
    }
  };
#pragma unroll
  for (int k = 0; k < kBatch; ++k) load(part * side + hs + k * step, va[k], vb[k]);
  angles(p, t, sc, lane);
  // y of the first chunk's element j: x_j a_j + (the pair's other) b_j; second chunk: e, f
  float ca[8], cb[8], ce[8], cf[8];
  auto coefficients = [&](bool k) {
    float wa[8] = {}, wb[8] = {};
    if (!idle) weight_chunk<F16>(np, k, d0, wa);
    if (two) weight_chunk<F16>(np, k, d1, wb);
    if constexpr (INTER) {
      const int live = min(8, max(0, half - 8 * c));  // pairs of the column that turn
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // elements 2j', 2j'+1 of a chunk are a pair: other = element j ^ 1
        const float2 u = j / 2 < live ? sc[8 * c + j / 2] : make_float2(1.f, 0.f);
        const float2 v = 4 + j / 2 < live ? sc[8 * c + 4 + j / 2] : make_float2(1.f, 0.f);
        ca[j] = wa[j] * u.x;
        cb[j] = wa[j ^ 1] * (j & 1 ? u.y : -u.y);
        ce[j] = wb[j] * v.x;
        cf[j] = wb[j ^ 1] * (j & 1 ? v.y : -v.y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 u = c < rcols ? sc[8 * c + j] : make_float2(1.f, 0.f);
        ca[j] = wa[j] * u.x;
        cb[j] = -wb[j] * u.y;
        ce[j] = wb[j] * u.x;
        cf[j] = wa[j] * u.y;
      }
    }
  };
  bool now_k = part * side + hs >= p.num_qo_heads;
  coefficients(now_k);
  // heads in turn, each one's place in the ring taken by the load of the one kBatch on
  for (int hb = part * side; hb < heads;) {  // (the whole warp together)
#pragma unroll
    for (int k = 0; k < kBatch; ++k, hb += step) {
      if (hb >= heads) break;
      const int h = hb + hs;
      float x[16];
      unpack_chunk<F16>(va[k], x);
      unpack_chunk<F16>(vb[k], x + 8);
      load(h + kBatch * step, va[k], vb[k]);
      const float r = head_factor<F16>(np, x, wide, inv_dim);
      if (h < heads && !idle) {
        if (h >= p.num_qo_heads && !now_k) {
          now_k = true;
          coefficients(true);
        }
        float ya[8], yb[8];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= r;  // (first: products of tiny values lose bits)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ya[j] = fmaf(x[j], ca[j], (INTER ? x[j ^ 1] : x[8 + j]) * cb[j]);
          yb[j] = fmaf(x[8 + j], ce[j], (INTER ? x[8 + (j ^ 1)] : x[j]) * cf[j]);
        }
        uint16_t* out = row_of(p, t, h).out;
        store_chunk<F16>(out + d0, ya);
        if (two) store_chunk<F16>(out + d1, yb);
      }
    }
  }
}

// The half layout where R/2 is not a multiple of 8 (as rope_odd_kernel): whole
// columns, CP of them a lane, and the other halves of the pairs from shared memory.  One
// head's loads are in flight (a rare layout): 16384 tokens x 40 heads of 128, 24 dims that turn,
// 158 us (60 for 32 dims, in norm_rope_kernel), 211 tokens x 18 heads of 256, 72 dims, 7.4.
template <bool F16, int CP>
__global__ void __launch_bounds__(32) norm_rope_odd_kernel(const NormRopeParams np, int splits) {
  __shared__ __align__(16) float2 sc[kMaxPairs];
  __shared__ float rows[256 * CP];  // the heads of a step side by side
  const RopeParams& p = np.rope;
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x / splits;
  const int part = static_cast<int>(blockIdx.x % splits);
  const int heads = p.num_qo_heads + p.num_kv_heads, half = p.rotary_dim / 2;
  const int cols = p.head_dim / 8, wide = lanes_for(min(32, cols));
  const int side = 32 / wide, step = splits * side;
  const int hs = lane / wide, col = lane % wide;
  const float inv_dim = 1.f / static_cast<float>(p.head_dim);
  float* row = rows + hs * p.head_dim;  // (side heads of head_dim <= 256 CP / side dims)
  angles(p, t, sc, lane);
  auto other = [&](int d) { return d < half ? d + half : d - half; };
  float ca[CP][8] = {}, cb[CP][8] = {};
  auto coefficients = [&](bool k) {
#pragma unroll
    for (int c = 0; c < CP; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = 8 * (col + 32 * c) + j;
        ca[c][j] = cb[c][j] = 0.f;
        if (d >= p.head_dim) continue;
        const bool turns = d < 2 * half;
        const float2 u = turns ? sc[d < half ? d : d - half] : make_float2(1.f, 0.f);
        ca[c][j] = weight<F16>(np, k, d) * u.x;
        if (turns) cb[c][j] = weight<F16>(np, k, other(d)) * (d < half ? -u.y : u.y);
      }
  };
  bool now_k = part * side + hs >= p.num_qo_heads;
  if (part * side + hs < heads) coefficients(now_k);  // (others may have no weights either)
  for (int hb = part * side; hb < heads; hb += step) {  // (the whole warp together)
    const int h = hb + hs;
    float x[8 * CP];
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      Chunk v{};
      if (h < heads && col + 32 * c < cols)
        v = load_chunk(row_of(p, t, h).in + 8 * (col + 32 * c));
      unpack_chunk<F16>(v, x + 8 * c);
    }
    const float r = head_factor<F16>(np, x, wide, inv_dim);
#pragma unroll
    for (int j = 0; j < 8 * CP; ++j) x[j] *= r;
    __syncwarp();  // the last step's rows have been read
#pragma unroll
    for (int c = 0; c < CP; ++c)
      if (col + 32 * c < cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) row[8 * (col + 32 * c) + j] = x[8 * c + j];
      }
    __syncwarp();
    if (h >= heads) continue;  // (no lane waits in what follows until the next step)
    if (h >= p.num_qo_heads && !now_k) {
      now_k = true;
      coefficients(true);
    }
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      if (col + 32 * c >= cols) continue;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = 8 * (col + 32 * c) + j;
        const float z = d < 2 * half ? row[other(d)] : 0.f;
        y[j] = fmaf(x[8 * c + j], ca[c][j], z * cb[c][j]);
      }
      store_chunk<F16>(row_of(p, t, h).out + 8 * (col + 32 * c), y);
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& np, cudaStream_t stream) {
  const RopeParams& p = np.rope;
  const int heads = p.num_qo_heads + p.num_kv_heads;
  if (p.num_tokens == 0 || heads == 0) return cudaSuccess;
  const bool odd = !p.interleaved && p.rotary_dim % 16 != 0;
  // heads over several warps while the tokens alone are few
  const int cols = odd ? p.head_dim / 8 : rope_columns(p);
  const int side = cols >= 32 ? 1 : 32 / lanes_for(cols);
  const int most = (heads + side - 1) / side;
  const int64_t want = ((int64_t)kFewest + p.num_tokens - 1) / p.num_tokens;
  const int splits = want < most ? static_cast<int>(want) : most;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.num_tokens) * splits);
  auto launch = [&](auto* bf16, auto* f16) {
    (p.f16 ? f16 : bf16)<<<grid, 32, 0, stream>>>(np, splits);
  };
  if (odd && cols > 32)
    launch(norm_rope_odd_kernel<false, 2>, norm_rope_odd_kernel<true, 2>);
  else if (odd)
    launch(norm_rope_odd_kernel<false, 1>, norm_rope_odd_kernel<true, 1>);
  else if (p.interleaved)
    launch(norm_rope_kernel<false, true>, norm_rope_kernel<true, true>);
  else
    launch(norm_rope_kernel<false, false>, norm_rope_kernel<true, false>);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
