// e4m3_append.cu -- new tokens into a paged cache of E4M3 codes with one
// float32 scale per page and kv head, sm_103a.
//
// A block is one page of one kv head of K or V.  A step that writes its slots
// [a, z) computes, with m the largest finite |x| of the new elements,
//   w = 2^e, the smallest e in [-64, 64] with 448 * 2^e >= m (e = -64 for m = 0),
//   s = w for a = 0, else max(s_old, w);
//   new codes  E4M3_RNE_satfinite(x / s);
//   where s > s_old and a > 0, slots [0, a) are coded anew: E4M3_RNE(code * (s_old / s)).
// Powers of two lose nothing against m / 448 (codes have their own exponent;
// the block's largest code lies in (224, 448]), make x / s and the re-coding
// of normal codes exact, and leave every rounding one decision of the
// hardware's conversion from float32: x / s is exact but for results below
// 2^-126, far under the smallest code's half step.  A scale that something
// else has put in the cache need not be a power of two: x / s is then one
// correctly rounded division before the conversion.
//
// Bound by HBM (2 B in, 1 B out an element) for prompts, by latency for a
// decode step.  A warp owns a block: its new elements stay in registers
// between the maximum (on the packed 16-bit patterns) and the conversion, so
// each is read once, and no other warp touches the block.  The rows' loads do
// not wait for the page id, which is on its way together with them.  Measured
// (replayed): 7 prompt chunks, 10.5 thousand tokens of 8 heads x (128 + 128),
// 16.6 us, 3.7 TB/s: the request list's loads and sums come first (4 us), then
// each warp's blocks in turn, a load's latency each; 16 requests of one token
// 6.2 us, a launch and four dependent loads.
#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "internal.h"

namespace nvfp4kv {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
using dev::unpack2;

// two E4M3 codes, a in the low byte
__device__ __forceinline__ uint32_t code2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// 2^e: the smallest power of two with 448 * 2^e >= m, e in [-64, 64].
// 448 = 1.75 * 2^8, so for m = f * 2^k (1 <= f < 2) e is k - 8, or k - 7 where
// f > 1.75.
__device__ __forceinline__ float scale_for(uint32_t m_bits) {
  int e = static_cast<int>(m_bits >> 23) - 127 - 8 + ((m_bits & 0x7FFFFFu) > 0x600000u);
  e = max(-64, min(64, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A lane keeps one 16-byte column of the new rows (two where a row has more
// than 32, CP) and every rpp-th row: NCH chunks, 16 rows at most.
template <bool F16, int NCH, int CP>
__device__ __forceinline__ void append_block(const E4m3AppendParams& p, int kv, int h,
                                             const int32_t* page_at, int a, int z, int64_t row0,
                                             int lane) {
  const int cols = p.dim[kv] / 8, wide = min(32, cols), rpp = 32 / wide;
  const int col = lane % wide, r0 = lane / wide, rows = r0 < rpp ? z - a : 0;
  const uint16_t* src = p.src[kv] + (row0 + r0) * p.src_tok[kv] + h * p.src_head[kv] + 8 * col;
  uint4 v[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int r = (i / CP) * rpp, c = (i % CP) * 256;  // row step, column step
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < rows && 8 * col + c < p.dim[kv])
      v[i] = *reinterpret_cast<const uint4*>(src + r * p.src_tok[kv] + c);
  }
  const int page = *page_at;  // on its way together with the rows
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0 && p.flags) atomicOr(p.flags, 0x2u);
    return;
  }
  uint8_t* dst = p.data[kv] + page * p.sp[kv] + h * p.sh[kv] + 8 * col;
  float* sc = reinterpret_cast<float*>(p.scale[kv] + page * p.scp[kv] + h * p.sch[kv]);
  float s_old = a > 0 ? *sc : 0.f;
  // largest |x|, two 16-bit patterns at a time (their order is that of the
  // sizes); non-finite values are left out only when there are any
  constexpr uint32_t kInf = F16 ? 0x7C00u : 0x7F80u;
  auto largest = [&](auto keep) {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, keep(w[j] & 0x7FFF7FFFu));
    }
    return __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  };
  uint32_t m = largest([](uint32_t w) { return w; });
  if (m >= kInf)
    m = largest([](uint32_t w) { return w & __vcmpltu2(w, kInf | (kInf << 16)); });
  m = __float_as_uint(unpack2<F16>(m).x);
  float s = scale_for(m);
  if (a > 0) {
    // no scale of this format: the nearer end, as the attention takes it (the
    // lower for a NaN)
    const float c_old = dev::clamped_scale(s_old);
    if (c_old != s_old && lane == 0 && p.flags) atomicOr(p.flags, 0x20u);
    s_old = c_old;
    s = fmaxf(s, s_old);
    if (s > s_old && r0 < rpp) {
      const float f = __fdiv_rn(s_old, s);
      for (int r = r0; r < a; r += rpp)
        for (int c = 0; 8 * col + c < p.dim[kv]; c += 256) {
          uint2* at = reinterpret_cast<uint2*>(dst + r * p.ss[kv] + c);
          const uint2 old = *at;
          const uint32_t w[2] = {old.x, old.y};
          uint32_t o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 lo = unpack2<true>(dev::e4m3x2_to_f16x2(w[j] & 0xFFFFu));
            const float2 hi = unpack2<true>(dev::e4m3x2_to_f16x2(w[j] >> 16));
            o[j] = code2(lo.x * f, lo.y * f) | (code2(hi.x * f, hi.y * f) << 16);
          }
          *at = make_uint2(o[0], o[1]);
        }
    }
  }
  dst += (a + r0) * p.ss[kv];
  auto store = [&](auto scaled) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int r = (i / CP) * rpp, c = (i % CP) * 256;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = unpack2<F16>(w[j]);
        o[j] = code2(scaled(x.x), scaled(x.y));
      }
      if (r0 + r < rows && 8 * col + c < p.dim[kv])
        *reinterpret_cast<uint2*>(dst + r * p.ss[kv] + c) =
            make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
  };
  if ((__float_as_uint(s) & 0x7FFFFFu) == 0) {  // a power of two: its reciprocal is exact
    const float inv = __uint_as_float((254u << 23) - (__float_as_uint(s) & 0x7F800000u));
    store([inv](float x) { return x * inv; });
  } else {
    store([s](float x) { return __fdiv_rn(x, s); });
  }
  if (lane == 0) *sc = s;
}

// 1-token pages: a block is one row, too little for a warp.  A warp takes a
// token's K or V: W lanes (4, 8, 16 or 32, a row's 16-byte columns rounded up) a
// head, 32 / W heads side by side, U such steps' loads in flight.  CP chunks of a
// row a lane (2 where it has more than 32).  8192 tokens x 8 heads x (128 + 128)
// in 21 us, 2.4 TB/s (a warp a block: 66 us).
template <bool F16, int U, int CP>
__device__ __forceinline__ void append_rows(const E4m3AppendParams& p, int kv,
                                            const int32_t* page_at, int64_t row, int lane) {
  constexpr uint32_t kInf = F16 ? 0x7C00u : 0x7F80u;
  const int cols = p.dim[kv] / 8, H = p.num_kv_heads;
  int W = 32;
  while (W / 2 >= cols) W /= 2;
  const int side = 32 / W, col = lane % W;
  const uint16_t* src = p.src[kv] + row * p.src_tok[kv] + 8 * col;
  int page = 0;
  for (int h0 = lane / W; h0 - lane / W < H; h0 += U * side) {  // (the whole warp together)
    uint4 v[U][CP];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        v[u][c] = make_uint4(0u, 0u, 0u, 0u);
        const uint16_t* from = src + (h0 + u * side) * p.src_head[kv] + 256 * c;
        if (h0 + u * side < H && col + 32 * c < cols) v[u][c] = *reinterpret_cast<const uint4*>(from);
      }
    if (h0 == lane / W) {
      page = *page_at;  // on its way together with the first rows
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0 && p.flags) atomicOr(p.flags, 0x2u);
        return;
      }
    }
    uint8_t* dst = p.data[kv] + page * p.sp[kv] + 8 * col;
    uint8_t* sc = p.scale[kv] + page * p.scp[kv];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * side;
      auto largest = [&](auto keep) {
        uint32_t m2 = 0;
#pragma unroll
        for (int c = 0; c < CP; ++c) {
          const uint32_t w[4] = {v[u][c].x, v[u][c].y, v[u][c].z, v[u][c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, keep(w[j] & 0x7FFF7FFFu));
        }
        uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
        for (int o = W / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
      };
      uint32_t m = largest([](uint32_t w) { return w; });
      if (__any_sync(0xffffffffu, m >= kInf))
        m = largest([](uint32_t w) { return w & __vcmpltu2(w, kInf | (kInf << 16)); });
      const float s = scale_for(__float_as_uint(unpack2<F16>(m).x));
      const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));  // a power of two
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const uint32_t w[4] = {v[u][c].x, v[u][c].y, v[u][c].z, v[u][c].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<F16>(w[j]);
          o[j] = code2(x.x * inv, x.y * inv);
        }
        if (h < H && col + 32 * c < cols)
          *reinterpret_cast<uint2*>(dst + h * p.sh[kv] + 256 * c) =
              make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
      }
      if (h < H && col == 0) *reinterpret_cast<float*>(sc + h * p.sch[kv]) = s;
    }
  }
}

// The (page, head, K or V) blocks of all requests (1-token pages: the (page, K or
// V) ones) form one list; warp w of the
// grid takes its entries w, w + W, ... (a CTA grid over requests would leave
// most CTAs without work when their lengths differ).  The requests pass through
// shared memory kThreads at a time: first row, tokens before the step and
// first page of each, and the sum of the pages that those before it write.
template <bool F16, int NCH, int CP, bool P1>
__global__ void __launch_bounds__(kThreads, NCH <= 8 ? 6 : NCH <= 16 ? 4 : 2)
    e4m3_append_kernel(const E4m3AppendParams p) {
  __shared__ int s_row[kThreads], s_new[kThreads], s_kv[kThreads], s_page[kThreads];
  __shared__ int64_t s_begin[kThreads], s_first[kThreads + 1], s_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = P1 ? 2 : 2 * p.num_kv_heads;
  // this warp's next entry: block r of the list's page c (stepped without a
  // division)
  const int wid = blockIdx.x * kWarps + warp, W = gridDim.x * kWarps;
  const int wc = W / blocks, wr = W % blocks;
  int64_t c = wid / blocks;
  int r = wid % blocks;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int count = 0;
    if (b < p.batch) {
      const int r0 = p.qo_indptr[b], r1 = p.qo_indptr[b + 1];
      const int k0 = p.kv_indptr[b], k1 = p.kv_indptr[b + 1], last = p.last_page_len[b];
      const int64_t n = (int64_t)r1 - r0, np = (int64_t)k1 - k0;
      const int64_t len = (np - 1) * p.page_size + last, begin = len - n;
      if (n != 0) {
        if (r0 < 0 || n < 0 || r1 > p.num_rows || k0 < 0 || np < 1 || last < 1 ||
            last > p.page_size || begin < 0) {
          if (blockIdx.x == 0 && p.flags) atomicOr(p.flags, 0x2u);
        } else {
          const int first = static_cast<int>(begin / p.page_size);
          count = static_cast<int>(np) - first;
          s_row[tid] = r0;
          s_new[tid] = static_cast<int>(n);
          s_kv[tid] = k0 + first;
          s_begin[tid] = begin;
          s_page[tid] = first;
        }
      }
    }
    int64_t sum = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) sum += s_sum[w];
    s_first[tid] = sum - count;
    if (tid == kThreads - 1) s_first[kThreads] = sum;
    __syncthreads();
    const int64_t pages = s_first[kThreads];
    while (c < pages) {
      int lo = 0, hi = kThreads;  // the request whose pages hold entry c
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= c) lo = mid; else hi = mid;
      }
      const int64_t begin = s_begin[lo], len = begin + s_new[lo];
      const int64_t pos = (s_page[lo] + c - s_first[lo]) * p.page_size;
      const int32_t* page_at = p.kv_indices + s_kv[lo] + c - s_first[lo];
      if constexpr (P1) {
        append_rows<F16, NCH, CP>(p, r, page_at, s_row[lo] + pos - begin, lane);
      } else {
        const int a = static_cast<int>(max(begin - pos, (int64_t)0));
        const int z = static_cast<int>(min(len - pos, (int64_t)p.page_size));
        append_block<F16, NCH, CP>(p, r & 1, r >> 1, page_at, a, z, s_row[lo] + pos + a - begin,
                                   lane);
      }
      c += wc;
      r += wr;
      if (r >= blocks) {
        r -= blocks;
        ++c;
      }
    }
    c -= pages;  // counted from the next requests' first page
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_e4m3_append(const E4m3AppendParams& p, cudaStream_t stream) {
  if (p.num_rows == 0 || p.batch == 0) return cudaSuccess;
  // every row may open a page of its own, else a request's rows fill theirs but
  // for two: as many warps as blocks at most, and a wave of CTAs
  int64_t pages = p.num_rows / p.page_size + 2 * (int64_t)p.batch;
  if (pages > p.num_rows) pages = p.num_rows;
  int64_t grid = (pages * 2 * (p.page_size == 1 ? 1 : p.num_kv_heads) + kWarps - 1) / kWarps;
  if (grid > 152 * 6) grid = 152 * 6;
  const int dmax = p.dim[0] > p.dim[1] ? p.dim[0] : p.dim[1];
#define NVFP4KV_E4M3_APPEND(NCH_, CP_, P1_)                                                   \
  (p.f16 ? e4m3_append_kernel<true, NCH_, CP_, P1_>                                           \
         : e4m3_append_kernel<false, NCH_, CP_, P1_>)<<<static_cast<int>(grid), kThreads, 0,   \
                                                        stream>>>(p)
  if (p.page_size == 1 && dmax <= 256)
    NVFP4KV_E4M3_APPEND(4, 1, true);
  else if (p.page_size == 1)
    NVFP4KV_E4M3_APPEND(2, 2, true);
  else if (dmax <= 64)
    NVFP4KV_E4M3_APPEND(4, 1, false);
  else if (dmax <= 128)
    NVFP4KV_E4M3_APPEND(8, 1, false);
  else if (dmax <= 256)
    NVFP4KV_E4M3_APPEND(16, 1, false);
  else
    NVFP4KV_E4M3_APPEND(32, 2, false);
#undef NVFP4KV_E4M3_APPEND
  return cudaGetLastError();
}

}  // namespace nvfp4kv
