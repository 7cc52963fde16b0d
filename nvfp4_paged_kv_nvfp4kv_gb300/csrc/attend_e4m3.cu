// attend_e4m3.cu -- attention over a paged cache of E4M3 codes with one scale
// per page and kv head, blocks of 8 or 16 query rows, sm_103a.
//
// With a_j, b_j the K and V scale of token j's page and c_j, d_j its codes:
//   s_j = sm_scale * a_j * (q . c_j),  o = sum_j p_j b_j d_j / sum_j p_j,
//   p_j = exp(s_j), over the keys that the row sees; lse = ln sum_j p_j.
//  * Codes are exact in f16 (cvt.rn.f16x2.e4m3x2), so both products run on
//    mma.sync m16n8k16 with f16 operands and f32 accumulators, and no element
//    is multiplied by a scale: a_j multiplies the score, b_j the weight.
//    m follows x_j + log2 b_j, x_j the score in log2 units: y_j = 2^(x_j - m)
//    goes into the row sum and p'_j = y_j b_j <= 2^8, rounded to f16, weighs the
//    codes.  y lies in [0, 2^72] and the largest of a row is at least 2^-64, so
//    float32 keeps every term of the sum that counts (a term taken as p'_j / b_j
//    is lost where p' underflows, from scales 2^116 apart on).  The sum's factors
//    2^(m - m_new) are taken as two halves: m may move by 2^128 without a score
//    changing.  f16 for p' is the rounding of 2^-11 that the product's operand
//    type costs; the row sum takes the float32 y.  (p' in two f16 pieces, 2^-22:
//    45.6 -> 46.2 us on 4 requests of 32771 tokens, 17.3 -> 18.2 on 16 of 512-4096,
//    with 16 rows 52.5 -> 59.1, for an error that an output's own rounding hides.)
//  * A warp owns every WARPS-th tile of 16 tokens (one page, or sixteen
//    1-token pages) and streams its K rows, V rows and scales through a ring
//    of STAGES stages with cp.async, rows and pages at any byte strides.
//  * S^T = C Q^T (M = 16 tokens, N = 8 query rows, once or twice): a lane's 16 contiguous
//    bytes of a K row are the A operand of four k-steps under a permutation
//    of the dims that Q's fragments share.  O^T += D^T P'^T with P' kept in
//    registers (movmatrix); the A operand interleaves two V rows bytewise.
//  * K chunks are stored xor 4 on odd rows and V chunks xor the row's bits
//    1-2, and a tile's tokens are taken in the order m -> m ^ ((m >> 1) & 1),
//    so the lanes' 16-byte reads hit distinct banks.
//  * The maximum is raised only when a value exceeds it by more than 2^8.
//  * NaN: a NaN score makes its row NaN.  A weight of 0 would carry a NaN value
//    code into the rows that do not see its token, so in tiles that some row
//    does not see whole the codes are taken out of the product, and the first
//    such token of each value dim makes that dim NaN in the rows that see it.
// HBM bounds it: Dk + Dv bytes a token and kv head.  Measured (replayed): 4
// requests of 32771 tokens, 8 kv heads of 128, 49.7 us, 5.4 TB/s (0.81 of a plain
// copy; the tile loop alone runs at 7); 16 of 512-4096 tokens 20.6 us, 3.6 TB/s:
// 4 us of launch, 3 to the first tile, 9 of loop, 2.4 of combining and folding the
// splits; 8 of 2048-8192 tokens at 512 / 256 dims 22 us, 2.9 TB/s; two short
// requests 6.2 us.  The same 4 requests, calls back to back in one graph (128/128
// 45.6 us), at 64/64, 256/128, 256/256, 512/256: 26.8, 63.7, 86.4, 118.7 us, 0.75 to
// 1.0 of a copy; with 1-token pages, a row's address and page id each: 42.3 (64/64),
// 64.0 (128/128), 110 (256/256), 146 us (512/256).
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "epilogue.cuh"
#include "internal.h"

namespace nvfp4kv {
namespace {

using namespace dev;

constexpr float kRaiseLog2 = 8.f;

template <int DK, int DV, int WARPS, int STAGES, int NT>
struct E4Traits {
  static constexpr int RB = 8 * NT;                   // query rows: NT product columns of 8
  static constexpr int K_BYTES = 16 * DK, V_BYTES = 16 * DV;
  static constexpr int OFF_V = K_BYTES, OFF_SC = OFF_V + V_BYTES;  // 16 K scales, 16 V scales
  static constexpr int STAGE_BYTES = OFF_SC + 128;
  static constexpr int KCH = DK / 64;                 // 16-byte chunks of a K row per lane
  static constexpr int KSTEPS = DK / 16;
  static constexpr int VCB = DV >= 128 ? 16 : DV / 8;  // V bytes per lane per chunk
  static constexpr int VCH = DV / 8 / VCB;            // V chunks per lane
  static constexpr int MT = DV / 16;                  // PV m-tiles
  static constexpr int PIPE_BYTES = WARPS * STAGES * STAGE_BYTES;
  static constexpr int OS = DV + 4;                   // row stride of the warps' results
  static constexpr int COMB_BYTES = WARPS * RB * (OS + 2) * 4;
  static constexpr int MAIN_BYTES = PIPE_BYTES > COMB_BYTES ? PIPE_BYTES : COMB_BYTES;
  static constexpr int QROW = DK + 8;                 // f16 elements, padded
  static constexpr int OFF_Q = MAIN_BYTES;
  static constexpr int OFF_ROW = OFF_Q + RB * QROW * 2;
  static constexpr int OFF_NAN = OFF_ROW + 2 * RB * 4 + 16;  // [DV] first NaN token taken out
  static constexpr int SMEM = OFF_NAN + DV * 4;
  static_assert(DK % 64 == 0 && DV % 64 == 0, "head dims");
};

__device__ __forceinline__ int tok_of(int m) { return m ^ ((m >> 1) & 1); }

// physical 16-byte chunk of logical chunk ch of row r
template <int DK>
__device__ __forceinline__ int k_pos(int r, int ch) {
  return DK >= 128 ? ch ^ ((r & 1) << 2) : ch;
}
template <int DV>
__device__ __forceinline__ int v_pos(int r, int ch) {
  return DV >= 128 ? ch ^ (r & 6) : ch ^ ((r >> 1) & 2);
}

__device__ __forceinline__ float lds_f32(uint32_t a) { return __uint_as_float(lds_u32<0>(a)); }

// the scale, or the nearer end of the range with the flag set
__device__ __forceinline__ float checked_scale(float s, uint32_t* flags) {
  const float c = clamped_scale(s);
  if (c != s) atomicOr(flags, 0x20u);
  return c;
}

// P1: 1-token pages
template <int DK, int DV, int WARPS, int STAGES, int NT, int MINB, bool P1>
__global__ void __launch_bounds__(WARPS * 32, MINB) attend_e4m3_kernel(const AttendParams p) {
  using T = E4Traits<DK, DV, WARPS, STAGES, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint16_t* sQ = reinterpret_cast<uint16_t*>(smem + T::OFF_Q);
  float* sRowF = reinterpret_cast<float*>(smem + T::OFF_ROW);
  int* sRowLim = reinterpret_cast<int*>(sRowF + T::RB);
  int* sNan = reinterpret_cast<int*>(smem + T::OFF_NAN);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const WorkUnit u = load_unit(p);
  const int G = p.group, R = G * u.qo_len;
  const int row0 = blockIdx.y * T::RB;
  if (row0 >= R) return;
  const int ntiles = P1 ? (u.num_pages + 15) / 16 : u.num_pages;
  const int npw = ntiles > warp ? (ntiles - warp + WARPS - 1) / WARPS : 0;
  const int32_t* pidx = p.kv_indices + u.page_begin;
  const CacheView& c = p.cache;

  // Page ids: 16-token pages, lane k holds the page of this warp's tile
  // 32 blk + k; 1-token pages, lane r (and r + 16) the page of row r of the
  // tile to be copied next.  An id out of the pool reads page 0, flagged.
  auto checked = [&](int32_t id) -> int32_t {
    if (id < 0 || id >= c.num_pages) {
      atomicOr(p.flags, 0x1u);
      return 0;
    }
    return id;
  };
  auto load_ids = [&](int blk) -> int32_t {
    int32_t id = 0;
    if constexpr (P1) {
      const int j = (warp + blk * WARPS) * 16 + (lane & 15);
      if (blk < npw) id = checked(__ldg(pidx + min(j, u.num_pages - 1)));
    } else {
      const int j = 32 * blk + lane;
      if (j < npw) id = checked(__ldg(pidx + warp + j * WARPS));
    }
    return id;
  };
  int32_t ids_cur = load_ids(0);
  int32_t ids_nxt = (P1 || npw > 32) ? load_ids(1) : 0;

  // ---- Q rows -------------------------------------------------------------
  constexpr int QCH = T::RB * DK / 8;
  constexpr int QPT = (QCH + WARPS * 32 - 1) / (WARPS * 32);
  uint4 qv[QPT];
#pragma unroll
  for (int k = 0; k < QPT; ++k) {
    const int ci = tid + k * WARPS * 32;
    const int r = row0 + ci / (DK / 8);
    qv[k] = make_uint4(0u, 0u, 0u, 0u);
    if (ci < QCH && r < R)
      qv[k] = *reinterpret_cast<const uint4*>(p.q + (int64_t)(u.qo_begin + r / G) * p.q_stride_tok +
                                              (int64_t)(u.h_kv * G + r % G) * p.q_stride_head +
                                              (ci % (DK / 8)) * 8);
  }
  if (tid < T::RB) reinterpret_cast<int*>(sRowF)[tid] = 0;  // per-row amax bits
  for (int d = tid; d < DV; d += WARPS * 32) sNan[d] = INT_MAX;
  __syncthreads();

  // ---- the tile pipeline ---------------------------------------------------
  const uint32_t ring = smem_addr(smem) + warp * STAGES * T::STAGE_BYTES;
  const uint8_t* kb = c.k_data + (int64_t)u.h_kv * c.k_sh;
  const uint8_t* vb = c.v_data + (int64_t)u.h_kv * c.v_sh;
  // scales: lanes 0-15 K, 16-31 V, of the page that holds row lane & 15
  const uint8_t* scb = lane < 16 ? c.k_sf + (int64_t)u.h_kv * c.ksf_sh
                                 : c.v_sf + (int64_t)u.h_kv * c.vsf_sh;
  const int64_t scp = lane < 16 ? c.ksf_sp : c.vsf_sp;
  constexpr int KR = DK / 16, VR = DV / 16;          // 16-byte chunks of a row
  constexpr int KN = KR / 2, VN = VR / 2;            // copies per lane
  constexpr int KRI = 32 / KR > 0 ? 32 / KR : 1;     // rows a copy of the warp covers
  constexpr int VRI = 32 / VR > 0 ? 32 / VR : 1;
  static_assert(KR <= 32 && VR <= 32, "row chunks");
  const int kr = lane / KR, kc = lane % KR, vr = lane / VR, vc = lane % VR;
  // the pages of the tile in a lane's page register
  auto issue = [&](int32_t ids, int jl, int js) {
    const uint32_t st = ring + js * T::STAGE_BYTES;
    const int32_t pg = P1 ? 0 : __shfl_sync(0xffffffffu, ids, jl & 31);
    const uint8_t* kpage = kb + (int64_t)pg * c.k_sp + 16 * kc;
    const uint8_t* vpage = vb + (int64_t)pg * c.v_sp + 16 * vc;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
      const int r = kr + i * KRI;
      const uint8_t* src = P1 ? kpage + (int64_t)__shfl_sync(0xffffffffu, ids, r) * c.k_sp
                              : kpage + r * c.k_ss;
      cp_async_16s(st + r * DK + 16 * k_pos<DK>(r, kc), src);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int r = vr + i * VRI;
      const uint8_t* src = P1 ? vpage + (int64_t)__shfl_sync(0xffffffffu, ids, r) * c.v_sp
                              : vpage + r * c.v_ss;
      cp_async_16s(st + T::OFF_V + r * DV + 16 * v_pos<DV>(r, vc), src);
    }
    cp_async_4s(st + T::OFF_SC + 4 * lane, scb + (int64_t)(P1 ? ids : pg) * scp);
    cp_async_commit();
  };
  // tile j of this warp into stage js; ids for it are in ids_cur
  auto advance = [&](int j, int js) {
    if (j < npw) {
      issue(ids_cur, j, js);
      if (P1 || (j & 31) == 31) {
        ids_cur = ids_nxt;
        ids_nxt = load_ids(P1 ? j + 2 : j / 32 + 2);
      }
    } else {
      cp_async_commit();  // one group per tile for the wait count
    }
  };
#pragma unroll
  for (int j = 0; j < STAGES - 1; ++j) advance(j, j);

  // ---- Q: per-row power-of-two prescale into f16, row limits ---------------
  auto q2 = [&](uint32_t w) -> float2 {
    return p.q_f16 ? unpack2<true>(w) : unpack2<false>(w);
  };
#pragma unroll
  for (int k = 0; k < QPT; ++k) {
    const int ci = tid + k * WARPS * 32;
    if (ci >= QCH) continue;
    const uint32_t w[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
    float am = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = q2(w[j]);
      am = fmaxf(am, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
    atomicMax(reinterpret_cast<int*>(sRowF) + ci / (DK / 8), __float_as_int(am));
  }
  __syncthreads();
  float rowf[QPT];
#pragma unroll
  for (int k = 0; k < QPT; ++k) {
    const int ci = tid + k * WARPS * 32;
    if (ci >= QCH) continue;
    const int rr = ci / (DK / 8), r = row0 + rr;
    const float amax = __int_as_float(reinterpret_cast<const int*>(sRowF)[rr]);
    int e = 0;  // amax * 2^e in [2^14, 2^15)
    if (amax > 0.f) e = 14 - (int)((__float_as_uint(amax) >> 23) & 0xFF) + 127;
    e = max(-120, min(120, e));
    // (an infinite element makes its row NaN, as 0 * inf does)
    const float up = isinf(amax) ? NAN : __uint_as_float((uint32_t)(127 + e) << 23);
    const uint32_t w[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = q2(w[j]);
      h[j] = f32x2_to_f16x2(x.x * up, x.y * up);
    }
    *reinterpret_cast<uint4*>(sQ + rr * T::QROW + (ci % (DK / 8)) * 8) =
        make_uint4(h[0], h[1], h[2], h[3]);
    if (ci % (DK / 8) == 0)
      sRowLim[rr] = r >= R ? -1 : (p.causal ? (u.kv_len - u.qo_len + r / G) : (u.kv_len - 1));
    rowf[k] = r >= R ? 0.f : p.qk_scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < QPT; ++k) {
    const int ci = tid + k * WARPS * 32;
    if (ci < QCH && ci % (DK / 8) == 0) sRowF[ci / (DK / 8)] = rowf[k];
  }
  __syncthreads();

  // this lane's query rows 8 n + 2t and 8 n + 2t + 1 (k = 2 n and 2 n + 1):
  // score factor, -m (m the running maximum of score + log2 b, once the row has
  // one: bit k of has_max) and sum
  constexpr int NR = 2 * NT;
  float f2[NR], nm2[NR], lrow[NR];
  int lim[NR];
  uint32_t has_max = 0;
  int min_lim = u.kv_len - 1;
  for (int rr = 0; rr < T::RB; ++rr)
    if (sRowLim[rr] >= 0) min_lim = min(min_lim, sRowLim[rr]);
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int rr = 8 * (k / 2) + 2 * t + k % 2;
    f2[k] = sRowF[rr];
    lim[k] = sRowLim[rr];
    nm2[k] = 0.f;
    lrow[k] = 0.f;
  }
  auto lane_threshold = [&]() {
    float th = INFINITY;
#pragma unroll
    for (int k = 0; k < NR; ++k)
      th = fminf(th, (has_max >> k) & 1u ? kRaiseLog2 : (lim[k] >= 0 ? -INFINITY : INFINITY));
    return th;
  };
  float thr_lane = lane_threshold();
  bool saw_nan = false;  // a NaN value code was taken out of this lane's products
  // Q fragments: k-step 4 cc + m covers the 4 dims 16 (4 cc + t) + 4 m ..
  uint32_t qreg[NT][T::KSTEPS][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int kk = 0; kk < T::KSTEPS; ++kk) {
      const uint2 lo = *reinterpret_cast<const uint2*>(
          sQ + (8 * n + g) * T::QROW + 16 * (4 * (kk / 4) + t) + 4 * (kk % 4));
      qreg[n][kk][0] = lo.x;
      qreg[n][kk][1] = lo.y;
    }
  float oacc[NT][T::MT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
      for (int k = 0; k < 4; ++k) oacc[n][mt][k] = 0.f;

  // rows this lane reads: tokens of mma rows g, g + 8 (K) and of P columns
  // 2t, 2t + 1, 2t + 8, 2t + 9 (V)
  const int kr0 = tok_of(g), vt0 = tok_of(2 * t), vt1 = vt0 ^ 1;

#pragma unroll 1
  for (int i = 0; i < npw; ++i) {
    const int is = i % STAGES;
    cp_async_wait<STAGES - 2>();
    __syncwarp();  // the stage has landed; the one before it has been read
    advance(i + STAGES - 1, (i + STAGES - 1) % STAGES);
    const uint32_t st = ring + is * T::STAGE_BYTES;
    const int tok0 = u.tok_begin + (warp + i * WARPS) * 16;

    // ---- S^T = C Q^T ------------------------------------------------------
    float sa[NT][4] = {}, sb[NT][4] = {};
#pragma unroll
    for (int cc = 0; cc < T::KCH; ++cc) {
      const uint32_t ka = st + kr0 * DK + 16 * k_pos<DK>(kr0, 4 * cc + t);
      const uint4 a4 = lds_v4<0>(ka), b4 = lds_v4<8 * DK>(ka);
      const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t f[4];
        e4m3x4_to_f16(a[m], f[0], f[2]);
        e4m3x4_to_f16(b[m], f[1], f[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_16816(m & 1 ? sb[n] : sa[n], f, qreg[n][4 * cc + m][0], qreg[n][4 * cc + m][1]);
      }
    }
    // ---- the tile's scales: tokens kr0 (A) and kr0 + 8 (B) -----------------
    const uint32_t sc = st + T::OFF_SC + 4 * kr0;
    const float ksA = checked_scale(lds_f32(sc), p.flags);
    const float vsA = checked_scale(lds_f32(sc + 64), p.flags), lvA = log2_scale(vsA);
    const float ksB = P1 ? checked_scale(lds_f32(sc + 32), p.flags) : ksA;
    const float vsB = P1 ? checked_scale(lds_f32(sc + 96), p.flags) : vsA;
    const float lvB = P1 ? log2_scale(vsB) : lvA;
    // (the scale times the sum: times the factor it could pass float32's range
    // where the score does not)
    // x[n][0..3] = tokens kr0, kr0, kr0 + 8, kr0 + 8 x rows 2n, 2n+1, 2n, 2n+1
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[n][k] = fmaf((sa[n][k] + sb[n][k]) * (k < 2 ? ksA : ksB), f2[2 * n + (k & 1)],
                       nm2[2 * n + (k & 1)]);
    const bool masked = tok0 + 15 > min_lim;  // some row does not see some token
    if (masked) {
      const int ta = tok0 + kr0, tb = ta + 8;
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        if (ta > lim[k]) x[k / 2][k % 2] = -INFINITY;
        if (tb > lim[k]) x[k / 2][2 + k % 2] = -INFINITY;
      }
    }
    float topA = fmaxf(x[0][0], x[0][1]), topB = fmaxf(x[0][2], x[0][3]);
#pragma unroll
    for (int n = 1; n < NT; ++n) {
      topA = fmaxf(topA, fmaxf(x[n][0], x[n][1]));
      topB = fmaxf(topB, fmaxf(x[n][2], x[n][3]));
    }
    const float top = P1 ? fmaxf(topA + lvA, topB + lvB) : fmaxf(topA, topB) + lvA;
    if (__builtin_expect(__any_sync(0xffffffffu, top > thr_lane), 0)) {
      // raise each row's maximum to this tile's (a row's values sit in the 8
      // lanes of the same t)
      float corr[NR];
      bool moved = false;
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        float mx = fmaxf(x[k / 2][k % 2] + lvA, x[k / 2][2 + k % 2] + lvB);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float half = 1.f;  // the square root of the row's factor
        const bool has = (has_max >> k) & 1u;
        if (mx != -INFINITY && (!has || mx > 0.f)) {
          if (has) half = ex2(-0.5f * mx);
          nm2[k] -= mx;
          has_max |= 1u << k;
          x[k / 2][k % 2] -= mx;
          x[k / 2][2 + k % 2] -= mx;
        }
        lrow[k] = lrow[k] * half * half;
        corr[k] = half * half;
        moved |= half != 1.f;
      }
      thr_lane = lane_threshold();
      if (moved) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int mt = 0; mt < T::MT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) oacc[n][mt][k] *= corr[2 * n + (k & 1)];
      }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float y0 = ex2(x[n][0]), y1 = ex2(x[n][1]), y2 = ex2(x[n][2]), y3 = ex2(x[n][3]);
      lrow[2 * n] += y0 + y2;
      lrow[2 * n + 1] += y1 + y3;
      pf[n][0] = movmatrix_trans(f32x2_to_f16x2(y0 * vsA, y1 * vsA));
      pf[n][1] = movmatrix_trans(f32x2_to_f16x2(y2 * vsB, y3 * vsB));
    }

    // ---- O^T += D^T P'^T ----------------------------------------------------
    const int valid = u.kv_len - tok0;  // slots past it may hold a NaN code
#pragma unroll
    for (int cc = 0; cc < T::VCH; ++cc) {
      constexpr int VW = T::VCB / 4;
      uint32_t w[4][VW];  // tokens vt0, vt1, vt0 + 8, vt1 + 8
      if constexpr (T::VCB == 16) {
        const uint32_t a0 = st + T::OFF_V + vt0 * DV + 16 * v_pos<DV>(vt0, 8 * cc + g);
        const uint32_t a1 = st + T::OFF_V + vt1 * DV + 16 * v_pos<DV>(vt1, 8 * cc + g);
        const uint4 q0 = lds_v4<0>(a0), q1 = lds_v4<0>(a1);
        const uint4 q2v = lds_v4<8 * DV>(a0), q3 = lds_v4<8 * DV>(a1);
        w[0][0] = q0.x; w[0][1] = q0.y; w[0][2] = q0.z; w[0][3] = q0.w;
        w[1][0] = q1.x; w[1][1] = q1.y; w[1][2] = q1.z; w[1][3] = q1.w;
        w[2][0] = q2v.x; w[2][1] = q2v.y; w[2][2] = q2v.z; w[2][3] = q2v.w;
        w[3][0] = q3.x; w[3][1] = q3.y; w[3][2] = q3.z; w[3][3] = q3.w;
      } else {
        const uint32_t a0 = st + T::OFF_V + vt0 * DV + 16 * v_pos<DV>(vt0, g / 2) + 8 * (g & 1);
        const uint32_t a1 = st + T::OFF_V + vt1 * DV + 16 * v_pos<DV>(vt1, g / 2) + 8 * (g & 1);
        const uint2 q0 = lds_v2<0>(a0), q1 = lds_v2<0>(a1);
        const uint2 q2v = lds_v2<8 * DV>(a0), q3 = lds_v2<8 * DV>(a1);
        w[0][0] = q0.x; w[0][1] = q0.y;
        w[1][0] = q1.x; w[1][1] = q1.y;
        w[2][0] = q2v.x; w[2][1] = q2v.y;
        w[3][0] = q3.x; w[3][1] = q3.y;
      }
      if (masked) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = (j & 1 ? vt1 : vt0) + (j & 2) * 4;
          uint32_t nan = 0;
#pragma unroll
          for (int k = 0; k < VW; ++k) {
            if (tok >= valid) w[j][k] = 0;
            nan |= ((w[j][k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          }
          if (nan) {
            saw_nan = true;
            const int d0 = 128 * cc + g * T::VCB;
            for (int b = 0; b < T::VCB; ++b) {
#pragma unroll
              for (int k = 0; k < VW; ++k)  // (registers have no index)
                if (b / 4 == k && ((w[j][k] >> (8 * (b % 4))) & 0x7Fu) == 0x7Fu) {
                  w[j][k] &= ~(0xFFu << (8 * (b % 4)));
                  atomicMin(&sNan[d0 + b], tok0 + tok);
                }
            }
          }
        }
      }
      // m-tile of byte pair m: rows g and g + 8 are the dims of bytes 2m, 2m+1
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        const uint32_t l0 = __byte_perm(w[0][k], w[1][k], 0x5140);
        const uint32_t h0 = __byte_perm(w[0][k], w[1][k], 0x7362);
        const uint32_t l1 = __byte_perm(w[2][k], w[3][k], 0x5140);
        const uint32_t h1 = __byte_perm(w[2][k], w[3][k], 0x7362);
        const int mt = cc * (T::VCB / 2) + 2 * k;
        uint32_t fa[4], fb[4];
        e4m3x4_to_f16(l0, fa[0], fa[1]);
        e4m3x4_to_f16(l1, fa[2], fa[3]);
        e4m3x4_to_f16(h0, fb[0], fb[1]);
        e4m3x4_to_f16(h1, fb[2], fb[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816(oacc[n][mt], fa, pf[n][0], pf[n][1]);
          mma_16816(oacc[n][mt + 1], fb, pf[n][0], pf[n][1]);
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---- combine the warps ---------------------------------------------------
#pragma unroll
  for (int k = 0; k < NR; ++k)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) lrow[k] += __shfl_xor_sync(0xffffffffu, lrow[k], o);
  const bool any_nan = __syncthreads_or(saw_nan);  // every warp is done with its ring
  float* sO = reinterpret_cast<float*>(smem);   // [WARPS][RB][OS]
  float* sM = sO + WARPS * T::RB * T::OS;       // [WARPS][RB]
  float* sL = sM + WARPS * T::RB;               // [WARPS][RB]
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r0 = warp * T::RB + 8 * n + 2 * t;
    if (g == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // (a NaN sum counts whatever the maximum, which no NaN score raises)
        sM[r0 + k] = isnan(lrow[2 * n + k])               ? 0.f
                     : (has_max >> (2 * n + k)) & 1u ? -nm2[2 * n + k]
                                                          : -INFINITY;
        sL[r0 + k] = lrow[2 * n + k];
      }
    }
#pragma unroll
    for (int mt = 0; mt < T::MT; ++mt) {
      constexpr int PC = T::VCB / 2;  // m-tiles of a chunk
      const int d = (mt / PC) * 128 + g * T::VCB + 2 * (mt % PC);
      float* o0 = sO + r0 * T::OS + d;
      *reinterpret_cast<float2*>(o0) = make_float2(oacc[n][mt][0], oacc[n][mt][2]);
      *reinterpret_cast<float2*>(o0 + T::OS) = make_float2(oacc[n][mt][1], oacc[n][mt][3]);
    }
  }
  __syncthreads();
  if (any_nan) {
    for (int i = tid; i < WARPS * T::RB * DV; i += WARPS * 32) {
      const int rr = i / DV, d = i % DV;
      if (sRowLim[rr % T::RB] >= sNan[d]) sO[rr * T::OS + d] = NAN;
    }
    __syncthreads();
  }
  finish_rows<T::RB, DV, WARPS, T::OS>(p, u, row0, R, sM, sL, sO, sRowF);
}

template <int DK, int DV, int WARPS, int STAGES, int NT, int MINB>
bool make_e4m3(bool page1, AttendConfig* cfg) {
  using T = E4Traits<DK, DV, WARPS, STAGES, NT>;
  cfg->kind = kKernelE4m3;
  cfg->dk = DK;
  cfg->dv = DV;
  cfg->rows = T::RB;
  cfg->warps = WARPS;
  cfg->smem_bytes = T::SMEM;
  cfg->units_per_cta = 1;
  cfg->func =
      page1 ? reinterpret_cast<const void*>(attend_e4m3_kernel<DK, DV, WARPS, STAGES, NT, MINB, true>)
            : reinterpret_cast<const void*>(attend_e4m3_kernel<DK, DV, WARPS, STAGES, NT, MINB, false>);
  return true;
}

}  // namespace

bool attend_config_e4m3(int dk, int dv, int page_size, int rows, AttendConfig* cfg) {
  // More than 16 rows: the tensor-memory kernel where it is built, else row
  // blocks that each read the keys again.  Both sides, here and there, 8 requests
  // of 2048-16384 tokens, us:
  //   rows a kv head            9          16          24          32
  //   128/128, 8 kv heads   38   49     40   49     70   52     71   53
  //            2            20   19     22   20     24   23     25   24
  //   256/256, 8            85   82     87   83    150   88    208   90
  //            2            28   30     29   32     37   36     47   40
  //   256/128, 8            69   72     70   73    120   76    168   77
  //            2            21   25     22   25     29   28     38   29
  if (rows > 16 && attend_config_e4m3_ext(dk, dv, page_size, rows, cfg)) return true;
  const bool p1 = page_size == 1, wide = rows > 8;
  if (dk == 64 && dv == 64)
    return wide ? make_e4m3<64, 64, 4, 3, 2, 3>(p1, cfg) : make_e4m3<64, 64, 4, 3, 1, 4>(p1, cfg);
  if (dk == 128 && dv == 128)
    return wide ? make_e4m3<128, 128, 4, 4, 2, 2>(p1, cfg) : make_e4m3<128, 128, 4, 3, 1, 3>(p1, cfg);
  if (dk == 256 && dv == 128) return make_e4m3<256, 128, 4, 3, 1, 2>(p1, cfg);
  if (dk == 256 && dv == 256) return make_e4m3<256, 256, 4, 3, 1, 2>(p1, cfg);
  if (dk == 512 && dv == 256) return make_e4m3<512, 256, 8, 2, 1, 1>(p1, cfg);
  return false;
}

}  // namespace nvfp4kv
