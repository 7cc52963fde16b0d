// attend_e4m3_ext.cu -- attention over a paged E4M3 cache for many query rows
// per kv head (extend, prompts) on the fifth-generation tensor cores, sm_103a.
//
// The same function as attend_e4m3.cu (which gives the formulas).  The cache's
// codes are operands of tcgen05.mma kind::f8f6f4 as they stand: no element of K
// or V is converted.  What is not E4M3 is split into 8-bit pieces whose sum is
// exact enough, and the pieces' products are summed by the tensor cores:
//  * Query rows, times a power of two that puts the row's largest |q| into
//    [2^14, 2^15): q = q0 + q1 + q2, E5M2 pieces (the operands of a product have
//    formats of their own), each the rounded rest.  A piece has three significant
//    bits and leaves a rest of at most 1/8: of an f16 value's eleven bits, 1024 to
//    2047 units, |rest| <= 128, then 8 units, which the third piece holds exactly;
//    bf16 has fewer.  The smallest code is 2^-16, so nothing above 2^-31 of the
//    row's largest |q| is lost.  (E4M3 pieces, four bits each, would spare bf16 the
//    third piece and end at 2^-17 of the largest: under one outlier dim the others
//    lose their bits.)  S^T = K (q0 + q1 + q2)^T accumulates in one tile of tensor
//    memory.
//  * Weights p' = y b (at most 2^8, rounded to f16): p' = w0 + w1 / 32 + w2 / 1024.  Each piece
//    has its own columns of O^T = V^T (w0 | w1 | w2)^T, added in the epilogue:
//    twelve bits of a weight, and a weight 2^-20 of the largest is still kept.
//    (Two pieces hold eight bits; to keep weights that small they allow only
//    three bits between a tile's maximum and the raise, and a raise of some of
//    the rows in most tiles then costs more than the third piece: 223 against
//    218 us on 32 requests of 2000-16000 tokens x 64 rows, when measured.)
//  * Row sums come from the float32 y = 2^(score - m), a register per query row
//    and thread, added up over the threads at the end.
//
// One CTA = one work unit (request, kv head, chunk of pages) x N = 32 or 64
// query rows (the G heads of the group times the query positions); tiles of
// 128 tokens; M = 128 tokens (S^T) or 128 value dims (O^T) fill the product
// for any N.  20 warps at N = 64:
//  * loaders (a warp for K and the scales, one for V): cp.async of a tile's rows
//    straight into the 128-byte-swizzled operand layout (K: K-major, V: MN-major,
//    both rows of 128 bytes), any byte strides and both page sizes;
//  * issue (two warps, one thread each): S^T = K Q^T into a ring of tiles in
//    tensor memory, and O^T += V^T P^T, each once its inputs are ready;
//  * softmax (four warps for each 16 query rows; thread = token of S^T): the
//    token's K scale multiplies the sum, its V scale the weight.
//    The work of a tile is dependent chains, so many warps with few rows each
//    beat few warps with many (8 warps of 32 rows 258, 16 of 16 rows 236 us).
// The running maximum is raised only when a value exceeds 2^8.  Every wait is
// bounded; one that runs out sets flag 0x4 and the CTA winds down.
//
// Measured: 32 requests of 2000-16000 tokens, 16 new rows of 32 heads each (64
// rows to a kv head), 170 us, 3.6 TB/s, 0.54 of a plain copy (1-token pages 296: the
// loaders form an address a row); 4 requests of 32771 tokens x 32 rows 73 us.  At
// 256/256 and 256/128, blocks of 32 rows that each read the keys, 493 and 419 us.  8
// prompts of 512 tokens from nothing 170 us.  No unit is full (issue slots
// 58 %, shared memory 45 %, products a third): a tile's way through the warps
// bounds it, 1.1 us at either N, and a unit's 12 tiles' worth of start and end.
// Timed with parts left out: two query pieces, half of O^T's products, no
// conversions of weights or no votes change nothing; no loads take 10 % off.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace nvfp4kv {
namespace {

using namespace dev;
using namespace tc5;

// Test build only: the K loader of CTA (0, 0) withholds its arrival for the
// first tile, so the S^T issuer's wait runs out and the CTA winds down.
#ifndef NVFP4KV_E4M3_TEST_SKIP_ARRIVE
#define NVFP4KV_E4M3_TEST_SKIP_ARRIVE 0
#endif
constexpr int kTileTok = 128;
constexpr int kLoaders = 2;  // warps: K, V
constexpr int kAllSoftmax = 5;  // named barriers 1 .. 4: the column groups
constexpr int kNanReady = 6;
constexpr int kPieces = 3;      // of a weight
constexpr float kRaise = 8.f;  // log2 of the largest weight before m is raised

// D[tmem] (+)= A[smem] . B[smem], 8-bit operands (the instruction descriptor of
// kind::f16; formats of A at bit 7 and B at bit 10: 0 E4M3, 1 E5M2)
__device__ __forceinline__ void umma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// four values (two f16x2) -> four E4M3 codes, the first in the low byte, and
// back (16-bit halves by register pairs: the conversions address them directly)
__device__ __forceinline__ uint32_t e4m3x4_of_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
// four float32 values -> four E5M2 codes, the first in the low byte, and back
__device__ __forceinline__ uint32_t e5m2x4_of_f32(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e5m2x2.f32 l, %2, %1;\n"
      " cvt.rn.satfinite.e5m2x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void e5m2x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e5m2x2 %0, l;\n"
      " cvt.rn.f16x2.e5m2x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// one arrival on `bar` once this thread's earlier cp.async copies have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_addr(bar))
               : "memory");
}
// pairs of f32 (Blackwell's two-wide float32 arithmetic)
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int DK, int DV, int N>
struct Ext {
  static constexpr int NH = 16;                    // query rows per softmax thread
  static constexpr int CG = N / NH;                // column groups of four warps
  static constexpr int SW = 4 * CG;                // softmax warps
  static constexpr int THREADS = 32 * (SW + kLoaders + 2);
  static constexpr int NQ = 3;                     // query pieces
  static constexpr int KB = kTileTok * DK, VB = kTileTok * DV;
  static constexpr int QB = N * DK;                // one query piece
  // P^T: a token's kPieces * N weight pieces, one product's N: at N = 32 a row of
  // 128 bytes a token, at N = 64 a block of 64-byte rows for each piece
  static constexpr int PN = kPieces * N;
  static constexpr int PROW = PN <= 128 ? 128 : 64;
  static constexpr int PBLK = kTileTok * PROW;
  static constexpr int PB = PROW == 128 ? PBLK : kPieces * PBLK;
  static_assert(PROW == 128 || N == 64, "a piece fills a 64-byte row");
  static constexpr int SCB = kTileTok * 8;         // K and V scale
  static constexpr int MISC = 4608;
  static constexpr int NPB = 2;                    // P^T buffers
  // Tests of a barrier before a loader or issuer suspends: with 8 softmax warps
  // there is room for more (1: 96, 16: 89 us, 4 requests of 32771 tokens x 32
  // rows), with 16 the tests take their issue slots (1: 184, 16: 189 us, 32 of
  // 2000-16000 x 64).
  static constexpr int SPINS = SW > 8 ? 1 : 16;
  // Rings: K tiles until their S^T is done, V tiles until their P^T V is (at 128
  // dims (3, 5) 181, (4, 4) 176, (5, 3) 184 us, a fifth S^T tile no gain), S^T
  // tiles in tensor memory and, behind both, the tokens' scales (read from a K
  // tile's copy until the softmax has passed it: KR + SB tiles at most).
  static constexpr int SB = 4, SR = 8;
  static constexpr int FIXED = NPB * PB + NQ * QB + SR * SCB + MISC + 1024;
  static constexpr int FIT = (232448 - FIXED) / 16384;  // 16 KB blocks that fit
  static constexpr int KR = DK == 128 ? 4 : DV == 128 ? 3 : 2;
  static constexpr int VR = DK == 128 ? 4 : DV == 128 ? 3 : 2;
  static_assert(KR * (DK / 128) + VR * (DV / 128) <= FIT && KR + SB <= SR, "rings");
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KR * KB;
  static constexpr int OFF_P = OFF_V + VR * VB;
  static constexpr int OFF_Q = OFF_P + NPB * PB;
  static constexpr int OFF_SC = OFF_Q + NQ * QB;
  static constexpr int OFF_MISC = OFF_SC + SR * SCB;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;  // + alignment slack
  static constexpr int SCOL = 0, OCOL = SB * N;    // S^T ring, O^T blocks of 128 value dims
  static constexpr int COLS = OCOL + (DV / 128) * PN;
  static constexpr int TCOLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr uint32_t IDESC_QK = idesc_f16(128, N, 0, 0) | 1u << 10;  // E4M3 . E5M2
  static constexpr uint32_t IDESC_PV = idesc_f16(128, PN, 1, 1);
  static_assert(DK % 128 == 0 && DV % 128 == 0, "operand rows of 128 bytes");
  static_assert(OFF_P % 1024 == 0 && OFF_Q % 1024 == 0 && OFF_MISC % 16 == 0, "align");
  static_assert(SMEM <= 232448 && COLS <= 512 && PN % 16 == 0 && PN <= 256, "resources");
  static_assert(60 * 8 + 16 + (7 * N + 2 * N + 4 + 4 * N + DV + 4) * 4 <= MISC, "misc");
};

// A V tile that some row of the block does not see whole (run by a warp): rows
// from `live` on are zeroed, NaN codes before them too, and first[d] becomes the
// first token (the tile begins with `tok0`) that had one in value dim d.
template <int DV>
__device__ __forceinline__ void no_nan(uint8_t* tile, int live, int tok0, int* first) {
  const int lane = threadIdx.x & 31;
  tile += 4 * lane;  // this lane's column of 4 bytes
  for (int row = max(live, 0); row < kTileTok; ++row)
#pragma unroll
    for (int b = 0; b < DV / 128; ++b)
      *reinterpret_cast<uint32_t*>(tile + b * (kTileTok * 128) + row * 128) = 0u;
#pragma unroll 1
  for (int k0 = 0; k0 < kTileTok * (DV / 128); k0 += 16) {  // rows of 128 dims
    uint8_t* at = tile + k0 * 128;
    uint32_t nan = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      nan |= (*reinterpret_cast<const uint32_t*>(at + 128 * k) & 0x7F7F7F7Fu) + 0x01010101u;
    if (!(nan & 0x80808080u)) continue;
    for (int k = 0; k < 16; ++k)
      for (int e = 0; e < 4; ++e)
        if ((at[128 * k + e] & 0x7F) == 0x7F) {
          const int row = (k0 + k) % kTileTok, blk = (k0 + k) / kTileTok;
          at[128 * k + e] = 0;
          atomicMin(&first[128 * blk + 16 * ((lane >> 2) ^ (row & 7)) + 4 * (lane & 3) + e],
                    tok0 + row);
        }
  }
}

// wait_bar for a barrier that mostly is ready, or soon will be: tested SPINS times
// first, as the suspending wait takes about 300 cycles even when it is
template <int SPINS>
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* flags) {
#pragma unroll 1
  for (int k = 0; k < SPINS; ++k)
    if (mbar_test_wait(bar, parity)) return true;
  return wait_bar(bar, parity, abort, flags);
}

// P1: 1-token pages
template <int DK, int DV, int N, bool P1>
__global__ void __launch_bounds__(Ext<DK, DV, N>::THREADS, 1)
    attend_e4m3_ext_kernel(const AttendParams p) {
  using T = Ext<DK, DV, N>;
  constexpr int NH = T::NH, KR = T::KR, VR = T::VR, SB = T::SB, SR = T::SR, NPB = T::NPB;
  constexpr int SW = T::SW, ST = 32 * SW;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset, not through an integer: the compiler then still knows
  // a shared pointer (through an integer, every access became a generic one with
  // 64-bit address arithmetic)
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* sK = smem + T::OFF_K;
  uint8_t* sV = smem + T::OFF_V;
  uint8_t* sP = smem + T::OFF_P;
  uint8_t* sQ = smem + T::OFF_Q;
  float* sSc = reinterpret_cast<float*>(smem + T::OFF_SC);  // [SR][2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_MISC);
  uint64_t* k_landed = bars;       // [KR] a K tile and its scales are in
  uint64_t* k_empty = bars + 8;    // [KR] S^T done, scales read
  uint64_t* v_landed = bars + 16;  // [VR] a V tile is in
  uint64_t* v_empty = bars + 24;   // [VR] P^T V done
  uint64_t* s_full = bars + 32;    // [SB] S^T done, scales in order -> softmax
  uint64_t* s_empty = bars + 40;   // [SB] S^T read
  uint64_t* p_full = bars + 48;    // [NPB] softmax -> O^T issue
  uint64_t* pv_done = bars + 52;   // [NPB] P^T V done -> softmax
  uint64_t* v_seen = bars + 54;    // O^T issue has seen V tile first_part + 1 - VR land
  uint64_t* q_full = bars + 56;    // Q ready -> S^T issue
  uint64_t* v_clean = bars + 57;   // the V tiles from first_part on hold no NaN code
  uint64_t* fin = bars + 58;       // [2] wind-down of the two issuers' products
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 60);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  // per query row: score factor, -m, raise threshold, causal limit
  float* s_f = reinterpret_cast<float*>(s_tmem + 4);
  float* s_nm = s_f + N;
  float* s_thr = s_nm + N;
  int* s_lim = reinterpret_cast<int*>(s_thr + N);
  float* s_m = reinterpret_cast<float*>(s_lim + N);  // m (log2), -inf before the first tile
  int* s_max = reinterpret_cast<int*>(s_m + N);      // reduction keys, then shifts
  float* s_half = reinterpret_cast<float*>(s_max + N);  // root of a raise's factor
  float* s_fin = s_half + N;                         // [2N + 4]
  float* s_l = s_fin + 2 * N + 4;                    // [4][N] row sums of the lane quarters
  int* s_nan = reinterpret_cast<int*>(s_l + 4 * N);  // [DV] first NaN token taken out of V
  int* s_tok = s_nan + DV;                           // tok_begin, tok_end of the unit

  const int G = p.group;
  const int row0 = blockIdx.y * N;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q4 = warp & 3;       // tensor-memory lane quarter
  const int j = 32 * q4 + lane;  // token of the tile / value dim
  const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
  const WorkUnit u = load_unit(p);
  const int R = G * u.qo_len;
  if (row0 >= R) return;  // uniform: before any barrier or tensor memory use
  // the unit's tokens in the cache, those that some row of the block sees, their
  // tiles; the last token that every row sees, the first tile that holds a later one
  const int unit_end = min(u.kv_len - u.tok_begin, (P1 ? 1 : kPageSize) * u.num_pages);
  int tok_end = u.tok_begin + unit_end, all_see = u.kv_len - 1;
  if (p.causal) {
    tok_end = min(tok_end, u.kv_len - u.qo_len + (min(R, row0 + N) - 1) / G + 1);
    all_see = u.kv_len - u.qo_len + row0 / G;
  }
  const int ntiles = max(0, (tok_end - u.tok_begin + kTileTok - 1) / kTileTok);
  const int first_part = max(min(all_see + 1 - u.tok_begin, unit_end), 0) / kTileTok;

  if (tid == 0) {
    for (int b = 0; b < KR; ++b) {
      mbar_init(&k_landed[b], 32);
      mbar_init(&k_empty[b], 1);
    }
    for (int b = 0; b < VR; ++b) {
      mbar_init(&v_landed[b], 32);
      mbar_init(&v_empty[b], 1);
    }
    for (int b = 0; b < SB; ++b) {
      mbar_init(&s_full[b], 2);
      mbar_init(&s_empty[b], SW);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&fin[b], 1);
    }
    for (int b = 0; b < T::NPB; ++b) {
      mbar_init(&p_full[b], SW);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, SW);
    mbar_init(v_clean, 1);
    mbar_init(v_seen, 1);
    mbar_init_fence();
    *s_abort = 0;
  }
  if (warp == 0) {
    tmem_alloc(s_tmem, T::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= SW && warp < SW + kLoaders) {
    // ================= loaders: warp SW K tiles and scales, SW + 1 V tiles =====
    const CacheView& c = p.cache;
    const bool isv = warp > SW;
    const int64_t sp = isv ? c.v_sp : c.k_sp, ss = isv ? c.v_ss : c.k_ss;
    // page ids of this lane's rows 32 g + lane of tile t, a tile ahead of their
    // use (where they are checked: a check here would wait for them); a row past
    // the unit's pages takes the last one (its K row is masked, its V row zeroed)
    auto load_pids = [&](int t, int32_t (&pid)[4]) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        pid[g] = 0;
        if (t >= ntiles) continue;
        const int rel = t * kTileTok + 32 * g + lane;
        pid[g] = __ldg(p.kv_indices + u.page_begin +
                       min(P1 ? rel : rel / kPageSize, u.num_pages - 1));
      }
    };
    // 8 lanes copy 128 bytes of a row, 4 rows an instruction: 16 rows (a page
    // at page size 16) from row 16 g of the tile
    const int r4 = lane >> 3, ch = lane & 7;
    // swizzled 16-byte chunk of this lane's rows 8 i + r4 and 8 i + 4 + r4
    const uint32_t at0 = r4 * 128 + ((ch ^ r4) << 4), at1 = (r4 + 4) * 128 + ((ch ^ (r4 + 4)) << 4);
    auto copy = [&](uint32_t tile, const uint8_t* from, const int32_t (&pid)[4]) {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const uint32_t dst = tile + g * 2048;
        if constexpr (P1) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int32_t pg = __shfl_sync(0xffffffffu, pid[g >> 1], 16 * (g & 1) + 4 * k + r4);
            cp_async_16s(dst + (k >> 1) * 1024 + (k & 1 ? at1 : at0), from + pg * sp + 16 * ch);
          }
        } else {
          const uint8_t* src =
              from + __shfl_sync(0xffffffffu, pid[g >> 1], 16 * (g & 1)) * sp + r4 * ss + 16 * ch;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            cp_async_16s(dst + (k >> 1) * 1024 + (k & 1 ? at1 : at0), src + 4 * k * ss);
        }
      }
    };
    const int ring = isv ? VR : KR, bytes = isv ? T::VB : T::KB;
    const int blocks = isv ? DV / 128 : DK / 128;
    const uint32_t s0 = smem_addr(isv ? sV : sK);
    uint64_t* empty = isv ? v_empty : k_empty;
    uint64_t* landed = isv ? v_landed : k_landed;
    bool alive = true;
    const int h = u.h_kv;
    const uint8_t* base = isv ? c.v_data + (int64_t)h * c.v_sh : c.k_data + (int64_t)h * c.k_sh;
    const uint8_t* ksb = c.k_sf + (int64_t)h * c.ksf_sh;
    const uint8_t* vsb = c.v_sf + (int64_t)h * c.vsf_sh;
    int32_t next[4];
    load_pids(0, next);
    // tile t goes to stage st for the round-th time
    for (int t = 0, st = 0, round = 0; t < ntiles; ++t) {
      if (round > 0) {
        if (lane == 0) alive = wait_soon<T::SPINS>(&empty[st], (round - 1) & 1, s_abort, p.flags);
        alive = __shfl_sync(0xffffffffu, alive, 0);
        if (!alive) break;
        tc_fence_after();
      }
      int32_t pid[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        pid[g] = next[g];
        if (pid[g] < 0 || pid[g] >= c.num_pages) {
          atomicOr(p.flags, 0x1u);
          pid[g] = 0;
        }
      }
      load_pids(t + 1, next);
#pragma unroll 1
      for (int b = 0; b < blocks; ++b)
        copy(s0 + st * bytes + b * (kTileTok * 128), base + 128 * b, pid);
      if (!isv) {
        const uint32_t sc = smem_addr(sSc) + (t % SR) * T::SCB + 4 * lane;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          cp_async_4s(sc + 128 * g, ksb + pid[g] * c.ksf_sp);
          cp_async_4s(sc + 128 * g + 4 * kTileTok, vsb + pid[g] * c.vsf_sp);
        }
      }
      const bool withhold = NVFP4KV_E4M3_TEST_SKIP_ARRIVE && blockIdx.x == 0 &&
                            blockIdx.y == 0 && !isv && t == 0;
      if (!withhold) cp_async_arrive(&landed[st]);  // once this thread's copies have landed
      if (++st == ring) {
        st = 0;
        ++round;
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == SW + kLoaders) {
    // ======== S^T issue: one thread the products ==============================
    const uint64_t kd0 = smem_desc(smem_addr(sK), 16, 1024, kSwz128);
    const uint64_t qd0 = smem_desc(smem_addr(sQ), 16, 1024, kSwz128);
    bool ok = true;
    if (lane == 0) ok = wait_soon<T::SPINS>(q_full, 0, s_abort, p.flags);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    for (int k = 0, st = 0, round = 0; k < ntiles && ok; ++k) {
      if (lane == 0) {
        ok = wait_soon<T::SPINS>(&k_landed[st], round & 1, s_abort, p.flags);
        if (ok && k >= SB)
          ok = wait_soon<T::SPINS>(&s_empty[k % SB], (k / SB - 1) & 1, s_abort, p.flags);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      fence_async_smem();
      if (lane == 0) {
        tc_fence_after();
        const uint32_t d = tmem + T::SCOL + N * (k % SB);
        const uint64_t kd = kd0 + ((st * T::KB) >> 4);
#pragma unroll 1
        for (int q = 0; q < T::NQ; ++q)
#pragma unroll
          for (int kk = 0; kk < DK / 32; ++kk)
            umma8_ss(d, kd + (((kk >> 2) * (kTileTok * 128) + (kk & 3) * 32) >> 4),
                     qd0 + ((q * T::QB + (kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4),
                     T::IDESC_QK, (q > 0 || kk > 0) ? 1u : 0u);
        mbar_arrive(&s_full[k % SB]);  // (the scales landed with K)
        umma_commit(&s_full[k % SB]);
        umma_commit(&k_empty[st]);
      }
      if (++st == KR) {
        st = 0;
        ++round;
      }
    }
    // The V tiles that some row does not see whole, the last one or two (the rows'
    // limits lie less than N <= 64 tokens apart): a weight of 0 must not meet a
    // NaN code.  Done here, as this warp is up to four tiles ahead (1 % of the
    // launch; in the warp that issues O^T 4 %).  A wait by parity tells a phase
    // from the one before it only, and this warp has not followed the V ring: the
    // O^T issuer, which has, says when the stages' earlier tiles have landed
    // (v_seen; tile first_part + 1 - VR is the later of the two, and neither it nor
    // a tile before it waits for v_clean).
    static_assert(N <= 64 && VR >= 2, "both tiles fit the ring while O^T waits for v_clean");
    for (int d = lane; d < DV; d += 32) s_nan[d] = INT_MAX;
    if (lane == 0 && ok && first_part < ntiles) ok = wait_soon<T::SPINS>(v_seen, 0, s_abort, p.flags);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    for (int t = first_part; t < ntiles && ok; ++t) {
      if (lane == 0) ok = wait_soon<T::SPINS>(&v_landed[t % VR], (t / VR) & 1, s_abort, p.flags);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      __syncwarp();  // (a shuffle orders no memory: the tile is lane 0's to see until here)
      if (ok)
        no_nan<DV>(sV + (t % VR) * T::VB, unit_end - t * kTileTok,
                   u.tok_begin + t * kTileTok, s_nan);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(v_clean);
    named_sync(kNanReady, ST + 32);  // s_nan is complete
    if (lane == 0) {
      umma_commit(&fin[0]);  // wind-down: every product issued has completed
      drain_bar(&fin[0], 0, p.flags);
    }
    __syncwarp();
  } else if (warp == SW + kLoaders + 1) {
    // ======== O^T issue: one thread the products ==============================
    const uint64_t vd0 = smem_desc(smem_addr(sV), kTileTok * 128, 1024, kSwz128);
    const uint64_t pd0 = smem_desc(smem_addr(sP), T::PBLK, 8 * T::PROW,
                                   T::PROW == 128 ? kSwz128 : kSwz64);
    bool ok = true;
    if (lane == 0 && first_part + 1 < VR) mbar_arrive(v_seen);  // (their stages' first tiles)
    for (int i = 0, st = 0, round = 0; i < ntiles; ++i) {
      if (lane == 0) {
        ok = wait_soon<T::SPINS>(&v_landed[st], round & 1, s_abort, p.flags);
        if (ok && i == first_part + 1 - VR) mbar_arrive(v_seen);
        if (ok && i >= first_part) ok = wait_soon<T::SPINS>(v_clean, 0, s_abort, p.flags);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        ok = wait_soon<T::SPINS>(&p_full[i % NPB], (i / NPB) & 1, s_abort, p.flags);
        if (ok) {
          tc_fence_after();
          const uint64_t vd = vd0 + ((st * T::VB) >> 4);
          const uint64_t buf = ((i % NPB) * T::PB) >> 4;
#pragma unroll
          for (int b = 0; b < DV / 128; ++b)
#pragma unroll
            for (int k = 0; k < kTileTok / 32; ++k) {
              const uint64_t vk = vd + ((b * (kTileTok * 128) + k * 32 * 128) >> 4);
              const uint32_t acc = (i > 0 || k > 0) ? 1u : 0u;
              umma8_ss(tmem + T::OCOL + b * T::PN, vk, pd0 + buf + ((k * 32 * T::PROW) >> 4),
                       T::IDESC_PV, acc);
            }
          umma_commit(&pv_done[i % NPB]);
          umma_commit(&v_empty[st]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (++st == VR) {
        st = 0;
        ++round;
      }
    }
    if (lane == 0) {
      umma_commit(&fin[1]);
      drain_bar(&fin[1], 0, p.flags);
    }
    __syncwarp();
  } else {
    // ================= softmax + epilogue ==================================
    const int c0 = (warp >> 2) * NH;  // this thread's first query row
    auto q2 = [&](uint32_t w) -> float2 {
      return p.q_f16 ? unpack2<true>(w) : unpack2<false>(w);
    };
    // ---- Q pieces, swizzled: a thread takes 8 dims (16 bytes) of a row, the
    // row's neighbouring DK / 8 threads share its largest |q| by shuffles --------
    constexpr int QW = DK / 8;
    static_assert(N * QW % 32 == 0 && ST % 32 == 0 && QW <= 32, "whole warps of whole rows");
    constexpr int QIT = N * QW / ST;
    uint4 qv[QIT];
#pragma unroll
    for (int k = 0; k < QIT; ++k) {
      const int ci = tid + k * ST, gr = row0 + ci / QW;
      qv[k] = make_uint4(0u, 0u, 0u, 0u);
      if (gr < R)
        qv[k] = *reinterpret_cast<const uint4*>(
            p.q + (int64_t)(u.qo_begin + gr / G) * p.q_stride_tok +
            (int64_t)(u.h_kv * G + gr % G) * p.q_stride_head + ci % QW * 8);
    }
#pragma unroll
    for (int k = 0; k < QIT; ++k) {
      const int ci = tid + k * ST, r = ci / QW, c8 = ci % QW, gr = row0 + r;
      const uint32_t w[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
      float2 rest[4];
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rest[e] = q2(w[e]);
        amax = fmaxf(amax, fmaxf(fabsf(rest[e].x), fabsf(rest[e].y)));
      }
#pragma unroll
      for (int o = QW / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      int ex = 0;  // amax * 2^ex in [2^14, 2^15)
      if (amax > 0.f) ex = 14 - (int)((__float_as_uint(amax) >> 23) & 0xFF) + 127;
      ex = max(-120, min(120, ex));
      // (an infinite element has no pieces: its row is NaN, as 0 * inf makes it)
      const float up = isinf(amax) ? NAN : __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rest[e].x *= up;
        rest[e].y *= up;
      }
      const uint32_t off = (uint32_t)(c8 >> 4) * (N * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                           (c8 & 15) * 8;
#pragma unroll 1
      for (int q = 0; q < T::NQ; ++q) {
        uint32_t h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          h[e] = e5m2x4_of_f32(rest[2 * e].x, rest[2 * e].y, rest[2 * e + 1].x, rest[2 * e + 1].y);
          uint32_t back[2];
          e5m2x4_to_f16(h[e], back[0], back[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = unpack2<true>(back[k]);
            rest[2 * e + k].x -= f.x;
            rest[2 * e + k].y -= f.y;
          }
        }
        *reinterpret_cast<uint2*>(sQ + q * T::QB + swz<3>(off)) = make_uint2(h[0], h[1]);
      }
      if (c8 == 0) {
        const bool real = gr < R;  // a padding row: every weight 0, never raises
        s_f[r] = real ? p.qk_scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23) : 0.f;
        s_nm[r] = real ? 0.f : -INFINITY;
        s_thr[r] = real ? -INFINITY : INFINITY;  // no maximum yet: any visible score raises
        s_lim[r] = !real ? -1 : p.causal ? u.kv_len - u.qo_len + gr / G : u.kv_len - 1;
        s_m[r] = -INFINITY;
      }
    }
    if (tid == 0) {
      s_tok[0] = u.tok_begin;
      s_tok[1] = tok_end;
    }
    fence_async_smem();
    named_sync(kAllSoftmax, ST);
    if (lane == 0) mbar_arrive(q_full);
    // the first tile with a token that some row does not see
    const int part = (min(all_see + 1, tok_end) - u.tok_begin) >> 7;
    static_assert(kTileTok == 128, "the shift");
    const int nvalid = min(N, R - row0);  // columns that are real query rows
    const bool active = c0 < nvalid;      // warp-uniform

    const int gbar = 1 + (warp >> 2), gtid = tid & 127;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {  // (every lane: no hand-over)
      wait_soon<1>(bar, parity, s_abort, p.flags);
      __syncwarp();
    };
    // The column groups (four warps each, the tile's 128 tokens) are
    // independent: each votes and reduces over its own 128 threads.  A wait
    // that runs out sets the abort flag; the loop then runs to its end with
    // every later wait returning at once, so no thread leaves a barrier
    // sequence the others still follow.
    bool unset = active;  // some column of this group has no maximum yet
    // where this thread's pieces go in a P^T buffer: its token's row, 16-byte
    // chunks xor-swizzled
    uint32_t p_at[kPieces];
#pragma unroll
    for (int q = 0; q < kPieces; ++q)
      p_at[q] = T::PROW == 128 ? swz<3>((uint32_t)j * 128 + q * N + c0)
                               : q * T::PBLK + swz<2>((uint32_t)j * 64 + c0);
    uint64_t lsum[NH / 2];  // this token's share of the row sums, two rows each
#pragma unroll
    for (int e = 0; e < NH / 2; ++e) lsum[e] = 0;
    // x: log2-domain scores of tile i less the running maxima, -inf where masked
    // or past the unit's end; vs: the token's V scale
    auto scores = [&](int i, float (&x)[NH], float& vs) {
      const float* sc = sSc + (i % SR) * (T::SCB / 4) + j;
      const float ks0 = sc[0], vs0 = sc[kTileTok];
      const float ks = clamped_scale(ks0);
      vs = clamped_scale(vs0);
      if (ks != ks0 || vs != vs0) atomicOr(p.flags, 0x20u);
      const uint64_t ks2 = pack_f32x2(ks, ks);
      uint32_t sv[NH];
      tmem_ld<NH>(tmem + lane_base + T::SCOL + N * (i % SB) + c0, sv);
      tmem_wait_ld<NH>(sv);
#pragma unroll
      for (int e4 = 0; e4 < NH; e4 += 4) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s_f + c0 + e4);
        const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(s_nm + c0 + e4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint64_t s2 = pack_f32x2(__uint_as_float(sv[e4 + 2 * e]),
                                         __uint_as_float(sv[e4 + 2 * e + 1]));
          unpack_f32x2(fma_f32x2(mul_f32x2(s2, ks2), e ? f.y : f.x, e ? nm.y : nm.x),
                       x[e4 + 2 * e], x[e4 + 2 * e + 1]);
        }
      }
      if (i >= part) {  // (a unit's last tiles)
        const int tok = s_tok[0] + i * kTileTok + j;
        const int past = tok >= s_tok[1] ? INT32_MIN : INT32_MAX;
#pragma unroll
        for (int e4 = 0; e4 < NH; e4 += 4) {
          const int4 lm = *reinterpret_cast<const int4*>(s_lim + c0 + e4);
          if (tok > min(lm.x, past)) x[e4] = -INFINITY;
          if (tok > min(lm.y, past)) x[e4 + 1] = -INFINITY;
          if (tok > min(lm.z, past)) x[e4 + 2] = -INFINITY;
          if (tok > min(lm.w, past)) x[e4 + 3] = -INFINITY;
        }
      }
    };
    for (int i = 0; i < ntiles; ++i) {
      const int sb = i % NPB;
      warp_wait(&s_full[i % SB], (i / SB) & 1);
      tc_fence_after();
      float x[NH];
      float vs = 1.f, lv = 0.f;  // the token's V scale and its log2
      bool trig = false;
      if (active) {
        scores(i, x, vs);
        lv = log2_scale(vs);
        if (unset) {
#pragma unroll
          for (int e4 = 0; e4 < NH; e4 += 4) {
            const float4 t4 = *reinterpret_cast<const float4*>(s_thr + c0 + e4);
            trig |= (x[e4] + lv > t4.x) | (x[e4 + 1] + lv > t4.y) | (x[e4 + 2] + lv > t4.z) |
                    (x[e4 + 3] + lv > t4.w);
          }
        } else {  // every real column has a maximum: one test of the largest
          float mx = fmaxf(x[0], x[1]);
#pragma unroll
          for (int e = 2; e < NH; e += 2) mx = fmax3(mx, x[e], x[e + 1]);
          trig = mx + lv > kRaise;
        }
      }
      if (named_or(gbar, 128, trig)) {
        // ---- raise this group's maxima to the tile's row maxima ---------------
        if (gtid < NH) s_max[c0 + gtid] = INT32_MIN;
        named_sync(gbar, 128);
        if (active) {  // lane e keeps column e's warp maximum: one atomic per lane
          int kk = INT32_MIN;
#pragma unroll
          for (int e = 0; e < NH; ++e) {
            const int k = __reduce_max_sync(0xffffffffu, fkey(x[e] + lv));
            kk = lane == e ? k : kk;
          }
          if (lane < NH) atomicMax(&s_max[c0 + lane], kk);
        }
        named_sync(gbar, 128);
        bool moved = false;
        if (gtid < NH) {
          const int r = c0 + gtid;
          const float tm = funkey(s_max[r]);  // tile maximum, relative to the old m
          const float m_old = s_m[r];
          float half = 1.f;  // the square root of the row's factor
          if (tm != -INFINITY && (m_old == -INFINITY || tm > 0.f)) {
            const float m_new = (m_old == -INFINITY ? 0.f : m_old) + tm;
            if (m_old != -INFINITY) half = ex2(0.5f * (m_old - m_new));
            s_m[r] = m_new;
            s_nm[r] = -m_new;
            s_thr[r] = kRaise;
            moved = half != 1.f;
          }
          s_half[r] = half;
        }
        const bool rescale = named_or(gbar, 128, moved) && i > 0;
        unset = named_or(gbar, 128, gtid < NH && c0 + gtid < nvalid && s_m[c0 + gtid] == -INFINITY);
        if (rescale && active) {  // O^T columns and row sums *= corr, once PV(i-1) is done
          warp_wait(&pv_done[(i - 1) % NPB], ((i - 1) / NPB) & 1);
          tc_fence_after();
#pragma unroll
          for (int e = 0; e < NH / 2; ++e) {
            const uint64_t half = *reinterpret_cast<const uint64_t*>(s_half + c0 + 2 * e);
            lsum[e] = mul_f32x2(mul_f32x2(lsum[e], half), half);
          }
          for (int blk = 0; blk < (DV / 128) * kPieces; ++blk) {
            uint32_t ov[NH];
            const uint32_t oa = tmem + lane_base + T::OCOL + blk * N + c0;
            tmem_ld<NH>(oa, ov);
            tmem_wait_ld<NH>(ov);
#pragma unroll
            for (int e = 0; e < NH; ++e)
              ov[e] = __float_as_uint(__uint_as_float(ov[e]) * (s_half[c0 + e] * s_half[c0 + e]));
            tmem_st<NH>(oa, ov);
          }
          tmem_wait_st();
        }
        if (active) scores(i, x, vs);  // (again: nothing of the tile is kept over a raise)
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[i % SB]);  // this warp has read S^T and the scales
      // ---- weights: the P^T row of this token, in pieces ----------------------
      if (i >= NPB) warp_wait(&pv_done[sb], (i / NPB - 1) & 1);  // P buffer sb is free
      if (active) {
        uint32_t h[kPieces][NH / 4];
        const uint64_t vs2 = pack_f32x2(vs, vs);
#pragma unroll
        for (int e = 0; e < NH / 4; ++e) {
          uint32_t rest[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int col = 4 * e + 2 * k;
            const uint64_t y = pack_f32x2(ex2(x[col]), ex2(x[col + 1]));
            lsum[col / 2] = add_f32x2(lsum[col / 2], y);
            float a, b;
            unpack_f32x2(mul_f32x2(y, vs2), a, b);
            rest[k] = f32x2_to_f16x2(a, b);
          }
#pragma unroll
          for (int q = 0; q < kPieces; ++q) {
            h[q][e] = e4m3x4_of_f16(rest[0], rest[1]);
            if (q + 1 < kPieces) {  // (rest - piece) * 32: exact in f16
              uint32_t back[2];
              e4m3x4_to_f16(h[q][e], back[0], back[1]);
              rest[0] = hmul2(hsub2(rest[0], back[0]), 0x50005000u);
              rest[1] = hmul2(hsub2(rest[1], back[1]), 0x50005000u);
            }
          }
        }
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
          uint8_t* at = sP + sb * T::PB + p_at[q];
          *reinterpret_cast<uint4*>(at) = make_uint4(h[q][0], h[q][1], h[q][2], h[q][3]);
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[sb]);
    }

    // ---- row sums over the 128 tokens: lane e of a warp holds row e ----------
    if (active) {
      float mine = 0.f;
#pragma unroll
      for (int e = 0; e < NH; ++e) {
        float lo, hi;
        unpack_f32x2(lsum[e / 2], lo, hi);
        float s = e & 1 ? hi : lo;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        mine = lane == e ? s : mine;
      }
      if (lane < NH) s_l[q4 * N + c0 + lane] = mine;
    }
    named_sync(gbar, 128);

    // ---- epilogue: O^T row of value dim j, this thread's query rows -----------
    // (the unit is read again: kept over the tiles, it would cost them registers)
    const WorkUnit end = load_unit(p);
    if (ntiles > 0) warp_wait(&pv_done[(ntiles - 1) % NPB], ((ntiles - 1) / NPB) & 1);
    named_sync(kNanReady, ST + 32);
    {
      tc_fence_after();
      constexpr float kLn2 = 0.69314718055994530942f;
      const bool partial = p.split && end.num_splits > 1;
      const int Hq = p.num_qo_heads;
      if (active) {
        // lane e (mod NH) derives normaliser and output row of column e, once
        const int e_l = lane & (NH - 1), col_l = c0 + e_l;
        uint16_t* const out_u = p.out + (int64_t)end.qo_begin * Hq * DV;
        float* const part_u = partial ? p.partial_o + (int64_t)end.partial_base * DV : nullptr;
        float f_l = 0.f;
        int off_l = 0;  // output row of the column, from the unit's first row
        if (col_l < nvalid) {
          const float L = s_l[col_l] + s_l[N + col_l] + s_l[2 * N + col_l] + s_l[3 * N + col_l];
          const float m = s_m[col_l];
          const bool any = m != -INFINITY || isnan(L);  // (a NaN score need not raise)
          f_l = any ? 1.f / L : 0.f;
          const float lse_v = any ? (m + log2f(L)) * kLn2 : -INFINITY;
          const int gr = row0 + col_l, qi = gr / G, head = end.h_kv * G + gr % G;
          off_l = partial ? (qi * Hq + head) * end.num_splits + end.split : qi * Hq + head;
          if (q4 == 0 && lane < NH) {
            if (!partial) {
              if (p.lse) p.lse[(int64_t)end.qo_begin * Hq + off_l] = lse_v;
            } else {
              p.partial_lse[(int64_t)end.partial_base + off_l] = lse_v;
            }
          }
        }
#pragma unroll
        for (int b = 0; b < DV / 128; ++b) {
          float o[NH];
#pragma unroll
          for (int q = kPieces - 1; q >= 0; --q) {  // o = o0 + (o1 + o2 / 32) / 32
            uint32_t ov[NH];
            tmem_ld<NH>(tmem + lane_base + T::OCOL + b * T::PN + q * N + c0, ov);
            tmem_wait_ld<NH>(ov);
#pragma unroll
            for (int e = 0; e < NH; ++e)
              o[e] = q == kPieces - 1 ? __uint_as_float(ov[e])
                                 : fmaf(o[e], 0.03125f, __uint_as_float(ov[e]));
          }
          if (const int first = s_nan[128 * b + j]; first != INT_MAX) {
#pragma unroll
            for (int e = 0; e < NH; ++e)
              if (s_lim[c0 + e] >= first) o[e] = NAN;
          }
#pragma unroll
          for (int e = 0; e < NH; ++e) {
            const float f = __shfl_sync(0xffffffffu, f_l, e);
            const int64_t off = __shfl_sync(0xffffffffu, off_l, e);
            if (c0 + e < nvalid) {
              const float v = f != 0.f ? o[e] * f : 0.f;
              if (!partial)
                out_u[off * DV + 128 * b + j] = pack_out1(v, p.out_f16);
              else
                part_u[off * DV + 128 * b + j] = v;
            }
          }
        }
      }
      if (partial)
        fold_if_last<N, DV, ST, 1, 4>(p, end, row0, nvalid, reinterpret_cast<int*>(s_fin + 2 * N),
                                      tid, [] { named_sync(kAllSoftmax, ST); });
    }
    tc_fence_before();
  }

  // ---- every role is done: release tensor memory -----------------------------
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, T::TCOLS);
  }
}

template <int DK, int DV, int N>
bool make_ext(bool p1, AttendConfig* cfg) {
  cfg->kind = kKernelE4m3;
  cfg->dk = DK;
  cfg->dv = DV;
  cfg->rows = N;
  cfg->warps = Ext<DK, DV, N>::THREADS / 32;
  cfg->units_per_cta = 1;
  cfg->smem_bytes = Ext<DK, DV, N>::SMEM;
  cfg->func = p1 ? reinterpret_cast<const void*>(attend_e4m3_ext_kernel<DK, DV, N, true>)
                 : reinterpret_cast<const void*>(attend_e4m3_ext_kernel<DK, DV, N, false>);
  return true;
}

}  // namespace

// The kernel for (dk, dv) and more than 16 query rows per kv head.
bool attend_config_e4m3_ext(int dk, int dv, int page_size, int rows, AttendConfig* cfg) {
  const bool p1 = page_size == 1;
  if (dk == 128 && dv == 128)
    return rows <= 32 ? make_ext<128, 128, 32>(p1, cfg) : make_ext<128, 128, 64>(p1, cfg);
  // 256 dims: 64 rows would leave at most two tiles in flight
  if (dk == 256 && dv == 128) return make_ext<256, 128, 32>(p1, cfg);
  if (dk == 256 && dv == 256) return make_ext<256, 256, 32>(p1, cfg);
  return false;
}

}  // namespace nvfp4kv
