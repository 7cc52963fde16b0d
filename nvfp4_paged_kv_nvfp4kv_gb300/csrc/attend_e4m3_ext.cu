// attend_e4m3_ext.cu -- attention over a paged E4M3 cache for many query rows
// per kv head (extend, prompts) on the fifth-generation tensor cores, sm_103a.
//
// The same function as attend_e4m3.cu (which gives the formulas).  The cache's
// codes are operands of tcgen05.mma kind::f8f6f4 as they stand: no element of K
// or V is converted.  What is not E4M3 is split into E4M3 pieces whose sum is
// exact enough, and the pieces' products are summed by the tensor cores:
//  * Query rows, times a power of two that puts the row's largest |q| into
//    [128, 256): q = q0 + q1 (+ q2), each piece the rounded rest.  A piece has
//    four significant bits, so two give a bf16 value's eight and three an f16
//    value's eleven, down to 2^-18 of the row's largest |q|.
//    S^T = K (q0 + q1 + ..)^T accumulates in one tile of tensor memory.
//  * Weights p' = 2^x (at most 2^8): p' = w0 + w1 / 32 (+ w2 / 1024).  Each
//    piece has its own columns of O^T = V^T (w0 | w1 | ..)^T, added in the
//    epilogue: eight bits of a weight with two pieces (bf16 outputs), twelve
//    with three (f16 outputs).  p' = 2^(x - m) lies at 2^5 where the tile
//    that set m had its largest, so a weight 2^-19 of that is still kept.
//  * Row sums come from the unsplit float32 weights, a register per query row
//    and thread, added up over the threads at the end.
//
// One CTA = one work unit (request, kv head, chunk of pages) x N = 16, 32 or
// 64 query rows (the G heads of the group times the query positions); tiles of
// 128 tokens; M = 128 tokens (S^T) or 128 value dims (O^T) fill the product
// for any N.  11 warps (12 would still leave a thread 168 registers, 13 only
// 128: the softmax threads then spill):
//  * loaders (warps 8-9): cp.async of the tile's K and V rows straight into
//    the 128-byte-swizzled operand layout (K: K-major, V: MN-major, both rows
//    of 128 bytes), any byte strides and both page sizes; V rows past the
//    request's end are zeroed (they may hold NaN codes);
//  * issue (warp 10, one thread): S^T = K Q^T into one of two tiles, O^T +=
//    V^T P^T, each once its inputs are ready;
//  * softmax (warps 0-7; thread = token of S^T, half of the query rows): the
//    token's K scale joins the row's factor, log2 of its V scale the exponent.
// The running maximum is raised only when a value exceeds 2^8.  Every wait is
// bounded; one that runs out sets flag 0x4 and the CTA winds down.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace nvfp4kv {
namespace {

using namespace dev;
using namespace tc5;

constexpr int kTileTok = 128;
constexpr int kThreads = 352;  // softmax warps 0-7, loaders 8-9, issue 10
constexpr int kLoaders = 2;  // warps, 64 rows of a tile each
constexpr float kRaise = 8.f;  // log2 of the largest weight before m is raised
constexpr float kPeak = 5.f;   // log2 of the weight of a new maximum
constexpr float kMinScale = 0x1p-64f, kMaxScale = 0x1p64f;

// D[tmem] (+)= A[smem] . B[smem], E4M3 operands (the instruction descriptor of
// kind::f16 with A and B formats 0 = E4M3)
__device__ __forceinline__ void umma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// two f32 -> two E4M3 codes (a in the low byte) and back to f16x2
__device__ __forceinline__ uint32_t e4m3x2_of_f32(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void cp_async_16a(uint32_t s, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(s), "l"(g));
}
__device__ __forceinline__ void cp_async_4(uint32_t s, const void* g) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(s), "l"(g));
}
__device__ __forceinline__ float log2_scale(float s) {
  const uint32_t u = __float_as_uint(s);
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float((u & 0x7FFFFFu) | 0x3F800000u)));
  return static_cast<float>(static_cast<int>(u >> 23) - 127) + r;
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

template <int DK, int DV, int N, int NP>
struct Ext {
  static constexpr int NH = N / 2;                 // query rows per softmax thread
  static constexpr int NQ = 3;                     // query pieces (2 used for bf16)
  static constexpr int KB = kTileTok * DK, VB = kTileTok * DV;
  static constexpr int QB = N * DK;                // one query piece
  // P^T rows: NP * N weight pieces of a token, in atoms of PA bytes
  static constexpr int PN = NP * N;
  static constexpr int PA = PN <= 32 ? 32 : PN <= 64 ? 64 : 128;
  static constexpr int PATOMS = (PN + PA - 1) / PA;
  static constexpr int PSTRIDE = kTileTok * PA;    // bytes of one atom column
  static constexpr int PB = PATOMS * PSTRIDE;
  static constexpr uint32_t PSWZ = PA == 32 ? kSwz32 : PA == 64 ? kSwz64 : kSwz128;
  static constexpr int PSWB = PA == 32 ? 1 : PA == 64 ? 2 : 3;
  static constexpr int SCB = kTileTok * 8;         // the tile's scales
  static constexpr int MISC = 8192;
  static constexpr int FIXED = 2 * PB + NQ * QB + MISC + 1024;
  static constexpr int KS = (232448 - FIXED) / (KB + VB + SCB) >= 4 ? 4 : 3;  // tiles in flight
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KS * KB;
  static constexpr int OFF_P = OFF_V + KS * VB;
  static constexpr int OFF_Q = OFF_P + 2 * PB;
  static constexpr int OFF_SC = OFF_Q + NQ * QB;
  static constexpr int OFF_MISC = OFF_SC + KS * SCB;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;  // + alignment slack
  static constexpr int SCOL = 0, OCOL = 2 * N;     // S^T x2, O^T blocks of 128 value dims
  static constexpr int COLS = OCOL + (DV / 128) * PN;
  static constexpr int TCOLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr uint32_t IDESC_QK = idesc_f16(128, N, 0, 0);
  static constexpr uint32_t IDESC_PV = idesc_f16(128, PN, 1, 1);
  static_assert(DK % 128 == 0 && DV % 128 == 0, "operand rows of 128 bytes");
  static_assert(OFF_P % 1024 == 0 && OFF_Q % 1024 == 0 && OFF_MISC % 16 == 0, "align");
  static_assert(SMEM <= 232448 && COLS <= 512 && PN % 16 == 0 && PN <= 256, "resources");
  static_assert(16 * 8 + 16 + (8 * N + 2 * N + 4 + 4 * N) * 4 <= MISC, "misc");
};

// P1: 1-token pages
template <int DK, int DV, int N, int NP, bool P1>
__global__ void __launch_bounds__(kThreads, 1) attend_e4m3_ext_kernel(const AttendParams p) {
  using T = Ext<DK, DV, N, NP>;
  constexpr int NH = T::NH, KS = T::KS;
  constexpr int CW = NH < 16 ? NH : 16;  // columns per softmax chunk
  constexpr int NCH = NH / CW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem + T::OFF_K;
  uint8_t* sV = smem + T::OFF_V;
  uint8_t* sP = smem + T::OFF_P;
  uint8_t* sQ = smem + T::OFF_Q;
  float* sSc = reinterpret_cast<float*>(smem + T::OFF_SC);  // [KS][K 128 | V 128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_MISC);
  uint64_t* kv_full = bars;       // [KS] loaders -> issue
  uint64_t* kv_empty = bars + 4;  // [KS] PV done -> loaders
  uint64_t* s_full = bars + 8;    // [2] QK done -> softmax
  uint64_t* p_full = bars + 10;   // [2] softmax -> issue
  uint64_t* pv_done = bars + 12;  // [2] PV done -> softmax
  uint64_t* q_full = bars + 14;   // Q ready -> issue
  uint64_t* fin = bars + 15;      // wind-down of the products
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_minlim = reinterpret_cast<int*>(s_tmem + 2);
  // per query row: score factor, -m, raise threshold, causal limit
  float* s_f = reinterpret_cast<float*>(s_tmem + 4);
  float* s_nm = s_f + N;
  float* s_thr = s_nm + N;
  int* s_lim = reinterpret_cast<int*>(s_thr + N);
  float* s_m = reinterpret_cast<float*>(s_lim + N);  // m (log2), -inf before the first tile
  int* s_max = reinterpret_cast<int*>(s_m + N);      // reduction keys, then shifts
  float* s_corr = reinterpret_cast<float*>(s_max + N);
  int* s_qamax = reinterpret_cast<int*>(s_corr + N);
  float* s_fin = reinterpret_cast<float*>(s_qamax + N);  // [2N + 4]
  float* s_l = s_fin + 2 * N + 4;                        // [4][N] row sums of the lane quarters

  const WorkUnit u = load_unit(p);
  const int G = p.group;
  const int R = G * u.qo_len;
  const int row0 = blockIdx.y * N;
  if (row0 >= R) return;  // uniform: before any barrier or tensor memory use
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q4 = warp & 3;       // tensor-memory lane quarter
  const int j = 32 * q4 + lane;  // token of the tile / value dim
  const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
  const int unit_tok = (P1 ? 1 : kPageSize) * u.num_pages;
  // tokens of the unit that some row of the block sees
  int tok_end = min(u.kv_len, u.tok_begin + unit_tok);
  if (p.causal) {
    const int last = min(R, row0 + N) - 1;
    tok_end = min(tok_end, u.kv_len - u.qo_len + last / G + 1);
  }
  const int ntiles = max(0, (tok_end - u.tok_begin + kTileTok - 1) / kTileTok);
  const int nq = p.q_f16 ? 3 : 2;

  if (tid == 0) {
    for (int b = 0; b < KS; ++b) {
      mbar_init(&kv_full[b], kLoaders);
      mbar_init(&kv_empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 8);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, 8);
    mbar_init(fin, 1);
    mbar_init_fence();
    *s_abort = 0;
    *s_minlim = INT32_MAX;
  }
  if (tid < N) s_qamax[tid] = 0;
  if (warp == 0) {
    tmem_alloc(s_tmem, T::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= 8 && warp < 8 + kLoaders) {
    // ================= loaders: warp 8 + w copies rows 64 w .. + 63 ==========
    const CacheView& c = p.cache;
    const int r0 = 64 * (warp - 8);
    const uint8_t* kb = c.k_data + (int64_t)u.h_kv * c.k_sh;
    const uint8_t* vb = c.v_data + (int64_t)u.h_kv * c.v_sh;
    const uint8_t* ksb = c.k_sf + (int64_t)u.h_kv * c.ksf_sh;
    const uint8_t* vsb = c.v_sf + (int64_t)u.h_kv * c.vsf_sh;
    // pages of this lane's rows r0 + lane and r0 + 32 + lane in tile t; a row
    // past the unit's pages takes the last one (its K row is masked, its V
    // row zeroed)
    auto load_pid = [&](int t, int half) -> int32_t {
      if (t >= ntiles) return 0;
      const int rel = t * kTileTok + r0 + 32 * half + lane;
      const int32_t id =
          __ldg(p.kv_indices + u.page_begin + min(P1 ? rel : rel / kPageSize, u.num_pages - 1));
      if (id < 0 || id >= c.num_pages) {
        atomicOr(p.flags, 0x1u);
        return 0;
      }
      return id;
    };
    // 8 lanes copy 128 bytes of a row, 4 rows an instruction
    auto copy = [&](uint32_t tile, const uint8_t* base, int64_t sp, int64_t ss, int32_t pid,
                    int half) {
      const int r4 = lane >> 3, ch = lane & 7;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + r4, row = r0 + 32 * half + r;
        const int32_t pg = __shfl_sync(0xffffffffu, pid, r);
        const uint8_t* src = base + pg * sp + (P1 ? 0 : (row % kPageSize) * ss) + 16 * ch;
        cp_async_16a(tile + row * 128 + ((ch ^ (row & 7)) << 4), src);
      }
    };
    auto issue = [&](int t, int32_t pid0, int32_t pid1) {
      const int st = t % KS;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int32_t pid = half ? pid1 : pid0;
#pragma unroll
        for (int b = 0; b < DK / 128; ++b)
          copy(smem_addr(sK) + st * T::KB + b * (kTileTok * 128), kb + 128 * b, c.k_sp, c.k_ss,
               pid, half);
#pragma unroll
        for (int b = 0; b < DV / 128; ++b)
          copy(smem_addr(sV) + st * T::VB + b * (kTileTok * 128), vb + 128 * b, c.v_sp, c.v_ss,
               pid, half);
        const uint32_t sc = smem_addr(sSc) + st * T::SCB + 4 * (r0 + 32 * half + lane);
        cp_async_4(sc, ksb + pid * c.ksf_sp);
        cp_async_4(sc + 4 * kTileTok, vsb + pid * c.vsf_sp);
      }
    };
    constexpr int LAG = KS - 2;  // tiles between a tile's copies and its hand-over
    int32_t next0 = load_pid(0, 0), next1 = load_pid(0, 1);
    for (int t = 0; t < ntiles + LAG; ++t) {
      if (t < ntiles) {
        if (t >= KS) {
          bool ok = true;
          if (lane == 0) ok = wait_bar(&kv_empty[t % KS], (t / KS - 1) & 1, s_abort, p.flags);
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          tc_fence_after();
        }
        const int32_t pid0 = next0, pid1 = next1;
        next0 = load_pid(t + 1, 0);
        next1 = load_pid(t + 1, 1);
        issue(t, pid0, pid1);
      }
      cp_async_commit();
      if (t < LAG) continue;
      cp_async_wait<LAG>();  // this thread's copies of tile i landed
      const int i = t - LAG;
      __syncwarp();
      // rows past the request's end or the unit's pages: no NaN code times 0
      const int live = min(u.kv_len - u.tok_begin, unit_tok) - i * kTileTok;
      for (int row = max(live, r0); row < r0 + 64; ++row)
#pragma unroll
        for (int b = 0; b < DV / 128; ++b)
          *reinterpret_cast<uint32_t*>(sV + (i % KS) * T::VB + b * (kTileTok * 128) + row * 128 +
                                       4 * lane) = 0u;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[i % KS]);
    }
    cp_async_wait<0>();
  } else if (warp == 8 + kLoaders) {
    // ================= product issue (one thread) ==========================
    if (lane == 0) {
      const uint64_t kd0 = smem_desc(smem_addr(sK), 16, 1024, kSwz128);
      const uint64_t qd0 = smem_desc(smem_addr(sQ), 16, 1024, kSwz128);
      const uint64_t vd0 = smem_desc(smem_addr(sV), kTileTok * 128, 1024, kSwz128);
      const uint64_t pd0 = smem_desc(smem_addr(sP), T::PSTRIDE, 8 * T::PA, T::PSWZ);
      auto issue_qk = [&](int k) {
        tc_fence_after();
        const uint32_t d = tmem + T::SCOL + N * (k & 1);
        const uint64_t kd = kd0 + (((k % KS) * T::KB) >> 4);
        for (int q = 0; q < nq; ++q)
#pragma unroll
          for (int kk = 0; kk < DK / 32; ++kk)
            umma8_ss(d, kd + (((kk >> 2) * (kTileTok * 128) + (kk & 3) * 32) >> 4),
                     qd0 + ((q * T::QB + (kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4),
                     T::IDESC_QK, (q > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&s_full[k & 1]);
      };
      auto issue_pv = [&](int i) {
        tc_fence_after();
        const uint64_t vd = vd0 + (((i % KS) * T::VB) >> 4);
        const uint64_t pd = pd0 + (((i & 1) * T::PB) >> 4);
#pragma unroll
        for (int b = 0; b < DV / 128; ++b)
#pragma unroll
          for (int k = 0; k < kTileTok / 32; ++k)
            umma8_ss(tmem + T::OCOL + b * T::PN,
                     vd + ((b * (kTileTok * 128) + k * 32 * 128) >> 4),
                     pd + ((k * 32 * T::PA) >> 4), T::IDESC_PV, (i > 0 || k > 0) ? 1u : 0u);
        umma_commit(&pv_done[i & 1]);
        umma_commit(&kv_empty[i % KS]);
      };
      // whichever product has its inputs: S(qk) once its tile is in and S
      // buffer qk & 1 was consumed (PV(qk - 2) issued), O += PV(pv) once P(pv)
      // is written
      bool ok = wait_bar(q_full, 0, s_abort, p.flags);
      int qk = 0, pv = 0;
      uint32_t idle = 0;
      while (ok && pv < ntiles) {
        bool prog = false;
        if (qk < ntiles && qk < pv + 2 && mbar_test_wait(&kv_full[qk % KS], (qk / KS) & 1)) {
          issue_qk(qk);
          ++qk;
          prog = true;
        }
        if (pv < qk && mbar_test_wait(&p_full[pv & 1], (pv >> 1) & 1)) {
          issue_pv(pv);
          ++pv;
          prog = true;
        }
        if (prog) {
          idle = 0;
          continue;
        }
        if (*s_abort) break;
        if (++idle > kIdlePolls) {
          *s_abort = 1;
          atomicOr(p.flags, 0x4u);
          break;
        }
        __nanosleep(32);
      }
      umma_commit(fin);  // wind-down: every product issued has completed
      drain_bar(fin, 0, p.flags);
    }
    __syncwarp();
  } else {
    // ================= softmax + epilogue (warps 0-7) ======================
    const int c0 = (warp >> 2) * NH;  // this thread's first query row
    auto q2 = [&](uint32_t w) -> float2 {
      if (p.q_f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
      return make_float2(bf16_bits_to_f32(w & 0xFFFFu), bf16_bits_to_f32(w >> 16));
    };
    // ---- Q pieces, swizzled: 8 dims (one 16-byte load) at a time ------------
    constexpr int QCH = N * DK / 8;
    auto q_load = [&](int ci) {
      const int gr = row0 + ci / (DK / 8);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (gr < R)
        v = *reinterpret_cast<const uint4*>(p.q + (int64_t)(u.qo_begin + gr / G) * p.q_stride_tok +
                                            (int64_t)(u.h_kv * G + gr % G) * p.q_stride_head +
                                            (ci % (DK / 8)) * 8);
      return v;
    };
#pragma unroll 4
    for (int ci = tid; ci < QCH; ci += 256) {
      const uint4 v = q_load(ci);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float am = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = q2(w[e]);
        am = fmaxf(am, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
      atomicMax(&s_qamax[ci / (DK / 8)], __float_as_int(am));
    }
    named_sync(3, 256);
    auto exp_of = [&](int r) {  // e with amax * 2^e in [128, 256)
      const float amax = __int_as_float(s_qamax[r]);
      int e = 0;
      if (amax > 0.f) e = 7 - (int)((__float_as_uint(amax) >> 23) & 0xFF) + 127;
      return max(-120, min(120, e));
    };
#pragma unroll 2
    for (int ci = tid; ci < QCH; ci += 256) {
      const uint4 v = q_load(ci);
      const int r = ci / (DK / 8), c8 = ci % (DK / 8);
      const float up = __uint_as_float((uint32_t)(127 + exp_of(r)) << 23);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float2 rest[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rest[e] = q2(w[e]);
        rest[e].x *= up;
        rest[e].y *= up;
      }
      const uint32_t off = (uint32_t)(c8 >> 4) * (N * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                           (c8 & 15) * 8;
      for (int q = 0; q < nq; ++q) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[e] = e4m3x2_of_f32(rest[e].x, rest[e].y);
          const uint32_t back = e4m3x2_to_f16x2(h[e]);
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
          rest[e].x -= b.x;
          rest[e].y -= b.y;
        }
        *reinterpret_cast<uint2*>(sQ + q * T::QB + swz<3>(off)) =
            make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
      }
    }
    if (tid < N) {
      const int r = tid, gr = row0 + r;
      if (gr < R) {
        const int lim = p.causal ? (u.kv_len - u.qo_len + gr / G) : (u.kv_len - 1);
        s_f[r] = p.qk_scale_log2 * __uint_as_float((uint32_t)(127 - exp_of(r)) << 23);
        s_nm[r] = 0.f;
        s_thr[r] = -INFINITY;  // no maximum yet: any visible score raises
        s_lim[r] = lim;
        atomicMin(s_minlim, lim);
      } else {  // padding row: every weight 0, never raises
        s_f[r] = 0.f;
        s_nm[r] = -INFINITY;
        s_thr[r] = INFINITY;
        s_lim[r] = -1;
      }
      s_m[r] = -INFINITY;
    }
    fence_async_smem();
    named_sync(3, 256);
    if (lane == 0) mbar_arrive(q_full);
    const int min_lim = *s_minlim;
    const int nvalid = min(N, R - row0);  // columns that are real query rows
    const bool active = c0 < nvalid;      // warp-uniform

    const int gbar = 1 + (warp >> 2), gtid = tid & 127;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      bool ok = true;
      if (lane == 0) ok = wait_bar(bar, parity, s_abort, p.flags);
      return __shfl_sync(0xffffffffu, ok, 0);
    };
    // The two column halves (warps 0-3 and 4-7) are independent groups: each
    // votes and reduces over its own 128 threads (barrier 1 + half).  A wait
    // that runs out sets the abort flag; the loop then runs to its end with
    // every later wait returning at once, so no thread leaves a barrier
    // sequence the others still follow.
    bool unset = active;  // some column of this half has no maximum yet
    uint64_t lsum[NH / 2];  // this token's share of the row sums, two rows each
#pragma unroll
    for (int e = 0; e < NH / 2; ++e) lsum[e] = 0;
    for (int i = 0; i < ntiles; ++i) {
      const int sb = i & 1;
      // S(i) done also means PV(i-2) done: P buffer sb is free again
      warp_wait(&kv_full[i % KS], (i / KS) & 1);  // (passed: the tile's scales are visible)
      warp_wait(&s_full[sb], (i >> 1) & 1);
      tc_fence_after();
      const int tile_tok0 = u.tok_begin + i * kTileTok;
      const int tok = tile_tok0 + j;
      const bool tok_ok = tok < tok_end;
      const bool mask_rows = tile_tok0 + kTileTok - 1 > min_lim;
      float x[NH];
      uint64_t iv2 = 0;
      bool trig = false;
      if (active) {
        // this token's scales
        const float* sc = sSc + (i % KS) * (T::SCB / 4);
        float ks = tok_ok ? sc[j] : 1.f, vs = tok_ok ? sc[kTileTok + j] : 1.f;
        const float ksc = fminf(fmaxf(ks, kMinScale), kMaxScale);
        const float vsc = fminf(fmaxf(vs, kMinScale), kMaxScale);
        if (ksc != ks || vsc != vs) atomicOr(p.flags, 0x20u);
        const float lv = log2_scale(vsc);
        const float iv1 = ex2(-lv);
        const uint64_t ks2 = pack_f32x2(ksc, ksc), lv2 = pack_f32x2(lv, lv);
        iv2 = pack_f32x2(iv1, iv1);
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          uint32_t sv[CW];
          const int cb = c0 + ch * CW;
          tmem_ld<CW>(tmem + lane_base + T::SCOL + N * sb + cb, sv);
          tmem_wait_ld<CW>(sv);
#pragma unroll
          for (int e4 = 0; e4 < CW; e4 += 4) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s_f + cb + e4);
            const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(s_nm + cb + e4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t s2 = pack_f32x2(__uint_as_float(sv[e4 + 2 * e]),
                                             __uint_as_float(sv[e4 + 2 * e + 1]));
              unpack_f32x2(fma_f32x2(s2, mul_f32x2(e ? f.y : f.x, ks2),
                                     add_f32x2(e ? nm.y : nm.x, lv2)),
                           x[ch * CW + e4 + 2 * e], x[ch * CW + e4 + 2 * e + 1]);
            }
          }
        }
        if (mask_rows) {
#pragma unroll
          for (int e4 = 0; e4 < NH; e4 += 4) {
            const int4 lm = *reinterpret_cast<const int4*>(s_lim + c0 + e4);
            if (tok > lm.x) x[e4] = -INFINITY;
            if (tok > lm.y) x[e4 + 1] = -INFINITY;
            if (tok > lm.z) x[e4 + 2] = -INFINITY;
            if (tok > lm.w) x[e4 + 3] = -INFINITY;
          }
        }
        if (unset) {
#pragma unroll
          for (int e4 = 0; e4 < NH; e4 += 4) {
            const float4 t4 = *reinterpret_cast<const float4*>(s_thr + c0 + e4);
            trig |= (x[e4] > t4.x) | (x[e4 + 1] > t4.y) | (x[e4 + 2] > t4.z) |
                    (x[e4 + 3] > t4.w);
          }
        } else {  // every real column has a maximum: one test of the largest
          float mx = fmaxf(x[0], x[1]);
#pragma unroll
          for (int e = 2; e < NH; e += 2) mx = fmax3(mx, x[e], x[e + 1]);
          trig = mx > kRaise;
        }
        trig = trig && tok_ok;
      }
      if (named_or(gbar, 128, trig)) {
        // ---- raise this half's maxima to the tile's row maxima ---------------
        if (gtid < NH) s_max[c0 + gtid] = INT32_MIN;
        named_sync(gbar, 128);
        if (active) {  // lane e keeps column e's warp maximum: one atomic per lane
          int kk = INT32_MIN;
#pragma unroll
          for (int e = 0; e < NH; ++e) {
            const int k = __reduce_max_sync(0xffffffffu, fkey(tok_ok ? x[e] : -INFINITY));
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
          float corr = 1.f, delta = 0.f;
          if (tm != -INFINITY && (m_old == -INFINITY || tm > kPeak)) {
            delta = tm - kPeak;
            const float m_new = (m_old == -INFINITY ? 0.f : m_old) + delta;
            if (m_old != -INFINITY) corr = ex2(m_old - m_new);
            s_m[r] = m_new;
            s_nm[r] = -m_new;
            s_thr[r] = kRaise;
            moved = corr != 1.f;
          }
          s_corr[r] = corr;
          s_max[r] = __float_as_int(delta);
        }
        const bool rescale = named_or(gbar, 128, moved) && i > 0;
        unset = named_or(gbar, 128, gtid < NH && c0 + gtid < nvalid && s_m[c0 + gtid] == -INFINITY);
#pragma unroll
        for (int e = 0; e < NH; ++e) x[e] -= __int_as_float(s_max[c0 + e]);
        if (rescale && active) {  // O^T columns and row sums *= corr, once PV(i-1) is done
          warp_wait(&pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int e = 0; e < NH / 2; ++e)
            lsum[e] = mul_f32x2(lsum[e], *reinterpret_cast<const uint64_t*>(s_corr + c0 + 2 * e));
          for (int blk = 0; blk < (DV / 128) * NP; ++blk)
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
              uint32_t ov[CW];
              const uint32_t oa = tmem + lane_base + T::OCOL + blk * N + c0 + ch * CW;
              tmem_ld<CW>(oa, ov);
              tmem_wait_ld<CW>(ov);
#pragma unroll
              for (int e = 0; e < CW; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * s_corr[c0 + ch * CW + e]);
              tmem_st<CW>(oa, ov);
            }
          tmem_wait_st();
        }
      }
      // ---- weights: the P^T row of this token, NP pieces ----------------------
      if (active) {
        // Row byte off of this token lies in atom off / PA; 16-byte chunks are
        // xor-swizzled inside the atom's 1024-byte blocks.
        uint8_t* pt = sP + sb * T::PB;
        const uint32_t pj = (uint32_t)(j >> 3) * (8 * T::PA) + (j & 7) * T::PA;
        auto at = [&](int piece, int e) {
          const uint32_t o = piece * N + c0 + e;
          return pt + (o / T::PA) * T::PSTRIDE + swz<T::PSWB>(pj + o % T::PA);
        };
#pragma unroll
        for (int e8 = 0; e8 < NH; e8 += 8) {
          uint32_t h[NP][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a = 0.f, b = 0.f;
            if (tok_ok) {
              a = ex2(x[e8 + 2 * e]);
              b = ex2(x[e8 + 2 * e + 1]);
            }
            lsum[e8 / 2 + e] = fma_f32x2(pack_f32x2(a, b), iv2, lsum[e8 / 2 + e]);
            uint32_t rest = f32x2_to_f16x2(a, b);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
              h[q][e] = e4m3x2_of_f16x2(rest);
              if (q + 1 < NP)  // (rest - piece) * 32: exact in f16
                rest = hmul2(hsub2(rest, e4m3x2_to_f16x2(h[q][e])), 0x50005000u);
            }
          }
#pragma unroll
          for (int q = 0; q < NP; ++q)
            *reinterpret_cast<uint2*>(at(q, e8)) =
                make_uint2(h[q][0] | (h[q][1] << 16), h[q][2] | (h[q][3] << 16));
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
    if (ntiles > 0) warp_wait(&pv_done[(ntiles - 1) & 1], ((ntiles - 1) >> 1) & 1);
    {
      tc_fence_after();
      constexpr float kLn2 = 0.69314718055994530942f;
      const bool partial = p.split && u.num_splits > 1;
      const int Hq = p.num_qo_heads;
      if (active) {
        // lane e (mod CW) derives normaliser and output row of column e, once
        const int e_l = lane & (CW - 1);
        uint16_t* const out_u = p.out + (int64_t)u.qo_begin * Hq * DV;
        float* const part_u = partial ? p.partial_o + (int64_t)u.partial_base * DV : nullptr;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          const int col_l = c0 + ch * CW + e_l;
          float f_l = 0.f;
          int64_t off_l = 0;  // output row of the column, from the unit's first row
          if (col_l < nvalid) {
            const float L = s_l[col_l] + s_l[N + col_l] + s_l[2 * N + col_l] + s_l[3 * N + col_l];
            const float m = s_m[col_l];
            const bool any = L > 0.f && m != -INFINITY;
            f_l = any ? 1.f / L : 0.f;
            const float lse_v = any ? (m + log2f(L)) * kLn2 : -INFINITY;
            const int gr = row0 + col_l, qi = gr / G, head = u.h_kv * G + gr % G;
            off_l = partial ? ((int64_t)qi * Hq + head) * u.num_splits + u.split
                            : (int64_t)qi * Hq + head;
            if (q4 == 0 && lane < CW) {
              if (!partial) {
                if (p.lse) p.lse[(int64_t)u.qo_begin * Hq + off_l] = lse_v;
              } else {
                p.partial_lse[(int64_t)u.partial_base + off_l] = lse_v;
              }
            }
          }
#pragma unroll
          for (int b = 0; b < DV / 128; ++b) {
            float o[CW];
#pragma unroll
            for (int q = NP - 1; q >= 0; --q) {  // o = o0 + (o1 + o2 / 32) / 32
              uint32_t ov[CW];
              tmem_ld<CW>(tmem + lane_base + T::OCOL + b * T::PN + q * N + c0 + ch * CW, ov);
              tmem_wait_ld<CW>(ov);
#pragma unroll
              for (int e = 0; e < CW; ++e)
                o[e] = q == NP - 1 ? __uint_as_float(ov[e])
                                   : fmaf(o[e], 0.03125f, __uint_as_float(ov[e]));
            }
#pragma unroll
            for (int e = 0; e < CW; ++e) {
              const float f = __shfl_sync(0xffffffffu, f_l, e);
              const int64_t off = __shfl_sync(0xffffffffu, off_l, e);
              if (c0 + ch * CW + e < nvalid) {
                const float v = f != 0.f ? o[e] * f : 0.f;
                if (!partial)
                  out_u[off * DV + 128 * b + j] = pack_out1(v, p.out_f16);
                else
                  part_u[off * DV + 128 * b + j] = v;
              }
            }
          }
        }
      }
      if (partial)
        merge_if_last<N, DV, 256, 4>(p, u, row0, R, s_fin, tid, [] { named_sync(3, 256); });
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

template <int DK, int DV, int N, int NP>
bool make_ext(bool p1, AttendConfig* cfg) {
  cfg->kind = kKernelE4m3;
  cfg->dk = DK;
  cfg->dv = DV;
  cfg->rows = N;
  cfg->warps = kThreads / 32;
  cfg->units_per_cta = 1;
  cfg->smem_bytes = Ext<DK, DV, N, NP>::SMEM;
  cfg->func = p1 ? reinterpret_cast<const void*>(attend_e4m3_ext_kernel<DK, DV, N, NP, true>)
                 : reinterpret_cast<const void*>(attend_e4m3_ext_kernel<DK, DV, N, NP, false>);
  return true;
}

}  // namespace

// The kernel for (dk, dv), up to `rows` query rows per CTA; f16 outputs take
// three weight pieces.
bool attend_config_e4m3_ext(int dk, int dv, int page_size, int rows, bool out_f16,
                            AttendConfig* cfg) {
  const bool p1 = page_size == 1;
#define NVFP4KV_EXT(DK_, DV_, N_) \
  return out_f16 ? make_ext<DK_, DV_, N_, 3>(p1, cfg) : make_ext<DK_, DV_, N_, 2>(p1, cfg)
  if (dk == 128 && dv == 128) {
    if (rows <= 16) NVFP4KV_EXT(128, 128, 16);
    if (rows <= 32) NVFP4KV_EXT(128, 128, 32);
    NVFP4KV_EXT(128, 128, 64);
  }
#undef NVFP4KV_EXT
  return false;
}

}  // namespace nvfp4kv
