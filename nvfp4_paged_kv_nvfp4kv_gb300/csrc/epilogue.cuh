// epilogue.cuh -- end of an attention work unit: combine the warps' online-
// softmax states of the CTA's query rows and store them; when the plan split
// the request, store an f32 partial state and let the last CTA of the
// (request, kv head, row block) fold all partials (log-sum-exp merge).
//
// The last CTA is found with a counter per (request, kv head, row block):
// every CTA publishes its partials (__threadfence) and then increments the
// counter; the CTA that sees num_splits - 1 is last, reads the partials
// through L2 (ld.global.cg) and resets the counter to 0 for the next run.
// No CTA waits for another.
#pragma once

#include <cstdint>

#include "device_common.cuh"
#include "internal.h"

namespace nvfp4kv {

// The split group's last CTA folds its partials.  Run by NTHREADS threads
// (tid in [0, NTHREADS)) that synchronise with `sync`; sFin: scratch of at
// least RB floats + 1 int.  Every thread must have stored its partials.
// Each thread folds whole (row, 4 dims) items: batches of MB partial states
// (their lse and o loaded together) with a running maximum, so the fold
// costs ceil(S / MB) dependent L2 round trips.
template <int RB, int DV, int NTHREADS, int MB = 8, class Sync>
__device__ __forceinline__ void merge_if_last(const AttendParams& p, const WorkUnit& u,
                                              int row0, int R, float* sFin, int tid,
                                              Sync sync) {
  using namespace dev;
  constexpr float kLog2e = 1.44269504088896340736f;
  constexpr float kLn2 = 0.69314718055994530942f;
  const int G = p.group, Hq = p.num_qo_heads;
  int* s_last = reinterpret_cast<int*>(sFin + 2 * RB);
  __threadfence();
  sync();
  if (tid == 0) {
    int* ctr = p.counters + (int64_t)u.pair * gridDim.y + blockIdx.y;
    const int old = atomicAdd(ctr, 1);
    *s_last = (old == u.num_splits - 1);
    if (*s_last) *ctr = 0;  // every other CTA of the group has arrived
  }
  sync();
  if (!*s_last) return;
  __threadfence();
  const int S = u.num_splits;
  constexpr int DQ = DV / 4;
  for (int idx = tid; idx < RB * DQ; idx += NTHREADS) {
    const int rr = idx / DQ, d4 = idx % DQ, r = row0 + rr;
    if (r >= R) continue;
    const int i = r / G, head = u.h_kv * G + r % G;
    const int64_t base = (int64_t)u.partial_base + ((int64_t)i * Hq + head) * S;
    float M = -INFINITY, L = 0.f;  // running max (log2 units) and sum
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += MB) {
      float lw[MB];
      float4 v[MB];
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        lw[j] = -INFINITY;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 + j < S) {
          lw[j] = __ldcg(p.partial_lse + base + s0 + j) * kLog2e;
          v[j] = __ldcg(reinterpret_cast<const float4*>(p.partial_o + (base + s0 + j) * DV) + d4);
        }
      }
      float mb = lw[0];
#pragma unroll
      for (int j = 1; j < MB; ++j) mb = fmaxf(mb, lw[j]);
      if (mb == -INFINITY) continue;
      const float mn = fmaxf(M, mb);
      const float cf = M == -INFINITY ? 0.f : ex2(M - mn);
      L *= cf;
      acc.x *= cf; acc.y *= cf; acc.z *= cf; acc.w *= cf;
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const float w = ex2(lw[j] - mn);  // 0 for lw = -inf
        L += w;
        acc.x += w * v[j].x; acc.y += w * v[j].y; acc.z += w * v[j].z; acc.w += w * v[j].w;
      }
      M = mn;
    }
    const bool any = M != -INFINITY && L > 0.f;
    const float inv = any ? 1.f / L : 0.f;
    const int64_t qrow = u.qo_begin + i;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (qrow * Hq + head) * DV + 4 * d4);
    dst[0] = pack_out2(acc.x * inv, acc.y * inv, p.out_f16);
    dst[1] = pack_out2(acc.z * inv, acc.w * inv, p.out_f16);
    if (d4 == 0 && p.lse) p.lse[qrow * Hq + head] = any ? (M + log2f(L)) * kLn2 : -INFINITY;
  }
}

// sM/sL: [WARPS][RB] running max (log2 domain) and sum of each warp;
// sO: [WARPS][RB][DV] each warp's un-normalised output rows;
// sFin: scratch of at least 2*RB floats + 1 int.  Run by the unit's
// WARPS * 32 threads (tid in [0, WARPS * 32)), which synchronise with `sync`.
template <int RB, int DV, int WARPS, class Sync>
__device__ __forceinline__ void finish_unit(const AttendParams& p, const WorkUnit& u,
                                            int row0, int R, const float* sM,
                                            const float* sL, const float* sO,
                                            float* sFin, int tid, Sync sync) {
  using namespace dev;
  constexpr float kLn2 = 0.69314718055994530942f;
  const int G = p.group, Hq = p.num_qo_heads;
  const bool partial = p.split && u.num_splits > 1;

  for (int idx = tid; idx < RB * (DV / 2); idx += WARPS * 32) {
    const int rr = idx / (DV / 2), d = 2 * (idx % (DV / 2));
    const int r = row0 + rr;
    if (r >= R) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sM[w * RB + rr]);
    float L = 0.f, o0 = 0.f, o1 = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float mw = sM[w * RB + rr];
        const float sc = (mw == -INFINITY) ? 0.f : ex2(mw - M);
        L += sL[w * RB + rr] * sc;
        const float2 ow = *reinterpret_cast<const float2*>(sO + (w * RB + rr) * DV + d);
        o0 += ow.x * sc;
        o1 += ow.y * sc;
      }
      const float inv = p.v_scale / L;
      o0 *= inv;
      o1 *= inv;
    }
    const float lse_v = (M == -INFINITY) ? -INFINITY : (M + log2f(L)) * kLn2;
    const int i = r / G, head = u.h_kv * G + r % G;
    const int64_t qrow = u.qo_begin + i;
    if (!partial) {
      *reinterpret_cast<uint32_t*>(p.out + (qrow * Hq + head) * DV + d) =
          pack_out2(o0, o1, p.out_f16);
      if (d == 0 && p.lse) p.lse[qrow * Hq + head] = lse_v;
    } else {
      const int64_t pi = (int64_t)u.partial_base +
                         ((int64_t)i * Hq + head) * u.num_splits + u.split;
      *reinterpret_cast<float2*>(p.partial_o + pi * DV + d) = make_float2(o0, o1);
      if (d == 0) p.partial_lse[pi] = lse_v;
    }
  }
  if (!partial) return;

  merge_if_last<RB, DV, WARPS * 32, 20>(p, u, row0, R, sFin, tid, sync);
}

// The same for a CTA that is one unit (all its threads, __syncthreads).
template <int RB, int DV, int WARPS>
__device__ __forceinline__ void finish_unit(const AttendParams& p, const WorkUnit& u,
                                            int row0, int R, const float* sM,
                                            const float* sL, const float* sO,
                                            float* sFin) {
  finish_unit<RB, DV, WARPS>(p, u, row0, R, sM, sL, sO, sFin, (int)threadIdx.x,
                             [] { __syncthreads(); });
}

// The split group's arrival and, in its last CTA, the fold of the partial
// states: NT threads (tid in [0, NT)) that synchronise with `sync`, `last` a
// word in shared memory.  The arrival is one acquire-release atomic after the
// barrier, which orders the CTA's partial stores before it and the last CTA's
// loads after it.  A thread folds IT items (row, four dims) at a time, MB
// partial states loaded together.  A state's factor is applied as two halves: one
// below 2^-126 counts where its state's values are that much larger (value scales
// 2^128 apart).  A NaN state (a NaN score in its chunk) makes the row NaN, lse too.
template <int RB, int DV, int NT, int IT, int MB, class Sync>
__device__ __forceinline__ void fold_if_last(const AttendParams& p, const WorkUnit& u, int row0,
                                             int rows, int* last, int tid, Sync sync) {
  using namespace dev;
  constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
  constexpr int DQ = DV / 4;
  const int G = p.group, Hq = p.num_qo_heads;
  sync();
  if (tid == 0) {
    int* ctr = p.counters + (int64_t)u.pair * gridDim.y + blockIdx.y;
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(ctr) : "memory");
    *last = old == u.num_splits - 1;
    if (*last) *ctr = 0;  // every other CTA of the group has arrived
  }
  sync();
  if (!*last) return;
  const int S = u.num_splits;
  for (int i0 = tid; i0 < rows * DQ; i0 += IT * NT) {
    float M[IT], L[IT];
    float4 acc[IT];
    int64_t base[IT];
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      const int idx = i0 + k * NT < rows * DQ ? i0 + k * NT : i0, r = row0 + idx / DQ;
      base[k] = (int64_t)u.partial_base +
                ((int64_t)(r / G) * Hq + u.h_kv * G + r % G) * S;
      M[k] = -INFINITY;
      L[k] = 0.f;
      acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int d4 = i0 % DQ;  // (NT is a multiple of DQ, or DQ of NT with IT = 1)
    static_assert(NT % DQ == 0, "a thread keeps its dims");
    for (int s0 = 0; s0 < S; s0 += MB) {
      float lw[IT][MB];
      float4 v[IT][MB];
#pragma unroll
      for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          lw[k][j] = -INFINITY;
          v[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (s0 + j < S) {
            lw[k][j] = __ldcg(p.partial_lse + base[k] + s0 + j) * kLog2e;
            v[k][j] = __ldcg(reinterpret_cast<const float4*>(p.partial_o + (base[k] + s0 + j) * DV) +
                             d4);
          }
        }
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        float mn = M[k];
#pragma unroll
        for (int j = 0; j < MB; ++j) mn = fmaxf(mn, lw[k][j]);
        if (mn == -INFINITY) {  // nothing yet, or NaN states alone
#pragma unroll
          for (int j = 0; j < MB; ++j)
            if (isnan(lw[k][j])) mn = 0.f;
          if (mn == -INFINITY) continue;
        }
        const float cf = ex2(0.5f * (M[k] - mn));  // 0 for -inf
        L[k] = L[k] * cf * cf;
        acc[k].x = acc[k].x * cf * cf;
        acc[k].y = acc[k].y * cf * cf;
        acc[k].z = acc[k].z * cf * cf;
        acc[k].w = acc[k].w * cf * cf;
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const float w = ex2(0.5f * (lw[k][j] - mn));
          L[k] = fmaf(w, w, L[k]);
          acc[k].x = fmaf(w, w * v[k][j].x, acc[k].x);
          acc[k].y = fmaf(w, w * v[k][j].y, acc[k].y);
          acc[k].z = fmaf(w, w * v[k][j].z, acc[k].z);
          acc[k].w = fmaf(w, w * v[k][j].w, acc[k].w);
        }
        M[k] = mn;
      }
    }
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      if (i0 + k * NT >= rows * DQ) break;
      const int r = row0 + (i0 + k * NT) / DQ;
      const int64_t row = (int64_t)(u.qo_begin + r / G) * Hq + u.h_kv * G + r % G;
      const bool any = M[k] != -INFINITY;
      const float inv = any ? 1.f / L[k] : 0.f;
      *reinterpret_cast<uint2*>(p.out + row * DV + 4 * d4) =
          make_uint2(pack_out2(acc[k].x * inv, acc[k].y * inv, p.out_f16),
                     pack_out2(acc[k].z * inv, acc[k].w * inv, p.out_f16));
      if (d4 == 0 && p.lse) p.lse[row] = any ? (M[k] + log2f(L[k])) * kLn2 : -INFINITY;
    }
  }
}

// finish_unit for a CTA that is one unit, four dims a thread and only the rows
// that exist, and fold_if_last in place of fences in every thread and an item at
// a time.  Measured on decode shapes: combine, store, arrival and fold 3.1 ->
// 2.4 us (head dims 128), 6.0 -> 4.1 us (512 / 256).
// sO rows lie OS floats apart (more than DV: the warps' stores into them then
// spread over the banks).
template <int RB, int DV, int WARPS, int OS>
__device__ __forceinline__ void finish_rows(const AttendParams& p, const WorkUnit& u, int row0,
                                            int R, const float* sM, const float* sL,
                                            const float* sO, float* sFin) {
  using namespace dev;
  constexpr float kLn2 = 0.69314718055994530942f;
  constexpr int NT = WARPS * 32, DQ = DV / 4;
  const int G = p.group, Hq = p.num_qo_heads, tid = threadIdx.x;
  const int rows = min(RB, R - row0);
  const bool partial = p.split && u.num_splits > 1;
  for (int idx = tid; idx < rows * DQ; idx += NT) {
    const int rr = idx / DQ, d = 4 * (idx % DQ), r = row0 + rr;
    float M = -INFINITY, L = 0.f;
    float mw[WARPS];
    float4 ow[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      mw[w] = sM[w * RB + rr];
      ow[w] = *reinterpret_cast<const float4*>(sO + (w * RB + rr) * OS + d);
      M = fmaxf(M, mw[w]);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        // 0 for -inf; as two halves, for maxima that differ by more than the sums do
        const float half = ex2(0.5f * (mw[w] - M)), sc = half * half;
        L = fmaf(sL[w * RB + rr] * half, half, L);
        if (mw[w] != -INFINITY) {
          o.x = fmaf(ow[w].x, sc, o.x);
          o.y = fmaf(ow[w].y, sc, o.y);
          o.z = fmaf(ow[w].z, sc, o.z);
          o.w = fmaf(ow[w].w, sc, o.w);
        }
      }
      const float inv = 1.f / L;
      o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    }
    const int i = r / G, head = u.h_kv * G + r % G;
    const int64_t row = (int64_t)(u.qo_begin + i) * Hq + head;
    if (!partial) {
      *reinterpret_cast<uint2*>(p.out + row * DV + d) =
          make_uint2(pack_out2(o.x, o.y, p.out_f16), pack_out2(o.z, o.w, p.out_f16));
      if (d == 0 && p.lse) p.lse[row] = M == -INFINITY ? M : (M + log2f(L)) * kLn2;
    } else {
      const int64_t pi = (int64_t)u.partial_base + ((int64_t)i * Hq + head) * u.num_splits + u.split;
      *reinterpret_cast<float4*>(p.partial_o + pi * DV + d) = o;
      if (d == 0) p.partial_lse[pi] = M == -INFINITY ? M : (M + log2f(L)) * kLn2;
    }
  }
  if (!partial) return;

  constexpr int IT = (RB * DQ + NT - 1) / NT < 2 ? 1 : 2;
  fold_if_last<RB, DV, NT, IT, IT == 1 ? 16 : 8>(p, u, row0, rows,
                                                 reinterpret_cast<int*>(sFin + 2 * RB), tid,
                                                 [] { __syncthreads(); });
}

}  // namespace nvfp4kv
