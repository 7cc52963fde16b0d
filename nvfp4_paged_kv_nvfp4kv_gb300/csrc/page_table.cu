// page_table.cu -- the step's page table and slot maps from request lengths,
// sm_103a.
//
// Request b holds L_b tokens after the step, n_b of them new, in pages of P
// tokens: every_b = ceil(L_b / P) pages, of which held_b = ceil((L_b - n_b) /
// P) stand in its row of the block table already; the other taken_b = every_b
// - held_b come off the free list in request order.  With the exclusive sums
// Q, K, F of n, every, taken over the requests:
//   page c of request b:  table[b][c]                       c < held_b
//                         free[head + F_b + c - held_b]     otherwise
//   kv_indices[K_b + c] = that page,
//   row Q_b + i: request b, position L_b - n_b + i, slot page * P + pos % P.
//
// Latency bounds the small calls and the table's bytes the large ones (4 B in
// and 4 B out per page).  One launch serves both: every CTA takes the three
// sums over all requests for itself (a few loads a thread; a second launch or
// a grid-wide wait would cost more than the loads), keeps them in shared
// memory and fills its share of the flat page and row lists, 256 neighbouring
// pages a warp at a time: two binary searches give the requests that they span.
// Whether the batch fits is known to every CTA after the sums, so a batch that
// does not fit writes nothing but the flag.
// Measured: 64 requests, one token each, 8.2 us replayed (lengths, sums, searches,
// ids and their stores one after another, 6 us of it the launch itself); 1000
// requests with 4.1 million pages 18.5 us, 2.0 TB/s: the same chain, then 13
// thousand page ids a CTA in three or four rounds of loads.
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace nvfp4kv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 8;
constexpr int64_t kMaxLen = (int64_t)1 << 30;  // tokens of a request, as in the planner

struct Sums {
  int64_t tokens, pages, taken;  // 64 bits: the totals are checked before they are narrowed
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tokens + b.tokens, a.pages + b.pages, a.taken + b.taken};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.tokens, o), __shfl_up_sync(0xffffffffu, a.pages, o),
          __shfl_up_sync(0xffffffffu, a.taken, o)};
}

// the last entry of first[lo .. hi) that is <= x, where first[lo] <= x < first[hi]
__device__ __forceinline__ int owner(const int32_t* first, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_table_kernel(const PageTableParams p) {
  extern __shared__ int32_t smem[];
  const int B = p.batch, P = p.page_size;
  int32_t* s_qo = smem;              // [B + 1] first row
  int32_t* s_kv = s_qo + B + 1;      // [B + 1] first page
  int32_t* s_free = s_kv + B + 1;    // [B + 1] first page taken
  int32_t* s_len = s_free + B + 1;   // [B]
  __shared__ Sums s_warp[kWarps];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = p.free_head ? *p.free_head : 0;
  if (tid == 0) s_bad = 0;

  // ---- the sums: this thread's neighbouring requests, then the CTA ---------
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  Sums mine{0, 0, 0};
  bool bad = false;
  auto item = [&](int len, int n) -> Sums {
    const int every = (len + P - 1) / P, held = (len - n + P - 1) / P;
    return {n, every, every - held};
  };
  for (int b = b0; b < b1; ++b) {
    const int len = p.kv_len[b], n = p.qo_len[b];
    if (n < 0 || len < n || len > kMaxLen || (len + P - 1) / P > p.table_width) {
      bad = true;
      continue;
    }
    s_len[b] = len;
    s_qo[b] = n;  // kept here until its sum takes the place
    mine = mine + item(len, n);
  }
  Sums run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up = shfl_up(run, o);
    if (lane >= o) run = run + up;
  }
  if (lane == 31) s_warp[warp] = run;
  __syncthreads();
  if (bad) atomicOr(&s_bad, 1);
  Sums before{0, 0, 0}, total{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = total;
    total = total + s_warp[w];
  }
  __syncthreads();
  if (s_bad || total.tokens > p.max_tokens || total.pages > p.max_pages || head < 0 ||
      (int64_t)head + total.taken > p.num_free) {
    if (blockIdx.x == 0 && tid == 0 && p.flags)
      atomicOr(p.flags, s_bad ? 0x40u : 0x80u);
    return;
  }
  Sums at{before.tokens + run.tokens - mine.tokens, before.pages + run.pages - mine.pages,
          before.taken + run.taken - mine.taken};
  for (int b = b0; b < b1; ++b) {
    const int len = s_len[b];
    const Sums add = item(len, s_qo[b]);
    s_qo[b] = (int32_t)at.tokens;
    s_kv[b] = (int32_t)at.pages;
    s_free[b] = (int32_t)at.taken;
    at = at + add;
  }
  if (tid == 0) {
    s_qo[B] = (int32_t)total.tokens;
    s_kv[B] = (int32_t)total.pages;
    s_free[B] = (int32_t)total.taken;
  }
  __syncthreads();

  // ---- the lists -----------------------------------------------------------
  const int nt = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
  for (int b = me; b <= B; b += nt) {
    p.qo_indptr[b] = s_qo[b];
    p.kv_indptr[b] = s_kv[b];
    if (b < B) {
      const int every = s_kv[b + 1] - s_kv[b];
      p.last_page_len[b] = every > 0 ? s_len[b] - (every - 1) * P : 0;
    }
  }
  if (me == 0) *p.free_head_out = head + (int)total.taken;

  const int pages = (int)total.pages, tokens = (int)total.tokens;
  // A warp takes kChunk * 32 neighbouring pages at a time: two searches give
  // the requests they span (one, for long requests nearly always), a lane's
  // own searches stay between those, and its loads, independent of one
  // another, are on their way together.
  const int nw = gridDim.x * kWarps;
  for (int64_t k0 = (int64_t)(blockIdx.x * kWarps + warp) * (32 * kChunk); k0 < pages;
       k0 += (int64_t)nw * (32 * kChunk)) {
    const int first = (int)k0, stop = (int)min(k0 + 32 * kChunk, (int64_t)pages);
    const int lo = owner(s_kv, 0, B, first);
    const int hi = stop <= s_kv[lo + 1] ? lo + 1 : owner(s_kv, lo, B, stop - 1) + 1;
    if (hi == lo + 1) {
      const int kv0 = s_kv[lo], taken = s_free[lo + 1] - s_free[lo];
      const int held = s_kv[lo + 1] - kv0 - taken, end = stop - kv0;
      int32_t* row = p.block_table + lo * p.table_stride;
      const int32_t* fresh = p.free_pages + (head + s_free[lo]);  // page `held` on
      const int c0 = first - kv0 + lane;
      int32_t id[kChunk];
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const int c = c0 + 32 * j;
        if (c < end) id[j] = c < held ? row[c] : fresh[c - held];
      }
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const int c = c0 + 32 * j;
        if (c < end) {
          p.kv_indices[kv0 + c] = id[j];
          if (c >= held) row[c] = id[j];
        }
      }
      continue;
    }
    int32_t id[kChunk];
    int32_t* enter[kChunk];  // where a taken page goes in the table
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int k = first + 32 * j + lane;
      enter[j] = nullptr;
      if (k < stop) {
        const int b = owner(s_kv, lo, hi, k), c = k - s_kv[b];
        const int taken = s_free[b + 1] - s_free[b], held = s_kv[b + 1] - s_kv[b] - taken;
        int32_t* at = p.block_table + b * p.table_stride + c;
        if (c >= held) enter[j] = at;
        id[j] = c < held ? *at : p.free_pages[head + s_free[b] + c - held];
      }
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int k = first + 32 * j + lane;
      if (k < stop) p.kv_indices[k] = id[j];
      if (enter[j]) *enter[j] = id[j];
    }
  }
  for (int64_t t = me; t < tokens; t += nt) {
    const int b = owner(s_qo, 0, B, (int)t);
    const int n = s_qo[b + 1] - s_qo[b];
    const int pos = s_len[b] - n + ((int)t - s_qo[b]);
    p.batch_idx[t] = b;
    p.positions[t] = pos;
    if (p.slot_map) {
      const int c = pos / P;
      const int taken = s_free[b + 1] - s_free[b], held = s_kv[b + 1] - s_kv[b] - taken;
      // (another CTA may be writing the table's new entries: they are taken
      // from the free list here too)
      const int32_t id = c < held ? p.block_table[b * p.table_stride + c]
                                  : p.free_pages[head + s_free[b] + c - held];
      p.slot_map[t] = (int64_t)id * P + pos % P;
    }
  }
}

}  // namespace

cudaError_t launch_page_table(const PageTableParams& p, cudaStream_t stream) {
  constexpr int kMaxSmem = (4 * kMaxPageTableBatch + 3) * 4;
  const int smem = (4 * p.batch + 3) * 4;
  if (smem > 40 * 1024) {
    // the most that any call takes: another thread's call must not find less
    cudaError_t e = cudaFuncSetAttribute(page_table_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  // one CTA per kWarps chunks of pages or kThreads rows, at most two an SM:
  // more would only repeat the sums
  const int64_t work = (int64_t)p.max_pages / kChunk + p.max_tokens + 1;
  int64_t blocks = (work + kThreads - 1) / kThreads;
  if (blocks > 152 * 2) blocks = 152 * 2;
  page_table_kernel<<<static_cast<int>(blocks), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
