// page_ops.cu -- requests that share pages: forked, their last pages copied, and
// given up again, sm_103a.
//
// page_shares[p] counts the owners of page p beyond the first, so a page that the page
// table's kernel takes off the free list has its 0 already.
//
// fork: with L tokens of the parent in pages of P, the child gets the parent's L / P
// whole pages (one more owner each) and, for a last page that is not full, a new page
// off the free list, in the order of the forks; (the parent's last page, the new page)
// goes on the list of copies.
// release: request b keeps K_b of its L_b tokens and gives up the pages ceil(K_b / P) ..
// ceil(L_b / P) of its row.  A page whose last owner gives it up goes back in front of
// the free list's head; the pages freed stand there in the order in which the call lists
// them first (rows, then columns).
//
// Both are a list of (row, column) entries over rows of unequal lengths: every CTA takes
// the sums over the rows for itself (as in page_table.cu) and fills its share of the
// entries.  The order of a call's atomics changes no result: owners are counted up and
// down by whole numbers, and of several entries that give up one page the first in the
// list is found by a minimum.
//
// Latency bounds them: launches, the chain of loads that finds an entry, and (release) the
// pages' words, random sectors of L2 or HBM, four times.  Measured (replayed): 16 requests of
// 512-4096 tokens forked once 6.5 us and released 11; 64 requests of 500-16384 tokens forked 8
// times each (270 k table entries copied, then given up) 8.8 and 37, of which the last two
// passes' cluster takes 25 (16 SMs' loads of random words; all SMs would need a place for the
// counts between launches, which the call does not ask for); the copies of the last pages 3.1
// and 4.9 us (17 MB, 3.5 TB/s).
#include <climits>
#include <cstdint>
#include <mutex>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace nvfp4kv {
namespace {

constexpr int64_t kMaxLen = (int64_t)1 << 30;  // tokens of a request, as in the planner
constexpr int kForkThreads = 512;
constexpr int kChunk = 8;  // entries a lane has in flight

// the last entry of first[lo .. hi) that is <= x, where first[lo] <= x < first[hi]
__device__ __forceinline__ int owner(const int32_t* first, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// exclusive sums over the CTA of two counts a thread; the totals too
template <int THREADS>
__device__ __forceinline__ longlong2 cta_sums(longlong2 mine, longlong2* total) {
  __shared__ longlong2 s_warp[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  longlong2 run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, run.x, o);
    const long long y = __shfl_up_sync(0xffffffffu, run.y, o);
    if (lane >= o) {
      run.x += x;
      run.y += y;
    }
  }
  if (lane == 31) s_warp[warp] = run;
  __syncthreads();
  longlong2 before = make_longlong2(0, 0), all = before;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = all;
    all.x += s_warp[w].x;
    all.y += s_warp[w].y;
  }
  *total = all;
  return make_longlong2(before.x + run.x - mine.x, before.y + run.y - mine.y);
}

// ---- fork ---------------------------------------------------------------------
// Every CTA checks all forks for itself, the children's lengths among what it reads, so these
// are written (`lengths`) once all CTAs have read them: behind a barrier of the one cluster
// that the launch is, or, where more CTAs fill the table (`fill`), by a launch of one CTA
// behind it, which finds the same inputs: it may start and check while the table is filled,
// and waits for the end of that before it writes.  Measured (replayed; us): 2048 entries (one
// CTA) 5.6, 16384 (a cluster of 4) 6.4, 65536 8.2, with an ordinary second launch 10.1;
// everything in one CTA: 16384 13, 65536 51.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkParams p, bool fill,
                                                            bool lengths) {
  extern __shared__ int32_t smem[];
  const int F = p.num_forks, P = p.page_size;
  int32_t* s_first = smem;              // [F + 1] first entry (whole page) of each fork
  int32_t* s_free = s_first + F + 1;    // [F + 1] new pages that the forks before it take
  int32_t* s_parent = s_free + F + 1;   // [F]
  uint32_t* s_child = reinterpret_cast<uint32_t*>(s_parent + F);  // a bit a row: a child
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31;
  if (!lengths) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int head = *p.free_head;
  if (tid == 0) s_bad = 0;
  const int words = (p.num_rows + 31) / 32;
  for (int w = tid; w < words; w += kForkThreads) s_child[w] = 0u;
  __syncthreads();

  // ---- this thread's neighbouring forks ---------------------------------------
  const int per = (F + kForkThreads - 1) / kForkThreads;
  const int f0 = min(F, tid * per), f1 = min(F, f0 + per);
  longlong2 mine = make_longlong2(0, 0);
  bool bad = false;
  for (int f = f0; f < f1; ++f) {
    const int from = p.parents[f], to = p.children[f];
    if (from < 0 || from >= p.num_rows || to < 0 || to >= p.num_rows) {
      bad = true;
      continue;
    }
    // (a row that two forks fill)
    if (atomicOr(&s_child[to >> 5], 1u << (to & 31)) >> (to & 31) & 1u) bad = true;
    // (a row that holds a request: its pages would be in no row and not on the free list)
    if (p.kv_len[to] != 0) bad = true;
    const int len = p.kv_len[from];
    if (len < 0 || len > kMaxLen || (len + P - 1) / P > p.table_width) {
      bad = true;
      continue;
    }
    s_parent[f] = from;
    s_first[f] = len;  // kept here until its sum takes the place
    mine.x += len / P;
    mine.y += len % P > 0;
  }
  longlong2 total;
  longlong2 at = cta_sums<kForkThreads>(mine, &total);  // (its barrier completes s_child)
  for (int f = f0; f < f1 && !bad; ++f)  // a row that is filled and read
    bad = s_child[s_parent[f] >> 5] >> (s_parent[f] & 31) & 1u;
  if (bad) atomicOr(&s_bad, 1);
  // (also where nothing is to be written: what comes next must find the other launch done)
  if (!fill) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  if (s_bad || total.x > INT_MAX || head < 0 || head + total.y > p.num_free) {
    if (fill && blockIdx.x == 0 && tid == 0 && p.flags) atomicOr(p.flags, s_bad ? 0x40u : 0x80u);
    return;
  }
  if (lengths) cooperative_groups::this_cluster().sync();
  const int nt = gridDim.x * kForkThreads, me = blockIdx.x * kForkThreads + tid;
  for (int f = f0; f < f1; ++f) {
    const int len = s_first[f], whole = len / P;
    const bool rest = len % P > 0;
    s_first[f] = static_cast<int32_t>(at.x);
    s_free[f] = static_cast<int32_t>(at.y);
    at.x += whole;
    at.y += rest;
    // the fork's own words, by the one CTA whose turn it is
    if (f % gridDim.x != blockIdx.x) continue;
    const int child = p.children[f];
    if (lengths) p.kv_len[child] = len;
    if (!fill) continue;
    int src = -1, dst = -1;
    if (rest) {
      src = p.block_table[s_parent[f] * p.table_stride + whole];
      dst = p.free_pages[head + s_free[f]];
      p.block_table[child * p.table_stride + whole] = dst;
    }
    p.copy_src[f] = src;
    p.copy_dst[f] = dst;
  }
  if (!fill) return;
  if (tid == 0) s_first[F] = static_cast<int32_t>(total.x);
  if (me == 0) *p.free_head_out = head + static_cast<int>(total.y);
  __syncthreads();

  // ---- the whole pages: a warp takes 32 * kChunk neighbouring entries ------------
  const int entries = static_cast<int>(total.x);
  const int64_t stride = (int64_t)(nt / 32) * (32 * kChunk);
  for (int64_t e0 = (int64_t)(me / 32) * (32 * kChunk); e0 < entries; e0 += stride) {
    const int first = static_cast<int>(e0);
    const int stop = static_cast<int>(min(e0 + 32 * kChunk, (int64_t)entries));
    const int lo = owner(s_first, 0, F, first);
    const int hi = stop <= s_first[lo + 1] ? lo + 1 : owner(s_first, lo, F, stop - 1) + 1;
    int32_t id[kChunk];
    int32_t* to[kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int e = first + 32 * j + lane;
      to[j] = nullptr;
      if (e < stop) {
        const int f = owner(s_first, lo, hi, e), c = e - s_first[f];
        id[j] = p.block_table[s_parent[f] * p.table_stride + c];
        to[j] = p.block_table + __ldg(p.children + f) * p.table_stride + c;
      }
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      if (!to[j]) continue;
      *to[j] = id[j];
      if (id[j] >= 0 && id[j] < p.num_pages)
        atomicAdd(p.page_shares + id[j], 1);
      else if (p.flags)
        atomicOr(p.flags, 0x1u);
    }
  }
}

// ---- release --------------------------------------------------------------------
// Four passes over the entries, loads and atomics on the pages' words in L2:
//   1  every entry counts its page's owners down;
//   2  where that went below 0, the page is free: its word becomes the least of
//      INT_MIN + entry;
//   3  the entry that finds its own number there is the page's first;
//   4  it puts the page on the free list, at the place that the count of such entries
//      before it gives, and the word back to 0.
// A small call is one launch of one CTA, a larger one of a cluster, which keep their
// entries' pages in registers over the passes.  Where they have no room, passes 1 and 2 are
// launches over all SMs (the random words want many loads in flight), 3 and 4 one cluster
// whose barrier joins the counts.
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kUnits = 4;  // units of 32 entries that a warp has in flight
// Entries up to which one CTA is used.  Measured with every page given up (replayed; one CTA /
// a cluster / three launches, us): 256 entries 8.4 / 10.6 / 14.1, 1024 10.3 / 11.5 / 15.2, 2048
// 12.8 / 11.9 / 15.7, 4096 18.7 / 12.5 / 16.4, 32768 - / 16.2 / 18.9, 65536 (as many as a
// cluster's registers hold) - / 22.3 / 21.8, with a tenth given up 35 / 13.1 / 16.4; 131072
// - / 46.5 / 37.2.
constexpr int kOneCta = kThreads;
constexpr int kMostMarks = 8192;  // units of a CTA whose marks are kept (others: all looked at)

// The rows that give up pages, in shared memory: the first entry of each (and the count of
// all), the first column that it gives up and its number.
struct Leaving {
  int32_t* first;  // [rows + 1]
  int32_t* col;    // [rows]
  int32_t* row;    // [rows]
  int rows, entries;
};

// (every thread of the CTA)  false, and flagged if `report`: a call that cannot be
template <int THREADS>
__device__ __forceinline__ bool leaving_rows(const ReleaseParams& p, int32_t* smem, bool report,
                                             Leaving* out) {
  __shared__ int s_bad;
  const int B = p.num_rows, P = p.page_size, tid = threadIdx.x;
  Leaving s{smem, smem + B + 1, smem + 2 * B + 1, 0, 0};
  const int head = *p.free_head;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  longlong2 mine = make_longlong2(0, 0);
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int len = p.kv_len[b], keep = p.keep_len[b];
    bad = bad || len < 0 || len > kMaxLen || keep < 0 || keep > len ||
          (len + P - 1) / P > p.table_width;
    const int n = bad ? 0 : (len + P - 1) / P - (keep + P - 1) / P;
    mine.x += n;
    mine.y += n > 0;
  }
  if (bad) atomicOr(&s_bad, 1);
  longlong2 total;
  longlong2 at = cta_sums<THREADS>(mine, &total);  // (its barrier completes s_bad)
  // (an entry's number and INT_MIN add up in 32 bits)
  const bool stop = s_bad || total.x >= INT_MAX / 2 || head < 0 || head > p.num_free;
  for (int b = b0; b < b1 && !stop; ++b) {
    const int lo = (p.keep_len[b] + P - 1) / P, n = (p.kv_len[b] + P - 1) / P - lo;
    if (n == 0) continue;
    s.first[at.y] = static_cast<int32_t>(at.x);
    s.col[at.y] = lo;
    s.row[at.y] = b;
    at.x += n;
    ++at.y;
  }
  s.rows = static_cast<int>(total.y);
  s.entries = static_cast<int>(total.x);
  if (tid == 0 && !stop) s.first[s.rows] = s.entries;
  if (tid == 0 && stop && report && p.flags) atomicOr(p.flags, s_bad ? 0x40u : 0x80u);
  __syncthreads();
  *out = s;
  return !stop;
}

// The pages of kUnits units from unit u on, those that `wanted` has a bit for, an entry a
// lane; -1: no entry below `last`, or a page that is not in the pool (flagged if `report`).
// `row`: the leaving row of an entry before (the whole warp alike); it follows the units.
__device__ __forceinline__ void pages_of(const ReleaseParams& p, const Leaving& s, int u, int last,
                                         uint32_t wanted, bool report, int& row,
                                         int32_t (&pg)[kUnits]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int e0 = (u + j) * 32, e = e0 + lane;
    pg[j] = -1;
    if (e0 >= last || !(wanted >> j & 1u)) continue;
    while (s.first[row + 1] <= e0) ++row;
    int b = row;
    // (a row has an entry at least: 32 entries lie in 32 rows at most)
    if (s.first[row + 1] < min(e0 + 32, last)) b = owner(s.first, row, min(row + 32, s.rows), e);
    if (e < last) pg[j] = p.block_table[s.row[b] * p.table_stride + s.col[b] + (e - s.first[b])];
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j)
    if (pg[j] < 0 || pg[j] >= p.num_pages) {
      if (report && (wanted >> j & 1u) && (u + j) * 32 + lane < last && p.flags)
        atomicOr(p.flags, 0x1u);
      pg[j] = -1;
    }
}

// Pass 1 and pass 2 of the units in hand.
__device__ __forceinline__ void count_down(const ReleaseParams& p, const int32_t (&pg)[kUnits]) {
#pragma unroll
  for (int j = 0; j < kUnits; ++j)
    if (pg[j] >= 0) atomicSub(p.page_shares + pg[j], 1);
}
// (returns the lane's free pages, a bit a unit)
__device__ __forceinline__ uint32_t least_entry(const ReleaseParams& p, int u, int entries,
                                                const int32_t (&pg)[kUnits]) {
  const int lane = threadIdx.x & 31;
  int v[kUnits];
  uint32_t free = 0;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) v[j] = pg[j] >= 0 ? __ldcg(p.page_shares + pg[j]) : 0;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    if (v[j] >= 0) continue;
    free |= 1u << j;
    atomicMin(p.page_shares + pg[j], INT_MIN + (u + j) * 32 + lane);
    // given up more often than it has owners (whoever changes the word first has read it
    // before)
    if (v[j] < -1 && v[j] >= INT_MIN + entries && p.flags) atomicOr(p.flags, 0x200u);
  }
  return free;
}

// Pass 1 or 2 over all SMs.
constexpr int kPassThreads = 256;
__global__ void __launch_bounds__(kPassThreads) release_pass_kernel(const ReleaseParams p,
                                                                    int pass) {
  extern __shared__ int32_t smem[];
  Leaving s;
  if (!leaving_rows<kPassThreads>(p, smem, false, &s)) return;
  const int units = (s.entries + 31) / 32, warps = gridDim.x * (kPassThreads / 32);
  const int share = (units + warps - 1) / warps;
  const int w = blockIdx.x * (kPassThreads / 32) + (threadIdx.x >> 5);
  const int u0 = static_cast<int>(min((int64_t)w * share, (int64_t)units));
  const int u1 = min(units, u0 + share), last = min(u1 * 32, s.entries);
  if (u0 == u1) return;
  int row = owner(s.first, 0, s.rows, u0 * 32);
  for (int u = u0; u < u1; u += kUnits) {
    int32_t pg[kUnits];
    pages_of(p, s, u, last, ~0u, pass == 1, row, pg);
    if (pass == 1)
      count_down(p, pg);
    else
      least_entry(p, u, s.entries, pg);
  }
}

// All passes (from = 1) or the last two (from = 3), one cluster.
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseParams p, int from) {
  namespace cg = cooperative_groups;
  extern __shared__ int32_t smem[];
  uint32_t* s_mark = reinterpret_cast<uint32_t*>(smem + 3 * p.num_rows + 1);  // [p.marks]
  __shared__ int s_freed[kWarps], s_mine;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = *p.free_head;
  Leaving s;
  // (every CTA alike, before the cluster's first barrier)
  if (!leaving_rows<kThreads>(p, smem, rank == 0, &s)) return;

  // this warp's units of 32 entries: neighbours, so that the free list keeps their order
  const int units = (s.entries + 31) / 32, warps = ranks * kWarps;
  const int share = (units + warps - 1) / warps;
  const int u0 = static_cast<int>(min((int64_t)(rank * kWarps + warp) * share, (int64_t)units));
  const int u1 = min(units, u0 + share), last = min(u1 * 32, s.entries);
  const int row0 = u0 < u1 ? owner(s.first, 0, s.rows, u0 * 32) : 0;
  const bool once = u1 - u0 <= kUnits;  // the pages stay in registers
  const bool marked = share * kWarps <= p.marks;
  uint32_t* mark = s_mark + warp * share;  // the entries of unit u0 + k that are first
  int row = row0;
  int32_t pg[kUnits];
  auto hold = [&](int u, uint32_t wanted, bool report) {
    pages_of(p, s, u, last, wanted, report, row, pg);
  };
  if (once) hold(u0, ~0u, from == 1);
  if (from == 1) {
    for (int u = u0; u < u1; u += kUnits) {
      if (!once) hold(u, ~0u, true);
      count_down(p, pg);
    }
    cluster.sync();
    row = row0;
    for (int u = u0; u < u1; u += kUnits) {
      if (!once) hold(u, ~0u, false);
      least_entry(p, u, s.entries, pg);
    }
    cluster.sync();
  }
  int freed = 0;
  row = row0;
  uint32_t firsts = 0;  // of the units in hand, a bit a unit
  auto find_firsts = [&](int u) {
    int v[kUnits];
    firsts = 0;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) v[j] = pg[j] >= 0 ? __ldcg(p.page_shares + pg[j]) : 0;
#pragma unroll
    for (int j = 0; j < kUnits; ++j)
      if (v[j] == INT_MIN + (u + j) * 32 + lane) firsts |= 1u << j;
  };
  for (int u = u0; u < u1; u += kUnits) {
    if (!once) hold(u, ~0u, false);
    find_firsts(u);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const uint32_t votes = __ballot_sync(0xffffffffu, firsts >> j & 1u);
      freed += __popc(votes);
      if (marked && lane == 0 && u + j < u1) mark[u + j - u0] = votes;
    }
  }
  if (lane == 0) s_freed[warp] = freed;
  __syncthreads();
  if (tid == 0) {
    int sum = 0;
    for (int w = 0; w < kWarps; ++w) sum += s_freed[w];
    s_mine = sum;
  }
  cluster.sync();
  int before = 0, all = 0;
  for (int k = 0; k < ranks; ++k) {
    const int n = *cluster.map_shared_rank(&s_mine, k);
    if (k < rank) before += n;
    all += n;
  }
  for (int w = 0; w < warp; ++w) before += s_freed[w];
  cluster.sync();  // (no CTA ends, and no word of a page is put back, while another reads)
  // More than were ever taken: the words are put back as they were (to -1 by the first
  // entry, then up by every one), nothing is listed.
  const bool undo = all > head;
  int place = head - all + before;
  row = row0;
  for (int u = u0; u < u1; u += kUnits) {
    uint32_t wanted = ~0u;
    if (marked) {
      wanted = __ballot_sync(0xffffffffu, lane < kUnits && u + lane < u1 &&
                                              mark[min(u + lane, u1 - 1) - u0] != 0);
      if (wanted == 0) continue;
    }
    if (!once) {
      hold(u, wanted, false);
      find_firsts(u);
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const bool mine = firsts >> j & 1u;
      const uint32_t votes = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        if (!undo) p.free_pages[place + __popc(votes & ((1u << lane) - 1u))] = pg[j];
        __stcg(p.page_shares + pg[j], undo ? -1 : 0);
      }
      place += __popc(votes);
    }
  }
  if (undo) {
    cluster.sync();
    row = row0;
    for (int u = u0; u < u1; u += kUnits) {
      if (!once) hold(u, ~0u, false);
      for (int j = 0; j < kUnits; ++j)
        if (pg[j] >= 0) atomicAdd(p.page_shares + pg[j], 1);
    }
    if (rank == 0 && tid == 0 && p.flags) atomicOr(p.flags, 0x80u);
    return;
  }
  for (int b = rank * kThreads + tid; b < p.num_rows; b += ranks * kThreads)
    p.kv_len[b] = p.keep_len[b];
  if (rank == 0 && tid == 0) *p.free_head_out = head - all;
}

// ---- copies -----------------------------------------------------------------------
// A warp takes a head of one copy: its rows' pieces, 16 bytes of codes or `small` bytes
// of scales, four a lane in flight.
__global__ void __launch_bounds__(128) copy_kernel(const PageCopyParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= (int64_t)p.num * p.num_kv_heads) return;
  const int i = static_cast<int>(id / p.num_kv_heads), h = static_cast<int>(id % p.num_kv_heads);
  const int src = p.src[i], dst = p.dst[i];
  if (src == -1 && dst == -1) return;  // nothing to copy
  if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages) {
    if (lane == 0 && p.flags) atomicOr(p.flags, 0x1u);
    return;
  }
  if (src == dst) return;
#pragma unroll 1
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t* from = p.data[kv] + src * p.sp[kv] + h * p.sh[kv];
    uint8_t* to = p.data[kv] + dst * p.sp[kv] + h * p.sh[kv];
    const int wide = p.row_bytes[kv] / 16, items = p.page_size * wide;
    for (int it0 = lane; it0 - lane < items; it0 += 128) {
      uint4 v[4];
      int64_t at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int it = it0 + 32 * k, row = it / wide;
        at[k] = row * p.ss[kv] + (it - row * wide) * 16;
        if (it < items) v[k] = *reinterpret_cast<const uint4*>(from + at[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (it0 + 32 * k < items) *reinterpret_cast<uint4*>(to + at[k]) = v[k];
    }
    from = p.scale[kv] + src * p.scp[kv] + h * p.sch[kv];
    to = p.scale[kv] + dst * p.scp[kv] + h * p.sch[kv];
    if (p.page_scales) {  // one a page and head
      if (lane == 0) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
      continue;
    }
    const int small = p.scale_bytes[kv] % 4 ? 2 : 4, each = p.scale_bytes[kv] / small;
    for (int it = lane; it < p.page_size * each; it += 32) {
      const int row = it / each;
      const int64_t off = row * p.scs[kv] + (it - row * each) * small;
      if (small == 4)
        *reinterpret_cast<uint32_t*>(to + off) = *reinterpret_cast<const uint32_t*>(from + off);
      else
        *reinterpret_cast<uint16_t*>(to + off) = *reinterpret_cast<const uint16_t*>(from + off);
    }
  }
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const int words = (p.num_rows + 31) / 32;
  constexpr int kMaxSmem = (3 * kMaxForks + 2 + kMaxForkRows / 32) * 4;
  const int smem = (3 * p.num_forks + 2 + words) * 4;
  if (smem > 40 * 1024) {
    // the most that any call takes: another thread's call must not find less
    cudaError_t e = cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  // at most two CTAs an SM (more would only repeat the sums), as many as the forks' rows
  // could fill; up to 8 as a cluster of a power of two
  int64_t blocks = ((int64_t)p.num_forks * p.table_width / kChunk + kForkThreads) / kForkThreads;
  if (blocks > 152 * 2) blocks = 152 * 2;
  const bool one = blocks <= 8;
  if (one && blocks > 1) blocks = blocks > 4 ? 8 : blocks > 2 ? 4 : 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kForkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = one ? static_cast<unsigned>(blocks) : 1;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fork_kernel, p, true, one);
  if (e != cudaSuccess || one) return e;
  cfg.gridDim = dim3(1);
  attr = cudaLaunchAttribute{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, fork_kernel, p, false, true);
}

// The largest cluster that the current device takes of release_kernel: 16 CTAs, or the 8
// that every device does.
static cudaError_t release_cluster(int smem, int* ctas) {
  static std::mutex mu;
  static int known[64];  // of the first devices; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && known[dev] != 0) {
    *ctas = known[dev];
    return cudaSuccess;
  }
  e = cudaFuncSetAttribute(release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(release_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  e = cudaOccupancyMaxActiveClusters(&clusters, release_kernel, &cfg);
  if (e != cudaSuccess) {
    cudaGetLastError();
    clusters = 0;
  }
  *ctas = clusters > 0 ? 16 : 8;
  if (dev < 64) known[dev] = *ctas;
  return cudaSuccess;
}

cudaError_t launch_release(ReleaseParams p, cudaStream_t stream) {
  constexpr int kRowsSmem = (3 * kMaxPageTableBatch + 1) * 4;
  constexpr int kMaxSmem = kRowsSmem + kMostMarks * 4;
  int ctas = 8;
  cudaError_t e = release_cluster(kMaxSmem, &ctas);
  if (e != cudaSuccess) return e;
  const int rows_smem = (3 * p.num_rows + 1) * 4;
  const int64_t most = (int64_t)p.num_rows * p.table_width;
  int from = 1;
  if (most <= kOneCta) {
    ctas = 1;
  } else if (most > (int64_t)ctas * kWarps * kUnits * 32) {
    if (rows_smem > 40 * 1024) {
      e = cudaFuncSetAttribute(release_pass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kRowsSmem);
      if (e != cudaSuccess) return e;
    }
    const int64_t want = most / (32 * kUnits * (kPassThreads / 32)) + 1;
    const int grid = static_cast<int>(want < 152 * 4 ? want : 152 * 4);
    for (int pass = 1; pass <= 2; ++pass)
      release_pass_kernel<<<grid, kPassThreads, rows_smem, stream>>>(p, pass);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    from = 3;
  }
  const int64_t units = ((most + 31) / 32 + ctas * kWarps - 1) / (ctas * kWarps) * kWarps;
  p.marks = static_cast<int>(units < kMostMarks ? units : kMostMarks);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = rows_smem + p.marks * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, release_kernel, p, from);
}

cudaError_t launch_page_copies(const PageCopyParams& p, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.num * p.num_kv_heads;
  if (warps == 0) return cudaSuccess;
  copy_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
