// compact.cu -- the accepted tokens of a drafted tree moved together in their pages,
// sm_103a.
//
// Request b holds L_b tokens, the last n_b of them drafted.  Of these the nodes
// path[b][0] < path[b][1] < ... < path[b][c_b - 1] were accepted: the token at position
// L_b - n_b + path[b][i] goes to position L_b - n_b + i, in every head of K and V, as if
// all were read before any is written.  path[b][i] >= i, so a token only ever moves
// down; the tokens behind the last one moved are left as they were.
//
// 4-bit cache, and 1-token pages of the E4M3 cache: a token's codes and scales are its
// own and are moved as bytes.
// E4M3 pages of 16 tokens share a scale a head: the page that the tokens go to gets the
// largest scale of the pages that its tokens come from (its own among them where it
// keeps older tokens), and codes of a page with a smaller scale become
// E4M3_RNE(code * (its scale / the new one)), exact but for subnormal codes (scales are
// powers of two).
//
// Latency bounds it: a launch and four dependent loads (lengths, path, page ids, codes),
// then the stores.  Measured (replayed): 6 of 16 drafted tokens of each of 16 requests, 4-bit
// cache, 4.3 us; 38 of 40-64 of 256 requests, E4M3 cache, 13.3 us (20 MB, 1.5 TB/s: three
// rounds of a page a head, each a chain of its own).  In place without a copy: a target holds a token that no later target
// of the list needs (its sources lie further up), so it is enough that the tokens of one
// round are all loaded, into registers, before the round's stores.
#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "internal.h"

namespace nvfp4kv {
namespace {

// One request of the call: what its warps need.
struct Drafts {
  int64_t begin;         // first drafted position
  int count;             // accepted nodes
  const int32_t* path;
  const int32_t* pages;  // the request's page ids
};

// (the whole warp together)  false where nothing is to be done, flagged where the
// request cannot be
__device__ __forceinline__ bool drafts_of(const CompactParams& p, int b, int lane, bool report,
                                          Drafts* d) {
  const int count = p.num_kept[b];
  const int r0 = p.qo_indptr[b], r1 = p.qo_indptr[b + 1];
  const int k0 = p.kv_indptr[b], k1 = p.kv_indptr[b + 1], last = p.last_page_len[b];
  if (count == 0) return false;
  const int64_t n = (int64_t)r1 - r0, np = (int64_t)k1 - k0;
  const int64_t len = (np - 1) * p.page_size + last;
  bool ok = count > 0 && n >= count && count <= p.path_width && k0 >= 0 && np >= 1 && last >= 1 &&
            last <= p.page_size && len >= n;
  d->begin = len - n;
  d->count = count;
  d->path = p.path + b * p.path_stride;
  d->pages = p.kv_indices + k0;
  if (ok) {  // nodes in order, all of the tree
    bool good = true;
    for (int i = lane; i < count; i += 32) {
      const int x = d->path[i], before = i > 0 ? d->path[i - 1] : -1;
      good = good && x > before && x < n;
    }
    ok = __all_sync(0xffffffffu, good);
  }
  if (!ok && report && lane == 0 && p.flags) atomicOr(p.flags, 0x2u);
  return ok;
}

// Tokens moved as bytes.  A warp takes a (request, head, K or V); its items are the
// pieces of the tokens' rows: 16 bytes of codes, or `small` bytes of scales (2 where the
// row of scales is no multiple of 4 bytes).
constexpr int kItems = 8;  // a lane has in flight
__global__ void __launch_bounds__(128) compact_bytes_kernel(const CompactParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int per = 2 * p.num_kv_heads;
  if (id >= (int64_t)p.batch * per) return;
  const int b = static_cast<int>(id / per), r = static_cast<int>(id % per);
  const int kv = r & 1, h = r >> 1;
  Drafts d;
  if (!drafts_of(p, b, lane, r == 0, &d)) return;
  const int wide = p.row_bytes[kv] / 16, small = p.scale_bytes[kv] % 4 ? 2 : 4;
  const int pieces = wide + p.scale_bytes[kv] / small;
  uint8_t* data = p.data[kv] + h * p.sh[kv];
  uint8_t* scale = p.scale[kv] + h * p.sch[kv];
  const int chunk = max(1, 32 * kItems / pieces);  // (at most 32 pieces of codes and 8 of scales)
  auto place = [&](int64_t pos, bool* ok) -> int64_t {  // page and slot of a position
    const int64_t pg = pos / p.page_size;
    const int id = d.pages[pg];
    if (id < 0 || id >= p.num_pages) {
      *ok = false;
      if (p.flags) atomicOr(p.flags, 0x1u);
    }
    return (int64_t)id << 32 | (pos - pg * p.page_size);
  };
  for (int i0 = 0; i0 < d.count; i0 += chunk) {
    const int items = min(chunk, d.count - i0) * pieces;
    uint4 v[kItems];
    uint8_t* to[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      to[k] = nullptr;
      const int it = lane + 32 * k;
      if (it >= items) continue;
      const int i = i0 + it / pieces, piece = it % pieces, node = d.path[i];
      if (node == i) continue;  // where it belongs already
      bool ok = true;
      const int64_t s = place(d.begin + node, &ok), t = place(d.begin + i, &ok);
      if (!ok) continue;
      const bool sc = piece >= wide;
      const int64_t sp = sc ? p.scp[kv] : p.sp[kv], ss = sc ? p.scs[kv] : p.ss[kv];
      uint8_t* base = sc ? scale + (piece - wide) * small : data + piece * 16;
      const uint8_t* from = base + (s >> 32) * sp + (s & 0xFFFFFFFF) * ss;
      to[k] = base + (t >> 32) * sp + (t & 0xFFFFFFFF) * ss;
      if (!sc)
        v[k] = *reinterpret_cast<const uint4*>(from);
      else if (small == 4)
        v[k].x = *reinterpret_cast<const uint32_t*>(from);
      else
        v[k].x = *reinterpret_cast<const uint16_t*>(from);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (!to[k]) continue;
      if ((lane + 32 * k) % pieces < wide)
        *reinterpret_cast<uint4*>(to[k]) = v[k];
      else if (small == 4)
        *reinterpret_cast<uint32_t*>(to[k]) = v[k].x;
      else
        *reinterpret_cast<uint16_t*>(to[k]) = static_cast<uint16_t>(v[k].x);
    }
    __syncwarp();
  }
}

// four E4M3 codes times f
__device__ __forceinline__ uint32_t recoded(uint32_t w, float f) {
  const float2 lo = dev::unpack2<true>(dev::e4m3x2_to_f16x2(w & 0xFFFFu));
  const float2 hi = dev::unpack2<true>(dev::e4m3x2_to_f16x2(w >> 16));
  unsigned short a, b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(lo.y * f), "f"(lo.x * f));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi.y * f), "f"(hi.x * f));
  return a | (uint32_t)b << 16;
}

// E4M3 pages of 16 tokens.  A CTA takes a (request, head, K or V), a warp one of the
// pages that its tokens go to; NCH 16-byte chunks a lane hold a page's rows of one head.
constexpr int kPageWarps = 4;
template <int NCH>
__global__ void __launch_bounds__(32 * kPageWarps) compact_e4m3_kernel(const CompactParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = 2 * p.num_kv_heads;
  const int b = static_cast<int>(blockIdx.x / per), r = static_cast<int>(blockIdx.x % per);
  const int kv = r & 1, h = r >> 1;
  Drafts d;
  if (!drafts_of(p, b, lane, r == 0 && warp == 0, &d)) return;  // (every warp alike)
  const int pieces = p.row_bytes[kv] / 16;
  uint8_t* data = p.data[kv] + h * p.sh[kv];
  uint8_t* scales = p.scale[kv] + h * p.sch[kv];
  const int64_t first = d.begin / kPageSize;
  const int pages = static_cast<int>((d.begin + d.count - 1) / kPageSize - first) + 1;
  for (int g = 0; g < pages; g += kPageWarps) {
    const int64_t pg = first + g + warp;
    bool live = g + warp < pages;
    // lane s (and s + 16): where slot s's token comes from
    const int slot = lane & 15;
    const int64_t rank = pg * kPageSize + slot - d.begin;
    const bool fresh = live && rank >= 0 && rank < d.count, old = live && rank < 0;
    int64_t source = pg * kPageSize + slot;
    if (fresh) source = d.begin + d.path[rank];
    int target = 0, from = 0;
    float had = 0.f;
    if (live) target = d.pages[pg];
    if (fresh || old) {
      from = d.pages[source / kPageSize];
      if (from < 0 || from >= p.num_pages || target < 0 || target >= p.num_pages) {
        if (p.flags) atomicOr(p.flags, 0x1u);
        live = false;  // (a page that is not in the pool: its tokens stay where they are)
      } else {
        const float s = *reinterpret_cast<const float*>(scales + from * p.scp[kv]);
        had = dev::clamped_scale(s);
        if (had != s && p.flags) atomicOr(p.flags, 0x20u);
      }
    }
    live = __all_sync(0xffffffffu, live);
    float now = had;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
    const float f = had > 0.f ? __fdiv_rn(had, now) : 1.f;
    const int64_t at = from * p.sp[kv] + (source & (kPageSize - 1)) * p.ss[kv];
    // a row is written where its token moved or its scale did
    const bool moved = (fresh && source != pg * kPageSize + slot) || ((fresh || old) && f != 1.f);
    uint4 v[NCH];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int it = lane + 32 * k, row = it / pieces;
      const int64_t row_at = __shfl_sync(0xffffffffu, at, row & 15);
      const bool takes = __shfl_sync(0xffffffffu, moved, row & 15);
      if (live && takes && row < kPageSize)
        v[k] = *reinterpret_cast<const uint4*>(data + row_at + (it % pieces) * 16);
    }
    __syncthreads();  // the round's tokens and scales are in registers
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int it = lane + 32 * k, row = it / pieces;
      const float fr = __shfl_sync(0xffffffffu, f, row & 15);
      const bool takes = __shfl_sync(0xffffffffu, moved, row & 15);
      if (live && takes && row < kPageSize) {
        if (fr != 1.f)
          v[k] = make_uint4(recoded(v[k].x, fr), recoded(v[k].y, fr), recoded(v[k].z, fr),
                            recoded(v[k].w, fr));
        *reinterpret_cast<uint4*>(data + target * p.sp[kv] + row * p.ss[kv] +
                                  (it % pieces) * 16) = v[k];
      }
    }
    if (live && lane == 0) *reinterpret_cast<float*>(scales + target * p.scp[kv]) = now;
    __syncthreads();  // (the next round's sources lie behind this one's targets)
  }
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.batch * 2 * p.num_kv_heads;
  if (units == 0) return cudaSuccess;
  if (!p.page_scales || p.page_size == 1) {
    compact_bytes_kernel<<<static_cast<unsigned>((units + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const unsigned grid = static_cast<unsigned>(units);
  const int row = p.row_bytes[0] > p.row_bytes[1] ? p.row_bytes[0] : p.row_bytes[1];
  if (row <= 128)
    compact_e4m3_kernel<4><<<grid, 32 * kPageWarps, 0, stream>>>(p);
  else if (row <= 256)
    compact_e4m3_kernel<8><<<grid, 32 * kPageWarps, 0, stream>>>(p);
  else
    compact_e4m3_kernel<16><<<grid, 32 * kPageWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
