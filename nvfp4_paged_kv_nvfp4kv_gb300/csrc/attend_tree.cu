// attend_tree.cu -- attention of drafted trees over the paged NVFP4 cache on the
// fifth-generation tensor cores, for more than 16 query rows a kv head and, of few short
// requests, more than 8, sm_103a.
//
// Row r (a node of request b's tree and a head of the kv head's group) sees token t where
//   t < L_b - n_b                       (before the tree), or
//   bit t - (L_b - n_b) of its words    (itself and what it continues);
//   s_t = sm_scale * q . k_t,  o = sum_t p_t v_t / sum_t p_t,  p_t = exp(s_t),
//   lse = ln sum_t p_t; a row that sees nothing has o = 0 and lse = -inf.
//
// One CTA takes up to 128 query rows on the M side of both products, so a tile of keys is
// dequantised once for all of them and a softmax row belongs to two threads:
//  * K and V loaders (a warp for each 32 tokens x 128 dims of a tile): cp.async of the packed
//    rows and scales (a warp its own tokens, RS tiles ahead), then e2m1 -> f16 times the
//    E4M3 block scale (exact) into the 128-byte-swizzled operand layouts in shared memory;
//  * issue (two warps, one thread each): S = Q K^T (A = Q in tensor memory, N = TT tokens),
//    and O += P V (A = P in tensor memory), each once its inputs are ready;
//  * softmax (8 warps): thread = row and half of the tile's tokens, so the maximum and the
//    sum need no shuffles.  Each half has an O, a maximum and a sum of its own, joined at the
//    end; where tensor memory has no room for that (ONE: 512 query dims), the halves share
//    them and meet in a barrier of their two warps once a tile.  The maximum is raised only
//    when a score exceeds it by 2^8 (then O is rescaled).  Sums are float32 of the unrounded
//    p; P is rounded to f16 (2^-11), the operand's type.  A tile that reaches into the tree
//    takes each row's 64 (32) bits at once.
// Value dims beyond 128 go to another CTA (VH of them), which forms the same S.
//
// The plan splits long requests for its own row blocks; here a cluster of CTAs divides a
// unit's tokens (and value dims) further, as many as the SMs allow, or those of all units of
// a request and kv head (uneven batches: in several waves, the longest first), and joins its
// states through distributed shared memory: no workspace beyond the plan's is needed, and
// each CTA stores a share of the rows.  Units of a split request that a cluster does not take
// as one fold as elsewhere (log-sum-exp over partial states, by the last CTA to arrive: 2.8
// us, and 0.4 for each state of 64 rows).
// Every wait is bounded; one that runs out sets flag 0x4 and the CTA winds down.
//
// Measured (replayed): 4 requests x 32771 tokens, 104 rows of 8 kv heads (128/128) 78 us, 720
// TFLOP/s of the rows that are there; 16 requests of 512-4096 tokens x 64 rows 39 us; 8
// requests of 2048-8192 tokens x 48-88 rows (512/256) 45 us; with the step's tokens appended in
// the launch 82, 40 and 48.  Neither memory (1.9 TB/s) nor
// the tensor cores (a third busy) are full: the softmax warps' chain of a tile (wait, load,
// maximum, 2^x, store: 2200 cycles of 128 tokens) and, at 512 dims, the dequantisation bound
// it, with half of the issue slots taken and an eighth of the warps' time spent fetching
// instructions; of the 39 us, 12 are the wait for the longest unit and 7 a CTA's start and end.
// Measured and not kept, against the kernel as it then was (16 requests / 4 x 32771 tokens /
// 512 dims): products issued by the loaders' first warps, which leaves 128 registers a thread,
// 53 / 120 / 64 for 42 / 89 / 47 us; barriers of their own for the halves' S 44 / 92 / 47;
// loaders of K and of V in code of their own 43 / 92 / 49 for 40 / 87 / 47; a half's blocks of
// 32 tokens one after the other, half the registers, 38 / 97 / 45 for 39 / 84 / 45; twice the
// CTAs, in two waves, 57 / 105 / 71; other shares of registers (setmaxnreg) slower.
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda_runtime.h>

#include "append_fused.cuh"
#include "device_common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace nvfp4kv {
namespace {

using namespace dev;
using namespace tc5;

constexpr int kRows = 128;
constexpr int kSoftmaxWarps = 8;
constexpr float kRaise = 8.f;  // log2 of the largest p before m is raised
// Test build only: the first K loader of CTA (0, 0) withholds its arrival for the first
// tile, so the issuer's wait runs out and the CTA winds down.
#ifndef NVFP4KV_TREE_TEST_SKIP_ARRIVE
#define NVFP4KV_TREE_TEST_SKIP_ARRIVE 0
#endif

// DVC: value dims of a CTA, DV = VH * DVC; TT: tokens of a tile.  ONE: the two halves of a
// tile's tokens share one O (and so one maximum), where tensor memory has no room for two.
template <int DK, int DVC, int VH, int TT, bool ONE>
struct Tree {
  static constexpr int DV = DVC * VH;
  // loader threads of a token's K and V: 64 or 128 dims each
  static constexpr int KP = DK > 128 ? DK / 128 : 1, VP = DVC > 128 ? DVC / 128 : 1;
  static constexpr int KLW = TT * KP / 32, VLW = TT * VP / 32;  // loader warps
  static constexpr int THREADS = 32 * (kSoftmaxWarps + KLW + VLW + 2);
  static constexpr int BT = TT / 4;                 // tokens of a softmax thread's block
  static constexpr int SEG = DK / 2 / KP, SF = DK / 16 / KP;  // packed and scale bytes of each
  static_assert(DVC / 2 / VP == SEG, "one loader for both");
  static constexpr int WARP = 32 * (SEG + SF);                // a warp's stage
  static constexpr int STAGE = (KLW + VLW) * WARP;
  static constexpr int KBYTES = TT * DK * 2, VBYTES = TT * DVC * 2;   // operand tiles
  static constexpr int KB = 2, VB = DK == 512 ? 2 : 3;
  static constexpr int RS = DK == 512 ? 2 : DK == 128 ? 3 : 4;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KB * KBYTES;
  static constexpr int OFF_RAW = OFF_V + VB * VBYTES;
  static constexpr int OFF_MISC = OFF_RAW + RS * STAGE;
  static constexpr int MISC = 256 + 6 * kRows * 4 + 64;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;  // + alignment slack
  static constexpr int OROW = DVC + 4;                 // floats of a row in the joined states
  // tensor memory columns: S, P, O of each half, Q
  static constexpr int SCOL = 0, PCOL = TT, OCOL = PCOL + TT / 2;
  static constexpr int QCOL = OCOL + (ONE ? 1 : 2) * DVC;
  static constexpr int COLS = QCOL + DK / 2, TCOLS = 512;
  static constexpr uint32_t IDESC_S = idesc_f16(kRows, TT, 0, 0);
  static constexpr uint32_t IDESC_O = idesc_f16(kRows, DVC, 0, 1);
  static_assert(COLS <= TCOLS && SMEM <= 232448, "resources");
  static_assert(2 * (SMEM + 1024) > 233472, "one CTA an SM: two clusters that share SMs might "
                                            "each hold the tensor memory that the other wants");
  static_assert(OFF_RAW % 1024 == 0 && OFF_MISC % 16 == 0, "alignment");
  static_assert(kRows * OROW * 4 <= OFF_RAW, "the joined states take the operands' place");
};

// wait_bar for a barrier that mostly is ready, or soon will be: tested first, as the
// suspending wait takes about 300 cycles even when it is
template <int SPINS>
__device__ __forceinline__ bool wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* flags) {
#pragma unroll 1
  for (int k = 0; k < SPINS; ++k)
    if (mbar_test_wait(bar, parity)) return true;
  return wait_bar(bar, parity, abort, flags);
}
// One lane of a warp that is there as a whole.  What it then runs counts as uniform: the
// descriptors of its products stay in uniform registers (issued behind lane == 0 instead, a
// product takes 80 to 100 cycles, 64 tokens x 16 dims 32).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n"
               ::: "memory");
}
// the address of shared memory `a` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_v4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ void sts_v4(uint32_t a, int off, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {  // (off: a constant once unrolled)
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a + off), "r"(x), "r"(y),
               "r"(z), "r"(w)
               : "memory");
}
// 4 elements of a row's output (the output is 4-byte aligned)
__device__ __forceinline__ void store_out4(uint16_t* at, const float4& o, bool f16) {
  uint32_t* w = reinterpret_cast<uint32_t*>(at);
  w[0] = pack_out2(o.x, o.y, f16);
  w[1] = pack_out2(o.z, o.w, f16);
}
// a token's scales: 4, 8 or 16 bytes
template <int N>
__device__ __forceinline__ void cp_async_sf(uint32_t s, const void* g) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(s), "l"(g));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(s), "l"(g), "n"(N));
}

// 16-byte chunk c of row r in a warp's stage (rows of SEG bytes): the lanes of a quarter
// warp, a row each, then read distinct banks
template <int SEG>
__device__ __forceinline__ int raw_chunk(int r, int c) {
  if constexpr (SEG == 32) return c ^ ((r >> 2) & 1);
  if constexpr (SEG == 64) return c ^ ((r >> 1) & 3);
  return c ^ (r & 7);
}

// Loader warp w of K or (of_v) V: its rows of the tiles [t0, t0 + ntiles) of unit u.  One code
// for both, as the warps wait for instructions otherwise.
template <class T, int TT>
__device__ __forceinline__ void load_tiles(const AttendParams& p, const WorkUnit& u, bool of_v,
                                           int w, int lane, int t0, int ntiles, int tok_end,
                                           int vh, uint8_t* smem, int q_stage, uint64_t* full,
                                           uint64_t* empty, uint64_t* q_full,
                                           volatile int* abort) {
  constexpr int SEG = T::SEG, SF = T::SF, RS = T::RS;
  const int bytes = of_v ? T::VBYTES : T::KBYTES, num = of_v ? T::VB : T::KB;
  constexpr int LPR = SEG / 16, RPI = 32 / LPR;  // lanes a row, rows a copy instruction
  const CacheView& c = p.cache;
  const int seg = w / (TT / 32);           // part of the row's dims
  const int first = 32 * (w % (TT / 32));  // this warp's first token of a tile
  const int shift = p.page_size == 1 ? 0 : 4, slots = (1 << shift) - 1;
  const int64_t sp = of_v ? c.v_sp : c.k_sp, ss = of_v ? c.v_ss : c.k_ss;
  const int64_t fsp = of_v ? c.vsf_sp : c.ksf_sp, fss = of_v ? c.vsf_ss : c.ksf_ss;
  const int part = of_v ? vh * T::VP + seg : seg;  // the warp's part of the whole row
  const uint8_t* data = (of_v ? c.v_data + u.h_kv * c.v_sh : c.k_data + u.h_kv * c.k_sh) + part * SEG;
  const uint8_t* sf = (of_v ? c.v_sf + u.h_kv * c.vsf_sh : c.k_sf + u.h_kv * c.ksf_sh) + part * SF;
  const int tiles = of_v ? T::OFF_V : T::OFF_K;
  const uint32_t mine = smem_addr(smem) + T::OFF_RAW + ((of_v ? T::KLW : 0) + w) * T::WARP;
  const int r0 = lane / LPR, ch = lane % LPR;
  // page id of this lane's token in tile i, a tile ahead of its use (where it is checked);
  // a token past the unit's pages takes the last one
  auto load_pid = [&](int i) -> int32_t {
    if (i >= ntiles) return 0;
    const int rel = (t0 + i) * TT + first + lane;
    return __ldg(p.kv_indices + u.page_begin + min(rel >> shift, u.num_pages - 1));
  };
  // (rows r0, r0 + RPI, ... of the warp's 32 tokens, which begin at a multiple of 16)
  const uint8_t* from = data + (r0 & slots) * ss + 16 * ch;
  const uint8_t* sf_from = sf + (lane & slots) * fss;
  auto issue = [&](uint32_t st, int32_t pid) {
    if (pid < 0 || pid >= c.num_pages) {
      atomicOr(p.flags, 0x1u);
      pid = 0;
    }
    const uint8_t* page = from;
#pragma unroll
    for (int k = 0; k < LPR; ++k) {
      const int r = r0 + k * RPI;
      // 16-token pages: the copies of a page differ by whole steps of RPI slots
      constexpr int PER = RPI < 16 ? 16 / RPI : 1;
      if (shift == 0 || RPI > 16 || k % PER == 0)
        page = from + __shfl_sync(0xffffffffu, pid, r) * sp;
      cp_async_16s(st + r * SEG + 16 * raw_chunk<SEG>(r, ch),
                   shift == 0 ? page : page + (k % PER) * (RPI * ss));
    }
    cp_async_sf<SF>(st + 32 * SEG + lane * SF, sf_from + pid * fsp);
  };
  int32_t pids[RS];
#pragma unroll
  for (int i = 0; i < RS; ++i) pids[i] = load_pid(i);
#pragma unroll
  for (int i = 0; i < RS; ++i) {
    if (i < ntiles) issue(mine + i * T::STAGE, pids[i]);
    cp_async_commit();
  }
  int32_t next = load_pid(RS);
  uint32_t st = mine;  // the stage of tile i
  const int tl = first + lane;  // this lane's token of a tile
  // its row, whose 16-byte chunks are xor-ed with the row's number
  const uint32_t row = smem_addr(smem) + tiles + (tl >> 3) * 1024 + (tl & 7) * 128 + ((tl & 7) << 4);
  // (Q's rows lie at the end of the operand tiles until they are read)
  if (ntiles > 0 && tiles + num * bytes > q_stage &&
      !__all_sync(0xffffffffu, wait_bar(q_full, 0, abort, p.flags)))
    ntiles = 0;
  for (int i = 0, b = 0, round = 0; i < ntiles; ++i) {
    cp_async_wait<RS - 1>();  // this thread's copies of tile i have landed
    __syncwarp();             // and those of the warp
    // slots past the request's end may hold a NaN scale: their values count as 0 (their
    // scores are replaced)
    const bool past = u.tok_begin + (t0 + i) * TT + tl >= tok_end;
    uint32_t scales[SF / 4];
#pragma unroll
    for (int k = 0; k < SF / 4; ++k) {
      scales[k] = lds_u32(st + 32 * SEG + lane * SF + 4 * k);
      if (past) scales[k] = 0;
    }
    uint4 q[LPR];
#pragma unroll
    for (int k = 0; k < LPR; ++k) q[k] = lds_v4(st + lane * SEG + 16 * raw_chunk<SEG>(lane, k));
    if (round > 0 &&
        !__all_sync(0xffffffffu, wait_soon<4>(&empty[b], (round - 1) & 1, abort, p.flags)))
      break;
    uint32_t out[8];  // the row's chunk c of each block of 64 dims
#pragma unroll
    for (int c8 = 0; c8 < 8; ++c8)
      out[c8] = (row + b * bytes + (2 * SEG / 64 * seg) * (TT * 128)) ^ (c8 << 4);
#pragma unroll
    for (int k = 0; k < LPR; ++k) {
      const uint32_t s2 = e4m3x2_to_f16x2(scales[k / 2] >> (16 * (k & 1)));
      const uint32_t lo = bcast_lo(s2), hi = bcast_hi(s2);
      const uint32_t words[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t h[4];
        e2m1x8_to_f16x8(words[e], h);
        const uint32_t s = e < 2 ? lo : hi;
        const int d = 32 * k + 8 * e;  // first of the 8 dims, from the thread's first
        static_assert(2 * SEG % 64 == 0, "a thread's dims fill blocks of 64");
        sts_v4(out[d % 64 / 8], d / 64 * (TT * 128), hmul2(h[0], s), hmul2(h[1], s),
               hmul2(h[2], s), hmul2(h[3], s));
      }
    }
    fence_async_smem();
    __syncwarp();
    const bool withhold = NVFP4KV_TREE_TEST_SKIP_ARRIVE && !of_v && blockIdx.x == 0 &&
                          blockIdx.y == 0 && w == 0 && i == 0;
    if (lane == 0 && !withhold) mbar_arrive(&full[b]);
    if (i + RS < ntiles) issue(st, next);  // (the warp has read the stage)
    cp_async_commit();
    next = load_pid(i + RS + 1);
    st = st == mine + (RS - 1) * T::STAGE ? mine : st + T::STAGE;
    if (++b == num) {
      b = 0;
      ++round;
    }
  }
  cp_async_wait<0>();
}

// The first unit of a pair of request and kv head (-1: none): the pair of this number, or
// (sorted) the one that as many are longer than.  `len`: room for a word a unit.  (A function
// of its own: inlined, it costs the loop over the tiles registers, 78 -> 83 us on 4 x 32771
// tokens.  The append or the fold of their own cost as much: 79 and 91 us.)
__device__ __noinline__ int first_unit(const WorkUnit* units, int num, int number, bool sorted,
                                       int* len, int* found) {
  if (threadIdx.x == 0) *found = -1;
  for (int i = threadIdx.x; sorted && i < num; i += blockDim.x)
    len[i] = units[i].split == 0 ? units[i].kv_len : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < num; i += blockDim.x) {
    if (units[i].split != 0) continue;
    int at = sorted ? 0 : units[i].pair;
    for (int k = 0; sorted && k < num; ++k) at += len[k] > len[i] || (len[k] == len[i] && k < i);
    if (at == number) *found = i;
  }
  __syncthreads();
  return *found;
}

template <int DK, int DVC, int VH, int TT, bool ONE>
__global__ void __launch_bounds__(Tree<DK, DVC, VH, TT, ONE>::THREADS, 1)
    attend_tree_kernel(const AttendParams p) {
  using T = Tree<DK, DVC, VH, TT, ONE>;
  constexpr int KB = T::KB, VB = T::VB, DV = T::DV, kThreads = T::THREADS;
  constexpr int kKWarp = kSoftmaxWarps, kVWarp = kKWarp + T::KLW, kSWarp = kVWarp + T::VLW;
  constexpr float kLn2 = 0.69314718055994530942f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_MISC);
  uint64_t* k_full = bars;        // [KB] K tile in its operand layout
  uint64_t* k_empty = bars + 3;   // [KB] S done
  uint64_t* v_full = bars + 6;    // [VB]
  uint64_t* v_empty = bars + 9;   // [VB] O done
  uint64_t* s_full = bars + 12;   // S done -> softmax
  uint64_t* s_empty = bars + 13;  // S read -> issue
  uint64_t* p_full = bars + 14;   // softmax -> issue
  uint64_t* pv_done = bars + 15;  // O done -> softmax
  uint64_t* q_full = bars + 18;
  uint64_t* fin = bars + 19;      // [2] wind-down of the two issuers' products
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 22);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_last = reinterpret_cast<int*>(s_tmem + 2);
  float* s_x = reinterpret_cast<float*>(smem + T::OFF_MISC + 256);  // [2][128] the halves' values
  float* s_ml = s_x + 2 * kRows;  // [2][128] the halves' maxima
  float* s_m = s_ml + 2 * kRows;  // [128] maxima, then
  float* s_l = s_m + kRows;       // [128] sums of the CTA's state

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int unit = blockIdx.x;
  if (p.tree_whole > 0) {
    unit = first_unit(p.units, p.tree_whole, unit, p.tree_sorted, reinterpret_cast<int*>(smem),
                      s_last);
    if (unit < 0) return;  // a request without rows
  }
  WorkUnit u = load_unit(p, unit, tid == 0);
  if (p.tree_whole > 0) {
    u.num_splits = 1;
    u.num_pages = (u.kv_len + p.page_size - 1) / p.page_size;
  }
  if (tid == 0) {  // (while the unit is on its way)
    for (int b = 0; b < KB; ++b) {
      mbar_init(&k_full[b], T::KLW);
      mbar_init(&k_empty[b], 1);
    }
    for (int b = 0; b < VB; ++b) {
      mbar_init(&v_full[b], T::VLW);
      mbar_init(&v_empty[b], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_empty, kSoftmaxWarps);
    mbar_init(p_full, kSoftmaxWarps);
    mbar_init(pv_done, 1);
    mbar_init(q_full, kSoftmaxWarps);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    mbar_init_fence();
    *s_abort = 0;
  }
  if (warp == kSoftmaxWarps) {
    tmem_alloc(s_tmem, T::TCOLS);
    tmem_relinquish();
  }
  const int G = p.group, R = G * u.qo_len, C = p.tree_ctas;
  const int block = blockIdx.y / C, rank = blockIdx.y % C;
  const int vh = rank % VH, part = rank / VH, parts = C / VH;
  const int row0 = block * kRows;
  if (row0 >= R) {  // the whole cluster
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftmaxWarps) tmem_dealloc(*s_tmem, T::TCOLS);
    return;
  }
  const int nrows = min(kRows, R - row0);
  // Up to 64 rows are held twice: the copies share each half's tokens, so that all warps
  // work (16 requests of 512-4096 tokens x 64 rows 48 -> 41 us).
  const int rows_held = nrows <= kRows / 2 ? kRows / 2 : kRows;
  // this CTA's tiles of the unit; tokens from tok_end on do not exist
  const int tok_end = min(u.kv_len, u.tok_begin + p.page_size * u.num_pages);
  const int all_tiles = (tok_end - u.tok_begin + TT - 1) / TT;
  const int t0 = static_cast<int>((int64_t)all_tiles * part / parts);
  const int ntiles = static_cast<int>((int64_t)all_tiles * (part + 1) / parts) - t0;

  // Q's rows on their way to tensor memory: whole lines at a time to shared memory, the end of
  // the operand tiles' place, their 16-byte chunks xor-ed with the row's number (a
  // thread's row straight from global memory would be a line a lane)
  const int q_stage = T::OFF_RAW - nrows * (DK * 2);
  if (warp < kSoftmaxWarps) {
    constexpr int CH = DK / 8;
    for (int idx = tid; idx < nrows * CH; idx += 32 * kSoftmaxWarps) {
      const int rr = idx / CH, c = idx % CH, gr = row0 + rr, node = gr / G;
      cp_async_16s(smem_addr(smem) + q_stage + rr * (DK * 2) + 16 * (c ^ (rr & 7)),
                   p.q + (int64_t)(u.qo_begin + node) * p.q_stride_tok +
                       (int64_t)(u.h_kv * G + gr - node * G) * p.q_stride_head + 8 * c);
    }
    cp_async_commit();
  }
  // fused append: the step's new tokens among this CTA's tiles, stored before any copy
  // reads them (CTAs that share tokens store the same bytes)
  if (p.new_k != nullptr) {
    const int lo = max(u.kv_len - u.qo_len, u.tok_begin + t0 * TT);
    const int hi = min(tok_end, u.tok_begin + (t0 + ntiles) * TT);
    if (lo < hi) append_unit_tokens<DK, DV>(p, u, lo, hi, tid, kThreads);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= kKWarp && warp < kSWarp) {
    const bool of_v = warp >= kVWarp;
    load_tiles<T, TT>(p, u, of_v, warp - (of_v ? kVWarp : kKWarp), lane, t0, ntiles, tok_end, vh,
                      smem, q_stage, of_v ? v_full : k_full, of_v ? v_empty : k_empty, q_full,
                      s_abort);
  } else if (warp == kSWarp) {
    // ================= issue of S = Q K^T (one thread) =========================
    if (elect_one()) {
      const uint64_t kd0 = smem_desc(smem_addr(smem + T::OFF_K), 16, 1024, kSwz128);
      bool ok = ntiles == 0 || wait_bar(q_full, 0, s_abort, p.flags);
      for (int i = 0, b = 0, round = 0; ok && i < ntiles; ++i) {
        ok = wait_soon<64>(&k_full[b], round & 1, s_abort, p.flags) &&
             (i == 0 || wait_soon<64>(s_empty, (i - 1) & 1, s_abort, p.flags));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = kd0 + ((b * T::KBYTES) >> 4);
#pragma unroll 8
        for (int kk = 0; kk < DK / 16; ++kk)
          umma_ts(tmem + T::SCOL, tmem + T::QCOL + 8 * kk,
                  kd + (((kk >> 2) * (TT * 128) + (kk & 3) * 32) >> 4), T::IDESC_S,
                  kk > 0 ? 1u : 0u);
        umma_commit(s_full);
        umma_commit(&k_empty[b]);
        if (++b == KB) {
          b = 0;
          ++round;
        }
      }
      umma_commit(&fin[0]);  // wind-down: every product issued has completed
      drain_bar(&fin[0], 0, p.flags);
    }
    __syncwarp();
  } else if (warp == kSWarp + 1) {
    // ================= issue of O += P V (one thread) ===========================
    if (elect_one()) {
      const uint64_t vd0 = smem_desc(smem_addr(smem + T::OFF_V), TT * 128, 1024, kSwz128);
      for (int i = 0, b = 0, round = 0; i < ntiles; ++i) {
        if (!wait_soon<64>(&v_full[b], round & 1, s_abort, p.flags) ||
            !wait_soon<64>(p_full, i & 1, s_abort, p.flags))
          break;
        tc_fence_after();
        const uint64_t vd = vd0 + ((b * T::VBYTES) >> 4);
#pragma unroll
        for (int k = 0; k < TT / 16; ++k) {
          const int h = ONE ? 0 : 16 * k / T::BT & 1;  // the half whose tokens these are
          const bool first = ONE ? k == 0 : 16 * k == h * T::BT;
          umma_ts(tmem + T::OCOL + h * DVC, tmem + T::PCOL + 8 * k, vd + ((k * 2048) >> 4),
                  T::IDESC_O, (i > 0 || !first) ? 1u : 0u);
        }
        umma_commit(pv_done);
        umma_commit(&v_empty[b]);
        if (++b == VB) {
          b = 0;
          ++round;
        }
      }
      umma_commit(&fin[1]);
      drain_bar(&fin[1], 0, p.flags);
    }
    __syncwarp();
  } else {
    // ================= softmax (thread = row, half of a tile's tokens) ===========
    const int q4 = warp & 3, half = warp >> 2, r = 32 * q4 + lane;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int copy = r / rows_held;  // of the row (0 where rows are not held twice)
    const int row_r = r - copy * rows_held;
    const bool active = 32 * q4 - copy * rows_held < nrows;  // warp-uniform
    const bool real = row_r < nrows;
    const int gr = row0 + (real ? row_r : 0), node = gr / G;
    // ---- Q: bf16 -> f16 times a power of two per row, into tensor memory ----------
    float f = 0.f;
    {
      const uint32_t q = smem_addr(smem) + q_stage + (real ? row_r : 0) * (DK * 2);
      auto load = [&](int c) -> uint4 {
        return real ? lds_v4(q + 16 * ((half * (DK / 16) + c) ^ (row_r & 7)))
                    : make_uint4(0u, 0u, 0u, 0u);
      };
      cp_async_wait<0>();
      named_sync(5, 32 * kSoftmaxWarps);
      float am = 0.f;
      if (active) {
#pragma unroll 8
        for (int c = 0; c < DK / 16; ++c) {
          const uint4 v = load(c);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            am = fmax3(am, fabsf(bf16_bits_to_f32(w[e] & 0xFFFFu)),
                       fabsf(bf16_bits_to_f32(w[e] >> 16)));
        }
        s_x[half * kRows + r] = am;
        named_sync(1 + q4, 64);
        am = fmaxf(am, s_x[(half ^ 1) * kRows + r]);
        int e = 0;  // amax * 2^e in [2^14, 2^15)
        if (am > 0.f) e = 14 - (int)((__float_as_uint(am) >> 23) & 0xFF) + 127;
        e = max(-120, min(120, e));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        // (above 0: it multiplies the -inf of tokens that are not seen)
        f = real ? fmaxf(p.qk_scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 0x1p-126f)
                 : 0.f;
#pragma unroll 2
        for (int c = 0; c < DK / 64; ++c) {  // 16 columns of two dims
          uint32_t h[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = load(4 * c + k);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
              h[4 * k + x] = f32x2_to_f16x2(bf16_bits_to_f32(w[x] & 0xFFFFu) * up,
                                            bf16_bits_to_f32(w[x] >> 16) * up);
          }
          tmem_st16(tmem + lane_base + T::QCOL + half * (DK / 4) + 16 * c, h);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    // ---- the tiles ---------------------------------------------------------------------
    const int before = u.kv_len - u.qo_len;  // tokens that every row sees
    const uint32_t* words = p.tree_mask + (int64_t)(u.qo_begin + node) * p.tree_words;
    auto word = [&](int k) -> uint32_t { return k < p.tree_words ? __ldg(words + k) : 0u; };
    // bit t: whether the row sees token tok + t (t < 32)
    auto visible = [&](int tok) -> uint32_t {
      const int j = tok - before, n = tok_end - tok;
      uint32_t v;
      if (j <= -32) {
        v = ~0u;
      } else if (j < 0) {
        v = word(0) << -j | ((1u << -j) - 1);
      } else {
        v = __funnelshift_r(word(j >> 5), word((j >> 5) + 1), j & 31);
      }
      if (n < 32) v = n <= 0 ? 0u : v & ((1u << n) - 1);
      return real ? v : 0u;
    };
    // the maximum (log2; ONE: of the row, else of this half's tokens), -m once there is one
    float m = -INFINITY, nm = 0.f;
    float thr = real ? -INFINITY : INFINITY;
    uint64_t lsum[2] = {0, 0};  // sums of p (ONE: over this half's tokens)
    const int some_hidden = min(before, tok_end);  // tiles that reach past it are masked
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // (every lane: no hand-over)
      wait_soon<16>(bar, parity, s_abort, p.flags);
      __syncwarp();
    };
    // A half has two blocks of a tile's tokens, the first and the third quarter or the second
    // and the fourth.  NB: the blocks that this thread looks at, from block k0.
    constexpr int BT = T::BT;
    auto tiles = [&](auto blocks, int k0) {
      constexpr int NB = decltype(blocks)::value;
      for (int i = 0; i < ntiles; ++i) {
        const int tok = u.tok_begin + (t0 + i) * TT + half * BT;
        const bool masked = u.tok_begin + (t0 + i + 1) * TT > some_hidden;
        wait(s_full, i & 1);
        tc_fence_after();
        uint32_t x[NB * BT];
#pragma unroll
        for (int k = 0; k < NB; ++k)
          tmem_ld<BT>(tmem + lane_base + T::SCOL + (k0 + k) * (TT / 2) + half * BT, x + k * BT);
        tmem_wait_ld<NB * BT>(x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        if (masked) {
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            const uint32_t see = visible(tok + (k0 + k) * (TT / 2));
#pragma unroll
            for (int e = 0; e < BT; ++e)
              if (!(see >> e & 1u)) x[k * BT + e] = 0xff800000u;  // -inf
          }
        }
        // the largest score (f > 0, so that of the sums); f = 0 for rows that are not there
        float mx[4] = {__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]),
                       __uint_as_float(x[3])};
#pragma unroll
        for (int e = 4; e + 7 < NB * BT; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmax3(mx[k], __uint_as_float(x[e + 2 * k]), __uint_as_float(x[e + 2 * k + 1]));
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(x[NB * BT - 4 + k]));
        float top = fmaf(fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]), f, nm);
        bool raise = top > thr;
        if constexpr (ONE)
          raise = named_or(1 + q4, 64, raise);
        else
          raise = __any_sync(0xffffffffu, raise);
        if (raise) {
          // ---- raise the maxima to this tile's ---------------------------------------
          if constexpr (ONE) {
            s_x[half * kRows + r] = top;
            named_sync(1 + q4, 64);
            top = fmaxf(top, s_x[(half ^ 1) * kRows + r]);
          }
          float corr = 1.f;
          if (real && top != -INFINITY && (m == -INFINITY || top > 0.f)) {
            if (m != -INFINITY) corr = ex2(-top);
            m = (m == -INFINITY ? 0.f : m) + top;
            nm = -m;
            thr = kRaise;
          }
          if (i > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
            float a, b;
            unpack_f32x2(add_f32x2(lsum[0], lsum[1]), a, b);
            lsum[0] = pack_f32x2((a + b) * corr, 0.f);
            lsum[1] = 0;
            wait(pv_done, (i - 1) & 1);
            tc_fence_after();
            constexpr int OD = ONE ? DVC / 2 : DVC;  // the dims that are this thread's to scale
#pragma unroll 1
            for (int c = 0; c < OD / 8; ++c) {
              uint32_t ov[8];
              const uint32_t oa = tmem + lane_base + T::OCOL + half * OD + 8 * c;
              tmem_ld8(oa, ov);
              tmem_wait_ld<8>(ov);
#pragma unroll
              for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
              tmem_st8(oa, ov);
            }
          }
        }
        // ---- p = 2^(score - m) ----------------------------------------------------------
        uint32_t h[NB * BT / 2];
        {
          const uint64_t f2 = pack_f32x2(f, f), n2 = pack_f32x2(nm, nm);
#pragma unroll
          for (int e = 0; e < NB * BT / 2; ++e) {
            float a, b;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[2 * e]),
                                              __uint_as_float(x[2 * e + 1])), f2, n2), a, b);
            a = ex2(a);
            b = ex2(b);
            lsum[e & 1] = add_f32x2(lsum[e & 1], pack_f32x2(a, b));
            h[e] = f32x2_to_f16x2(a, b);
          }
        }
        if (i > 0) wait(pv_done, (i - 1) & 1);  // P's columns are free
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < NB; ++k)
          tmem_st<BT / 2>(tmem + lane_base + T::PCOL + (k0 + k) * (TT / 4) + half * (BT / 2),
                          h + k * (BT / 2));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
    };
    if (!active) {
      // (nothing to do for the rows that are not there but to keep the counts)
      for (int i = 0; i < ntiles; ++i) {
        wait(s_full, i & 1);
        if (lane == 0) mbar_arrive(s_empty);
        if (i > 0) wait(pv_done, (i - 1) & 1);  // (an arrival counts for the phase that is open)
        if (lane == 0) mbar_arrive(p_full);
      }
    } else if (rows_held < kRows) {
      // the other copy's block: its weights are 0 for this row
      uint32_t zero[BT / 2] = {};
      tmem_st<BT / 2>(tmem + lane_base + T::PCOL + (1 - copy) * (TT / 4) + half * (BT / 2), zero);
      tiles(std::integral_constant<int, 1>{}, copy);
    } else {
      tiles(std::integral_constant<int, 2>{}, 0);
    }
    // ---- the CTA's state: sums of the halves, then O ------------------------------------
    if (active) {
      if (ntiles > 0) wait(pv_done, (ntiles - 1) & 1);
      float l;
      {
        float a, b;
        unpack_f32x2(add_f32x2(lsum[0], lsum[1]), a, b);
        l = a + b;
      }
      // (only now: the other half may have been reading the words for its last raise)
      s_x[half * kRows + r] = l;
      if constexpr (!ONE) s_ml[half * kRows + r] = m;
      named_sync(1 + q4, 64);
      const float l1 = s_x[(half ^ 1) * kRows + r];
      float w[2] = {1.f, 1.f};  // the factors of the halves' O
      if constexpr (ONE) {
        l += l1;
      } else {
        const float m1 = s_ml[(half ^ 1) * kRows + r], top = fmaxf(m, m1);
        const float mine = m == -INFINITY ? 0.f : ex2(m - top);
        const float other = m1 == -INFINITY ? 0.f : ex2(m1 - top);
        // (the same sum in both threads: each row's first half first)
        l = half ? fmaf(l1, other, l * mine) : fmaf(l, mine, l1 * other);
        w[0] = half ? other : mine;
        w[1] = half ? mine : other;
        m = top;
      }
      tc_fence_after();
      const bool any = m != -INFINITY;
      const uint32_t oa = tmem + lane_base + T::OCOL + half * (DVC / 2);
      // 16 dims of the row, the halves' states joined
      auto state16 = [&](int c, float (&o)[16]) {
        uint32_t ov[16];
        tmem_ld16(oa + 16 * c, ov);
        if constexpr (ONE) {
          tmem_wait_ld<16>(ov);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = any ? __uint_as_float(ov[e]) : 0.f;
        } else {
          uint32_t ow[16];
          tmem_ld16(oa + DVC + 16 * c, ow);
          tmem_wait_ld<16>(ov);
          tmem_wait_ld<16>(ow);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = (w[0] != 0.f ? __uint_as_float(ov[e]) * w[0] : 0.f) +
                   (w[1] != 0.f ? __uint_as_float(ow[e]) * w[1] : 0.f);
        }
      };
      if (parts == 1 && rows_held == kRows) {
        const bool partial = p.split && u.num_splits > 1;
        const float scale = any ? p.v_scale / l : 0.f;
        const float lse = any ? (m + log2f(l)) * kLn2 : -INFINITY;
        const int head = u.h_kv * G + gr % G;
        const int64_t row = (int64_t)(u.qo_begin + node) * p.num_qo_heads + head;
        const int64_t pi = (int64_t)u.partial_base +
                           ((int64_t)node * p.num_qo_heads + head) * u.num_splits + u.split;
        if (real && half == 0 && vh == 0) {
          if (partial)
            p.partial_lse[pi] = lse;
          else if (p.lse)
            p.lse[row] = lse;
        }
        const int d0 = vh * DVC + half * (DVC / 2);
#pragma unroll 1
        for (int c = 0; c < DVC / 32; ++c) {
          float o[16];
          state16(c, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= scale;
          if (real && partial) {
            float4* at = reinterpret_cast<float4*>(p.partial_o + pi * DV + d0 + 16 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              at[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else if (real) {
            uint32_t* at = reinterpret_cast<uint32_t*>(p.out + row * DV + d0 + 16 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e) at[e] = pack_out2(o[2 * e], o[2 * e + 1], p.out_f16);
          }
          __syncwarp();
        }
      } else {
        // (the operand tiles are free: every product is done)
        float* so = reinterpret_cast<float*>(smem) + r * T::OROW + half * (DVC / 2);
        if (half == 0) {
          s_m[r] = m;
          s_l[r] = l;
        }
#pragma unroll 1
        for (int c = 0; c < DVC / 32; ++c) {
          float o[16];
          state16(c, o);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<float4*>(so + 16 * c + 4 * e) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
    }
    tc_fence_before();
  }

  // ---- every role is done: release tensor memory ---------------------------------------
  __syncthreads();
  if (warp == kSoftmaxWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, T::TCOLS);
  }
  const bool partial = p.split && u.num_splits > 1;
  const int copies = kRows / rows_held;
  if (parts * copies > 1) {
    // ---- join the states of the rows' copies in the cluster's CTAs, a share of the rows each
    __syncwarp();
    if (parts > 1) cluster_arrive_wait();
    const int n = parts * copies;  // states of a row (a power of two, at most 16)
    const int share = rows_held / parts, first = part * share;  // n * share = kRows
    const int rows = min(share, nrows - first);
    const uint32_t so = smem_addr(smem);
    if (tid < kRows) {  // a lane a state: its weight in its row's result, to s_x
      const int s = tid % n, rr = first + tid / n;
      const int at = s / copies * VH + vh, row = rr + s % copies * rows_held;
      const float m = peer_f32(peer(smem_addr(s_m) + 4 * row, at));
      const float l = peer_f32(peer(smem_addr(s_l) + 4 * row, at));
      float top = m;
      for (int k = 1; k < n; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const bool any = top != -INFINITY;
      const float w = any ? ex2(m - top) : 0.f;  // 0 for m = -inf
      float L = l * w;
      for (int k = 1; k < n; k *= 2) L += __shfl_xor_sync(0xffffffffu, L, k);
      s_x[tid] = any ? w * (p.v_scale / L) : 0.f;
      if (s == 0 && vh == 0 && rr - first < rows) {
        const float lse = any ? (top + log2f(L)) * kLn2 : -INFINITY;
        const int gr = row0 + rr, node = gr / G, head = u.h_kv * G + gr % G;
        const int64_t at_head = (int64_t)node * p.num_qo_heads + head;
        if (partial)
          p.partial_lse[u.partial_base + at_head * u.num_splits + u.split] = lse;
        else if (p.lse)
          p.lse[(int64_t)u.qo_begin * p.num_qo_heads + at_head] = lse;
      }
    }
    __syncthreads();
    constexpr int DQ = DVC / 4, MB = 4;
    for (int idx = tid; idx < rows * DQ; idx += kThreads) {
      const int rr = idx / DQ, d = 4 * (idx % DQ), gr = row0 + first + rr, node = gr / G;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = 0; s0 < n; s0 += MB) {
        float4 os[MB];
        float w[MB];
#pragma unroll
        for (int k = 0; k < MB; ++k) {
          if (s0 + k >= n) break;
          const int at = (s0 + k) / copies * VH + vh;
          const int row = first + rr + (s0 + k) % copies * rows_held;
          w[k] = s_x[rr * n + s0 + k];
          os[k] = peer_v4(peer(so + 4 * (row * T::OROW + d), at));
        }
#pragma unroll
        for (int k = 0; k < MB; ++k) {
          if (s0 + k >= n) break;
          o.x = fmaf(os[k].x, w[k], o.x);
          o.y = fmaf(os[k].y, w[k], o.y);
          o.z = fmaf(os[k].z, w[k], o.z);
          o.w = fmaf(os[k].w, w[k], o.w);
        }
      }
      const int64_t at_head = (int64_t)node * p.num_qo_heads + u.h_kv * G + gr - node * G;
      if (partial)
        *reinterpret_cast<float4*>(
            p.partial_o + (u.partial_base + at_head * u.num_splits + u.split) * DV + vh * DVC +
            d) = o;
      else
        store_out4(p.out + ((int64_t)u.qo_begin * p.num_qo_heads + at_head) * DV + vh * DVC + d,
                   o, p.out_f16);
    }
    if (parts > 1) {
      __syncwarp();
      cluster_arrive_wait();  // no CTA ends while another reads its state
    }
  }
  if (!partial) return;
  // ---- the last CTA of the request's units to arrive folds their states --------------------
  __syncthreads();
  if (tid == 0) {
    int* ctr = p.counters + (int64_t)u.pair * p.row_blocks + block;
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(ctr) : "memory");
    *s_last = old == u.num_splits * C - 1;
    if (*s_last) *ctr = 0;  // every other CTA has arrived
  }
  __syncthreads();
  if (!*s_last) return;
  constexpr int DQ = DV / 4, MB = 8;
  constexpr float kLog2e = 1.44269504088896340736f;
  for (int idx = tid; idx < nrows * DQ; idx += kThreads) {
    const int gr = row0 + idx / DQ, d = 4 * (idx % DQ), node = gr / G, head = u.h_kv * G + gr % G;
    const int64_t base = (int64_t)u.partial_base +
                         ((int64_t)node * p.num_qo_heads + head) * u.num_splits;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < u.num_splits; s0 += MB) {
      float lw[MB];
      float4 v[MB];
      float mb = M;
#pragma unroll
      for (int k = 0; k < MB; ++k) {
        lw[k] = -INFINITY;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 + k < u.num_splits) {
          lw[k] = __ldcg(p.partial_lse + base + s0 + k) * kLog2e;
          v[k] = __ldcg(reinterpret_cast<const float4*>(p.partial_o + (base + s0 + k) * DV + d));
        }
      }
#pragma unroll
      for (int k = 0; k < MB; ++k) mb = fmaxf(mb, lw[k]);
      if (mb == -INFINITY) continue;
      const float cf = ex2(M - mb);  // 0 for -inf
      L *= cf;
      o.x *= cf; o.y *= cf; o.z *= cf; o.w *= cf;
#pragma unroll
      for (int k = 0; k < MB; ++k) {
        const float w = ex2(lw[k] - mb);
        L += w;
        o.x = fmaf(w, v[k].x, o.x);
        o.y = fmaf(w, v[k].y, o.y);
        o.z = fmaf(w, v[k].z, o.z);
        o.w = fmaf(w, v[k].w, o.w);
      }
      M = mb;
    }
    const float inv = M != -INFINITY ? 1.f / L : 0.f;
    const int64_t row = (int64_t)(u.qo_begin + node) * p.num_qo_heads + head;
    store_out4(p.out + row * DV + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv),
               p.out_f16);
    if (d == 0 && p.lse) p.lse[row] = M != -INFINITY ? (M + log2f(L)) * kLn2 : -INFINITY;
  }
}

template <int DK, int DVC, int VH, int TT, bool ONE = false>
bool make_tree(TreeConfig* cfg) {
  using T = Tree<DK, DVC, VH, TT, ONE>;
  cfg->func = reinterpret_cast<const void*>(attend_tree_kernel<DK, DVC, VH, TT, ONE>);
  cfg->smem_bytes = T::SMEM;
  cfg->value_parts = VH;
  cfg->tile_tokens = TT;
  cfg->threads = T::THREADS;
  return true;
}

}  // namespace

bool attend_config_tree(int dk, int dv, TreeConfig* cfg) {
  // tiles of 64 tokens from 256 dims on: two of K's operand tiles, and tensor memory for
  // two S tiles beside Q and O
  if (dk == 64 && dv == 64) return make_tree<64, 64, 1, 128>(cfg);
  if (dk == 128 && dv == 128) return make_tree<128, 128, 1, 128>(cfg);
  if (dk == 256 && dv == 128) return make_tree<256, 128, 1, 64>(cfg);
  if (dk == 256 && dv == 256) return make_tree<256, 128, 2, 64>(cfg);
  if (dk == 512 && dv == 256) return make_tree<512, 128, 2, 64, true>(cfg);
  return false;
}

static void tree_launch(const TreeConfig& cfg, int grid, int rows, int ctas,
                        cudaLaunchAttribute* attr, cudaLaunchConfig_t* lc) {
  *lc = cudaLaunchConfig_t{};
  lc->gridDim = dim3(grid, rows * ctas);
  lc->blockDim = dim3(cfg.threads);
  lc->dynamicSmemBytes = cfg.smem_bytes;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = 1;
  attr->val.clusterDim.y = ctas;
  attr->val.clusterDim.z = 1;
  lc->attrs = attr;
  lc->numAttrs = 1;
}

// A property of the current device and the kernel, asked for once.
int tree_max_clusters(const TreeConfig& cfg, int ctas) {
  struct Known {
    const void* func;
    int dev, ctas, clusters;
  };
  static std::mutex mu;
  static Known known[64];
  static int count = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < count; ++i)
    if (known[i].func == cfg.func && known[i].dev == dev && known[i].ctas == ctas)
      return known[i].clusters;
  cudaLaunchAttribute attr{};
  cudaLaunchConfig_t lc;
  tree_launch(cfg, 1, 1, ctas, &attr, &lc);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, cfg.func, &lc) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (count < 64) known[count++] = {cfg.func, dev, ctas, n};  // (else asked again)
  return n;
}

cudaError_t launch_attend_tree(const TreeConfig& cfg, AttendParams p, int grid, int row_blocks,
                               int ctas, cudaStream_t stream) {
  p.tree_ctas = ctas;
  cudaLaunchAttribute attr{};
  cudaLaunchConfig_t lc;
  tree_launch(cfg, grid, row_blocks, ctas, &attr, &lc);
  lc.stream = stream;
  void* args[] = {&p};
  return cudaLaunchKernelExC(&lc, cfg.func, args);
}

}  // namespace nvfp4kv
