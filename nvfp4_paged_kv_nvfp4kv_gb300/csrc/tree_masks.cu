// tree_masks.cu -- what each node of a drafted tree sees, from the nodes' parents,
// sm_103a.
//
// Request b drafts n_b nodes, its rows qo_indptr[b] .. qo_indptr[b + 1), as a tree:
// parent(i) < i is the node that node i continues, -1 for a root.  With A(i) the set
// {i, parent(i), parent(parent(i)), ...}:
//   bit j of row i's mask words = (j in A(i)),
//   position of row i = L_b - n_b + |A(i)| - 1
// (a node stands as far behind the L_b - n_b tokens before the tree as it is deep).
//
// Latency bounds it: a launch, then the request's three lengths, its parents and a
// walk up the tree, whose length is the deepest node's depth.  One CTA takes a
// request and keeps the parents in shared memory; a thread walks up from its node.
// As parents come before their children, the walk meets the words of the mask in
// falling order: each is complete when the walk leaves it, so it stays in a
// register until it is stored and the words without a bit are filled in between.
// Measured (replayed): 16 trees of 5-16 nodes 2.4 us, 1000 of 31-130 nodes 4.9 us (2.3 MB, 0.5
// TB/s: the walks and, of the larger call, seven waves of CTAs of a few hundred cycles each).
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace nvfp4kv {
namespace {

__global__ void tree_masks_kernel(const TreeMaskParams p) {
  __shared__ int32_t s_up[kMaxTreeNodes];
  const int b = blockIdx.x;
  const int64_t r0 = p.qo_indptr[b], n64 = p.qo_indptr[b + 1] - r0;
  const int len = p.kv_len[b];
  if (n64 == 0) return;
  if (r0 < 0 || n64 < 0 || r0 + n64 > p.num_rows || n64 > kMaxTreeNodes ||
      n64 > 32 * p.mask_words || len < n64) {
    if (threadIdx.x == 0 && p.flags) atomicOr(p.flags, 0x40u);
    return;
  }
  const int n = static_cast<int>(n64);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int up = p.parents[r0 + i];
    if (up < -1 || up >= i) {  // no tree: the node stands as a root
      if (p.flags) atomicOr(p.flags, 0x100u);
      up = -1;
    }
    s_up[i] = up;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    uint32_t* row = p.tree_mask + (r0 + i) * p.mask_words;
    int word = p.mask_words - 1, depth = 0;
    uint32_t bits = 0;
    for (int j = i; j >= 0; j = s_up[j]) {
      for (; word > j >> 5; --word) {
        row[word] = bits;
        bits = 0;
      }
      bits |= 1u << (j & 31);
      ++depth;
    }
    for (; word >= 0; --word) {
      row[word] = bits;
      bits = 0;
    }
    p.positions[r0 + i] = len - n + depth - 1;
  }
}

}  // namespace

cudaError_t launch_tree_masks(const TreeMaskParams& p, cudaStream_t stream) {
  if (p.batch == 0 || p.num_rows == 0) return cudaSuccess;
  // a thread a node where the words allow so many, 256 at most (larger trees are rare
  // and loop)
  const int threads = 32 * p.mask_words < 256 ? 32 * p.mask_words : 256;
  tree_masks_kernel<<<p.batch, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
