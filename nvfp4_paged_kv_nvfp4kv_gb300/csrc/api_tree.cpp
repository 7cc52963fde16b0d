// api_tree.cpp -- host side of the entry points of a step that verifies drafted
// tokens (argument validation and dispatch): tree masks, accepted tokens moved
// together, pages with several owners.  The attention of such a step is in api.cpp.
#include "nvfp4kv.h"

#include <cuda_runtime_api.h>

#include "checks.h"
#include "internal.h"

using namespace nvfp4kv;

namespace {

CacheRows rows_of(const nvfp4kv_paged_cache* c) {
  CacheRows r{};
  r.data[0] = c->k_data; r.data[1] = c->v_data;
  r.scale[0] = c->k_sf; r.scale[1] = c->v_sf;
  r.sp[0] = c->k_stride_page; r.ss[0] = c->k_stride_slot; r.sh[0] = c->k_stride_head;
  r.sp[1] = c->v_stride_page; r.ss[1] = c->v_stride_slot; r.sh[1] = c->v_stride_head;
  r.scp[0] = c->k_sf_stride_page; r.scs[0] = c->k_sf_stride_slot; r.sch[0] = c->k_sf_stride_head;
  r.scp[1] = c->v_sf_stride_page; r.scs[1] = c->v_sf_stride_slot; r.sch[1] = c->v_sf_stride_head;
  r.row_bytes[0] = c->head_dim_qk / 2; r.row_bytes[1] = c->head_dim_vo / 2;
  r.scale_bytes[0] = c->head_dim_qk / kBlock; r.scale_bytes[1] = c->head_dim_vo / kBlock;
  r.num_pages = c->num_pages;
  r.page_size = c->page_size;
  r.num_kv_heads = c->num_kv_heads;
  return r;
}

CacheRows rows_of(const nvfp4kv_e4m3_cache* c) {
  CacheRows r{};
  r.data[0] = c->k_data; r.data[1] = c->v_data;
  r.scale[0] = reinterpret_cast<uint8_t*>(c->k_scale);
  r.scale[1] = reinterpret_cast<uint8_t*>(c->v_scale);
  r.sp[0] = c->k_stride_page; r.ss[0] = c->k_stride_slot; r.sh[0] = c->k_stride_head;
  r.sp[1] = c->v_stride_page; r.ss[1] = c->v_stride_slot; r.sh[1] = c->v_stride_head;
  r.scp[0] = c->k_scale_stride_page; r.sch[0] = c->k_scale_stride_head;
  r.scp[1] = c->v_scale_stride_page; r.sch[1] = c->v_scale_stride_head;
  r.row_bytes[0] = c->head_dim_qk; r.row_bytes[1] = c->head_dim_vo;
  r.scale_bytes[0] = r.scale_bytes[1] = 4;
  r.num_pages = c->num_pages;
  r.page_size = c->page_size;
  r.num_kv_heads = c->num_kv_heads;
  r.page_scales = 1;
  return r;
}

int compact(const CacheRows& rows, const int32_t* path, int64_t path_stride, int32_t path_width,
            const int32_t* num_kept, const int32_t* qo_indptr, const int32_t* kv_indptr,
            const int32_t* kv_indices, const int32_t* last_page_len, int32_t batch,
            uint32_t* device_flags, cudaStream_t stream) {
  if (batch < 0 || path_width < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "batch %d / path_width %d negative", batch,
                path_width);
  if (path_stride < 0 || (batch > 1 && path_stride < path_width))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "path rows overlap");
  if ((int64_t)batch * 2 * rows.num_kv_heads > INT32_MAX)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "batch %d x %d kv heads: too many", batch,
                rows.num_kv_heads);
  if (batch == 0 || path_width == 0) return ok();
  if (!path || !num_kept || !qo_indptr || !kv_indptr || !kv_indices || !last_page_len)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null input pointer");
  CompactParams p{};
  static_cast<CacheRows&>(p) = rows;
  p.path = path;
  p.path_stride = path_stride;
  p.path_width = path_width;
  p.batch = batch;
  p.num_kept = num_kept;
  p.qo_indptr = qo_indptr;
  p.kv_indptr = kv_indptr;
  p.kv_indices = kv_indices;
  p.last_page_len = last_page_len;
  p.flags = device_flags;
  return launched(launch_compact(p, stream), "compact_tokens launch");
}

int copy_pages(const CacheRows& rows, const int32_t* src, const int32_t* dst, int32_t num,
               uint32_t* device_flags, cudaStream_t stream) {
  if (num < 0) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num %d negative", num);
  if ((int64_t)num * rows.num_kv_heads > INT32_MAX)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "%d pages x %d kv heads: too many", num,
                rows.num_kv_heads);
  if (num == 0) return ok();
  if (!src || !dst) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null list");
  PageCopyParams p{};
  static_cast<CacheRows&>(p) = rows;
  p.src = src;
  p.dst = dst;
  p.num = num;
  p.flags = device_flags;
  return launched(launch_page_copies(p, stream), "copy_pages launch");
}

// What fork and release have in common: the block table, the pool and the free list.
int check_pool(int32_t num_rows, int32_t most_rows, int32_t page_size, const int32_t* block_table,
               int64_t table_stride, int32_t table_width, const int32_t* page_shares,
               int32_t num_pages, const int32_t* free_pages, int32_t num_free,
               const int32_t* free_head, const int32_t* free_head_out, const int32_t* kv_len) {
  if (num_rows < 0 || table_width < 0 || num_pages < 0 || num_free < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "num_rows, max_pages_per_request, num_pages or num_free < 0");
  if (num_rows > most_rows)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "%d rows (at most %d)", num_rows, most_rows);
  if (page_size < 1 || page_size > 65536)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "page_size %d (1 to 65536)", page_size);
  if (!free_head || !free_head_out)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "free_head or free_head_out is null");
  if (num_rows > 0 && !kv_len) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "kv_len is null");
  if ((num_rows > 0 && table_width > 0 && !block_table) || (num_pages > 0 && !page_shares) ||
      (num_free > 0 && !free_pages))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null table, page_shares or free list");
  if (num_rows > 1 && table_stride < table_width)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "block table rows overlap");
  return NVFP4KV_OK;
}

}  // namespace

extern "C" {

int nvfp4kv_tree_masks(const int32_t* parents, const int32_t* qo_indptr, const int32_t* kv_len,
                       int32_t batch, int32_t num_rows, int32_t mask_words, uint32_t* tree_mask,
                       int32_t* positions, uint32_t* device_flags, cudaStream_t stream) {
  if (batch < 0 || num_rows < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "batch %d / num_rows %d negative", batch, num_rows);
  if (mask_words < 1 || mask_words > kMaxTreeNodes / 32)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "mask_words %d (1 to %d)", mask_words,
                kMaxTreeNodes / 32);
  if (batch == 0 || num_rows == 0) return ok();
  if (!parents || !qo_indptr || !kv_len || !tree_mask || !positions)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null pointer");
  TreeMaskParams p{};
  p.parents = parents;
  p.qo_indptr = qo_indptr;
  p.kv_len = kv_len;
  p.batch = batch;
  p.num_rows = num_rows;
  p.mask_words = mask_words;
  p.tree_mask = tree_mask;
  p.positions = positions;
  p.flags = device_flags;
  return launched(launch_tree_masks(p, stream), "tree_masks launch");
}

int nvfp4kv_compact_tokens(const nvfp4kv_paged_cache* cache, const int32_t* path,
                           int64_t path_stride, int32_t path_width, const int32_t* num_kept,
                           const int32_t* qo_indptr, const int32_t* kv_indptr,
                           const int32_t* kv_indices, const int32_t* last_page_len, int32_t batch,
                           uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_paged_cache(cache, false)) return st;
  return compact(rows_of(cache), path, path_stride, path_width, num_kept, qo_indptr, kv_indptr,
                 kv_indices, last_page_len, batch, device_flags, stream);
}

int nvfp4kv_e4m3_compact_tokens(const nvfp4kv_e4m3_cache* cache, const int32_t* path,
                                int64_t path_stride, int32_t path_width, const int32_t* num_kept,
                                const int32_t* qo_indptr, const int32_t* kv_indptr,
                                const int32_t* kv_indices, const int32_t* last_page_len,
                                int32_t batch, uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_e4m3_cache(cache)) return st;
  return compact(rows_of(cache), path, path_stride, path_width, num_kept, qo_indptr, kv_indptr,
                 kv_indices, last_page_len, batch, device_flags, stream);
}

int nvfp4kv_fork_pages(const int32_t* parents, const int32_t* children, int32_t num_forks,
                       int32_t* kv_len, int32_t num_rows, int32_t page_size,
                       int32_t* block_table, int64_t block_table_stride,
                       int32_t max_pages_per_request, int32_t* page_shares, int32_t num_pages,
                       const int32_t* free_pages, int32_t num_free, const int32_t* free_head,
                       int32_t* free_head_out, int32_t* copy_src, int32_t* copy_dst,
                       uint32_t* device_flags, cudaStream_t stream) {
  if (num_forks < 0) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num_forks %d negative", num_forks);
  if (num_forks > kMaxForks)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "%d forks (at most %d)", num_forks, kMaxForks);
  if (int st = check_pool(num_rows, kMaxForkRows, page_size, block_table, block_table_stride,
                          max_pages_per_request, page_shares, num_pages, free_pages, num_free,
                          free_head, free_head_out, kv_len))
    return st;
  if (free_head == free_head_out)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "the new free head must not overwrite the one that is read");
  if (num_forks > 0 && (!parents || !children || !copy_src || !copy_dst))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null list of forks or copies");
  ForkParams p{};
  p.parents = parents;
  p.children = children;
  p.kv_len = kv_len;
  p.block_table = block_table;
  p.table_stride = block_table_stride;
  p.page_shares = page_shares;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.free_head_out = free_head_out;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.num_forks = num_forks;
  p.num_rows = num_rows;
  p.page_size = page_size;
  p.table_width = max_pages_per_request;
  p.num_pages = num_pages;
  p.num_free = num_free;
  p.flags = device_flags;
  return launched(launch_fork(p, stream), "fork_pages launch");
}

int nvfp4kv_copy_pages(const nvfp4kv_paged_cache* cache, const int32_t* src, const int32_t* dst,
                       int32_t num, uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_paged_cache(cache, false)) return st;
  return copy_pages(rows_of(cache), src, dst, num, device_flags, stream);
}

int nvfp4kv_e4m3_copy_pages(const nvfp4kv_e4m3_cache* cache, const int32_t* src,
                            const int32_t* dst, int32_t num, uint32_t* device_flags,
                            cudaStream_t stream) {
  if (int st = check_e4m3_cache(cache)) return st;
  return copy_pages(rows_of(cache), src, dst, num, device_flags, stream);
}

int nvfp4kv_release_pages(const int32_t* keep_len, int32_t* kv_len, int32_t num_rows,
                          int32_t page_size, const int32_t* block_table,
                          int64_t block_table_stride, int32_t max_pages_per_request,
                          int32_t* page_shares, int32_t num_pages, int32_t* free_pages,
                          int32_t num_free, const int32_t* free_head, int32_t* free_head_out,
                          uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_pool(num_rows, kMaxPageTableBatch, page_size, block_table,
                          block_table_stride, max_pages_per_request, page_shares, num_pages,
                          free_pages, num_free, free_head, free_head_out, kv_len))
    return st;
  if (num_rows > 0 && !keep_len)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "keep_len is null");
  ReleaseParams p{};
  p.keep_len = keep_len;
  p.kv_len = kv_len;
  p.block_table = block_table;
  p.table_stride = block_table_stride;
  p.page_shares = page_shares;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.free_head_out = free_head_out;
  p.num_rows = num_rows;
  p.page_size = page_size;
  p.table_width = max_pages_per_request;
  p.num_pages = num_pages;
  p.num_free = num_free;
  p.flags = device_flags;
  return launched(launch_release(p, stream), "release_pages launch");
}

}  // extern "C"
