// api.cpp -- host side of the C ABI declared in include/nvfp4kv.h:
// argument validation, the split-KV planner and kernel dispatch.
#include "nvfp4kv.h"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <functional>
#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include <cuda_runtime_api.h>

#include "internal.h"

namespace nvfp4kv {
bool attend_config_tc(int dk, int dv, int rows, bool tree, AttendConfig* cfg);
bool attend_config_simt(int dk, int dv, int rows, AttendConfig* cfg);
bool attend_config_tcgen05(int dk, int dv, int rows, AttendConfig* cfg);
bool attend_config_dec(int dk, int dv, int rows, int quads, AttendConfig* cfg);
bool attend_config_tc_fp4qp(int dk, int dv, int rows, int pass, AttendConfig* cfg);
cudaError_t prepare_kernel(const AttendConfig& cfg);
}  // namespace nvfp4kv

using namespace nvfp4kv;

namespace {
int fail(int status, const char* fmt, ...);
}

namespace nvfp4kv {
int set_error_detail(int status, const char* message) { return fail(status, "%s", message); }
}  // namespace nvfp4kv

namespace {

thread_local std::string g_detail;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_detail = buf;
  return status;
}

int ok() {
  g_detail.clear();
  return NVFP4KV_OK;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(NVFP4KV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uint64_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

uint64_t align_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

bool attention_dims_supported(int dk, int dv) {
  return (dk == 64 && dv == 64) || (dk == 128 && dv == 128) ||
         (dk == 256 && dv == 256) || (dk == 256 && dv == 128) ||
         (dk == 512 && dv == 256);
}

// Common cache checks.  `for_attention` adds the head-dim whitelist and the
// cp.async alignment rules.
int check_cache(const nvfp4kv_paged_cache* c, bool for_attention) {
  if (!c) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache is null");
  if (!c->k_data || !c->v_data || !c->k_sf || !c->v_sf)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache buffer pointer is null");
  if (c->page_size != kPageSize && c->page_size != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "page_size %d (16 and 1 are supported)", c->page_size);
  if (c->num_pages <= 0 || c->num_kv_heads <= 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num_pages %d / num_kv_heads %d must be > 0",
                c->num_pages, c->num_kv_heads);
  if (c->head_dim_qk <= 0 || c->head_dim_vo <= 0 || c->head_dim_qk % 32 ||
      c->head_dim_vo % 32 || c->head_dim_qk > 512 || c->head_dim_vo > 512)
    return fail(NVFP4KV_ERR_UNSUPPORTED,
                "head dims (%d, %d): each must be a multiple of 32 and at most 512",
                c->head_dim_qk, c->head_dim_vo);
  if (for_attention && !attention_dims_supported(c->head_dim_qk, c->head_dim_vo))
    return fail(NVFP4KV_ERR_UNSUPPORTED,
                "attention head dims (%d, %d) not built; supported: (64,64), "
                "(128,128), (256,256), (256,128), (512,256)",
                c->head_dim_qk, c->head_dim_vo);
  const float gmin = std::ldexp(1.0f, -64), gmax = std::ldexp(1.0f, 64);
  if (!(c->k_global_scale >= gmin && c->k_global_scale <= gmax) ||
      !(c->v_global_scale >= gmin && c->v_global_scale <= gmax))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "global scales must lie in [2^-64, 2^64]");
  const int64_t kd[3] = {c->k_stride_page, c->k_stride_slot, c->k_stride_head};
  const int64_t vd[3] = {c->v_stride_page, c->v_stride_slot, c->v_stride_head};
  const int64_t ks[3] = {c->k_sf_stride_page, c->k_sf_stride_slot, c->k_sf_stride_head};
  const int64_t vs[3] = {c->v_sf_stride_page, c->v_sf_stride_slot, c->v_sf_stride_head};
  const int64_t ksa = std::min(16, c->head_dim_qk / 16), vsa = std::min(16, c->head_dim_vo / 16);
  for (int i = 0; i < 3; ++i) {
    if (kd[i] < 0 || vd[i] < 0 || ks[i] < 0 || vs[i] < 0)
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "negative cache stride");
    if (kd[i] % 16 || vd[i] % 16)
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                  "K/V data strides must be multiples of 16 bytes");
    if (ks[i] % ksa || vs[i] % vsa)
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                  "scale strides must be multiples of min(16, D/16) bytes");
  }
  if (!aligned(c->k_data, 16) || !aligned(c->v_data, 16) || !aligned(c->k_sf, ksa) ||
      !aligned(c->v_sf, vsa))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache buffer misaligned");
  // the innermost row must not overlap the next slot/head (rows are contiguous)
  if (std::min(c->k_stride_slot, c->k_stride_head) < c->head_dim_qk / 2 ||
      std::min(c->v_stride_slot, c->v_stride_head) < c->head_dim_vo / 2 ||
      std::min(c->k_sf_stride_slot, c->k_sf_stride_head) < c->head_dim_qk / 16 ||
      std::min(c->v_sf_stride_slot, c->v_sf_stride_head) < c->head_dim_vo / 16)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache strides overlap a row");
  return NVFP4KV_OK;
}

CacheView view_of(const nvfp4kv_paged_cache* c) {
  CacheView v;
  v.k_data = c->k_data;
  v.v_data = c->v_data;
  v.k_sf = c->k_sf;
  v.v_sf = c->v_sf;
  v.k_sp = c->k_stride_page; v.k_ss = c->k_stride_slot; v.k_sh = c->k_stride_head;
  v.v_sp = c->v_stride_page; v.v_ss = c->v_stride_slot; v.v_sh = c->v_stride_head;
  v.ksf_sp = c->k_sf_stride_page; v.ksf_ss = c->k_sf_stride_slot; v.ksf_sh = c->k_sf_stride_head;
  v.vsf_sp = c->v_sf_stride_page; v.vsf_ss = c->v_sf_stride_slot; v.vsf_sh = c->v_sf_stride_head;
  v.num_pages = c->num_pages;
  return v;
}

// `tree`: the kernel's form that looks the step's tokens up in the rows' masks
bool lookup_kernel(int kind, int dk, int dv, int page_size, int rows, AttendConfig* cfg,
                   bool tree = false) {
  if (kind == kKernelTensorCore) return attend_config_tc(dk, dv, rows, tree, cfg);
  if (tree) return false;
  if (kind == kKernelTcgen05) return attend_config_tcgen05(dk, dv, rows, cfg);
  if (kind == kKernelCudaCore) return attend_config_simt(dk, dv, rows, cfg);
  if (kind == kKernelFp4QP) return attend_config_tc_fp4qp(dk, dv, rows, 2, cfg);
  if (kind == kKernelE4m3) return attend_config_e4m3(dk, dv, page_size, rows, cfg);
  return false;
}

// What a unit of the E4M3 extend kernel costs beside its tiles of 128 tokens, in
// tiles: 25 plans (batches of 13-100 requests, 1 to 6 pieces the longest) fit
// time = 1.16 us x the busiest SM's tiles and units to 3 % with 12.
constexpr int64_t kUnitTiles = 12;
constexpr int kMostModelled = 4096;  // CTAs of a plan whose loads the planner models
constexpr int kMinChunkPages = 8;

// The bulk-copy decode kernel reads each (page, head) region of the four
// buffers with one copy: the 16 slots' rows must be contiguous, every region
// must start 16-byte aligned, and a page offset must fit 32 bits.
bool bulk_decode_layout(const nvfp4kv_paged_cache* c) {
  const int64_t kr = c->head_dim_qk / 2, vr = c->head_dim_vo / 2;
  const int64_t ksr = c->head_dim_qk / 16, vsr = c->head_dim_vo / 16;
  const int64_t lim = (int64_t)1 << 32;
  return c->k_stride_slot == kr && c->v_stride_slot == vr && c->k_sf_stride_slot == ksr &&
         c->v_sf_stride_slot == vsr && aligned(c->k_sf, 16) && aligned(c->v_sf, 16) &&
         c->k_sf_stride_page % 16 == 0 && c->k_sf_stride_head % 16 == 0 &&
         c->v_sf_stride_page % 16 == 0 && c->v_sf_stride_head % 16 == 0 &&
         c->k_stride_page < lim && c->v_stride_page < lim && c->k_sf_stride_page < lim &&
         c->v_sf_stride_page < lim;
}

}  // namespace

extern "C" {

const char* nvfp4kv_status_string(int status) {
  switch (status) {
    case NVFP4KV_OK: return "ok";
    case NVFP4KV_ERR_INVALID_ARGUMENT: return "invalid argument";
    case NVFP4KV_ERR_UNSUPPORTED: return "unsupported";
    case NVFP4KV_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case NVFP4KV_ERR_CUDA: return "CUDA error";
    case NVFP4KV_ERR_DEVICE_CHECK: return "device check failed";
    case NVFP4KV_ERR_PLAN_MISMATCH: return "arguments do not match the plan";
    default: return "unknown status";
  }
}

const char* nvfp4kv_last_error_detail(void) { return g_detail.c_str(); }

int nvfp4kv_dequantize_paged(const nvfp4kv_paged_cache* cache, const int32_t* page_ids,
                             int32_t num_ids, float* k_out, float* v_out,
                             uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_cache(cache, false)) return st;
  if (num_ids < 0) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num_ids %d negative", num_ids);
  if (num_ids == 0 || (!k_out && !v_out)) return ok();
  if (!page_ids) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "page_ids is null");
  if ((k_out && !aligned(k_out, 16)) || (v_out && !aligned(v_out, 16)))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "outputs must be 16-byte aligned");
  DequantParams p{};
  p.k_data = cache->k_data; p.v_data = cache->v_data;
  p.k_sf = cache->k_sf; p.v_sf = cache->v_sf;
  p.k_sp = cache->k_stride_page; p.k_ss = cache->k_stride_slot; p.k_sh = cache->k_stride_head;
  p.v_sp = cache->v_stride_page; p.v_ss = cache->v_stride_slot; p.v_sh = cache->v_stride_head;
  p.ksf_sp = cache->k_sf_stride_page; p.ksf_ss = cache->k_sf_stride_slot;
  p.ksf_sh = cache->k_sf_stride_head;
  p.vsf_sp = cache->v_sf_stride_page; p.vsf_ss = cache->v_sf_stride_slot;
  p.vsf_sh = cache->v_sf_stride_head;
  p.num_pages = cache->num_pages;
  p.num_kv_heads = cache->num_kv_heads;
  p.head_dim_qk = cache->head_dim_qk;
  p.head_dim_vo = cache->head_dim_vo;
  p.page_size = cache->page_size;
  p.k_global_scale = cache->k_global_scale;
  p.v_global_scale = cache->v_global_scale;
  p.page_ids = page_ids;
  p.num_ids = num_ids;
  p.k_out = k_out;
  p.v_out = v_out;
  p.flags = device_flags;
  cudaError_t e = launch_dequantize(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "dequantize launch");
  return ok();
}

int nvfp4kv_quantize_append(const nvfp4kv_paged_cache* cache, const void* k_bf16,
                            int64_t k_stride_tok, int64_t k_stride_head,
                            const void* v_bf16, int64_t v_stride_tok,
                            int64_t v_stride_head, int32_t nnz,
                            const int32_t* batch_idx, const int32_t* positions,
                            const int32_t* kv_indices, const int32_t* kv_indptr,
                            const int32_t* last_page_len, int32_t batch,
                            uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_cache(cache, false)) return st;
  if (nnz < 0 || batch < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "nnz %d / batch %d negative", nnz, batch);
  if (nnz == 0) return ok();
  if (!k_bf16 || !v_bf16 || !batch_idx || !positions || !kv_indices || !kv_indptr ||
      !last_page_len)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null input pointer");
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || k_stride_tok % 8 ||
      k_stride_head % 8 || v_stride_tok % 8 || v_stride_head % 8 || k_stride_tok < 0 ||
      k_stride_head < 0 || v_stride_tok < 0 || v_stride_head < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "bf16 inputs must be 16-byte aligned with strides multiple of 8 elements");
  AppendParams p{};
  p.k_data = cache->k_data; p.v_data = cache->v_data;
  p.k_sf = cache->k_sf; p.v_sf = cache->v_sf;
  p.k_sp = cache->k_stride_page; p.k_ss = cache->k_stride_slot; p.k_sh = cache->k_stride_head;
  p.v_sp = cache->v_stride_page; p.v_ss = cache->v_stride_slot; p.v_sh = cache->v_stride_head;
  p.ksf_sp = cache->k_sf_stride_page; p.ksf_ss = cache->k_sf_stride_slot;
  p.ksf_sh = cache->k_sf_stride_head;
  p.vsf_sp = cache->v_sf_stride_page; p.vsf_ss = cache->v_sf_stride_slot;
  p.vsf_sh = cache->v_sf_stride_head;
  p.num_pages = cache->num_pages;
  p.num_kv_heads = cache->num_kv_heads;
  p.head_dim_qk = cache->head_dim_qk;
  p.head_dim_vo = cache->head_dim_vo;
  p.page_size = cache->page_size;
  p.k_global_scale = cache->k_global_scale;
  p.v_global_scale = cache->v_global_scale;
  p.k = static_cast<const uint16_t*>(k_bf16);
  p.v = static_cast<const uint16_t*>(v_bf16);
  p.k_stride_tok = k_stride_tok; p.k_stride_head = k_stride_head;
  p.v_stride_tok = v_stride_tok; p.v_stride_head = v_stride_head;
  p.nnz = nnz;
  p.batch = batch;
  p.batch_idx = batch_idx;
  p.positions = positions;
  p.kv_indices = kv_indices;
  p.kv_indptr = kv_indptr;
  p.last_page_len = last_page_len;
  p.flags = device_flags;
  cudaError_t e = launch_append(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "quantize_append launch");
  return ok();
}

int nvfp4kv_decode_plan(const int32_t* qo_indptr_h, const int32_t* kv_indptr_h,
                        const int32_t* last_page_len_h, int32_t batch,
                        int32_t num_qo_heads, int32_t num_kv_heads,
                        int32_t head_dim_qk, int32_t head_dim_vo, int32_t page_size,
                        const nvfp4kv_plan_options* opts_in, int32_t device,
                        void* plan_host, uint64_t plan_host_bytes, void* workspace,
                        uint64_t workspace_bytes, cudaStream_t stream,
                        nvfp4kv_plan_info* info) {
  if (!info) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "info is null");
  std::memset(info, 0, sizeof *info);
  nvfp4kv_plan_options opts{};
  if (opts_in) opts = *opts_in;
  if (batch < 0) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "batch %d < 0", batch);
  if (batch > 0 && (!qo_indptr_h || !kv_indptr_h || !last_page_len_h))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null indptr / last_page_len");
  if (num_qo_heads <= 0 || num_kv_heads <= 0 || num_qo_heads % num_kv_heads)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "num_qo_heads %d must be a positive multiple of num_kv_heads %d",
                num_qo_heads, num_kv_heads);
  if (page_size != kPageSize && page_size != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "page_size %d (16 and 1 are supported)", page_size);
  if (opts.out_dtype != 0 && opts.out_dtype != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "out_dtype %d (0 bf16, 1 f16)", opts.out_dtype);
  if (!attention_dims_supported(head_dim_qk, head_dim_vo))
    return fail(NVFP4KV_ERR_UNSUPPORTED, "attention head dims (%d, %d) not built",
                head_dim_qk, head_dim_vo);
  if (opts.force_chunk_tokens < 0 || opts.force_chunk_tokens % kPageSize)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "force_chunk_tokens %d must be a non-negative multiple of 16",
                opts.force_chunk_tokens);
  if (opts.max_splits < 0 || opts.num_sms < 0 || opts.ctas_per_sm < 0 || opts.kernel < 0 ||
      opts.kernel > kKernelE4m3)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "bad plan option");
  const int G = num_qo_heads / num_kv_heads;

  // ---- batch description ------------------------------------------------
  if (batch > 0 && qo_indptr_h[0] != 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "qo_indptr[0] must be 0");
  // the planner counts 16-token tiles: one page at page size 16, PT pages
  // at page size 1
  const int PT = kPageSize / page_size;
  std::vector<int32_t> np(batch), nq(batch), nt(batch);
  int64_t total_pages = 0;
  int max_rows = 0, max_np = 0;
  for (int b = 0; b < batch; ++b) {
    nq[b] = qo_indptr_h[b + 1] - qo_indptr_h[b];
    np[b] = kv_indptr_h[b + 1] - kv_indptr_h[b];
    if (nq[b] < 0 || np[b] < 0)
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "indptr decreases at request %d", b);
    if (kv_indptr_h[b] < 0)
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "kv_indptr[%d] < 0", b);
    int64_t L = 0;
    if (np[b] > 0) {
      if (last_page_len_h[b] < 1 || last_page_len_h[b] > page_size)
        return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "last_page_len[%d] = %d not in [1, %d]", b,
                    last_page_len_h[b], page_size);
      L = static_cast<int64_t>(np[b] - 1) * page_size + last_page_len_h[b];
    }
    nt[b] = (np[b] + PT - 1) / PT;
    if (L < nq[b])
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                  "request %d has %d query rows but only %lld kv tokens", b, nq[b],
                  static_cast<long long>(L));
    if (L > (int64_t)1 << 30)
      return fail(NVFP4KV_ERR_UNSUPPORTED, "request %d longer than 2^30 tokens", b);
    if (nq[b] > 0) {
      total_pages += np[b];
      max_np = std::max(max_np, nt[b]);  // in tiles from here on
      max_rows = std::max(max_rows, nq[b] * G);
    }
  }
  const int32_t total_rows = batch > 0 ? qo_indptr_h[batch] : 0;

  // ---- kernel choice and occupancy --------------------------------------
  int kind = opts.kernel;
  AttendConfig cfg{};
  // auto: the tcgen05 kernel where a kv head has many query rows (extend):
  // it dequantises each page once for all of them and its products grow
  // with the rows; for a few rows (decode) the mma.sync register path is
  // cheaper (a tcgen05 product costs ~54 cycles to issue whatever its N)
  if (kind == 0)
    kind = (head_dim_qk == 128 && head_dim_vo == 128 && max_rows > 16) ? kKernelTcgen05
                                                                       : kKernelTensorCore;
  const int want_rows = kind == kKernelTcgen05 || kind == kKernelE4m3 ? std::max(max_rows, 1)
                                                                      : (max_rows <= 8 ? 8 : 16);
  if (!lookup_kernel(kind, head_dim_qk, head_dim_vo, page_size, want_rows, &cfg))
    return fail(NVFP4KV_ERR_UNSUPPORTED, "no %s kernel for head dims (%d, %d)%s",
                kind == kKernelTensorCore ? "tensor-core"
                : kind == kKernelTcgen05  ? "tcgen05"
                : kind == kKernelFp4QP    ? "FP4 query/probability"
                : kind == kKernelE4m3     ? "E4M3-cache"
                                          : "CUDA-core",
                head_dim_qk, head_dim_vo,
                kind == kKernelFp4QP && want_rows > 8 ? " and more than 8 query rows per kv head"
                                                      : "");
  const int rows_per_block = cfg.rows;
  // A tensor-core plan of one block of <= 8 rows at page size 16 runs the
  // decode kernel where the cache layout allows it; that kernel takes several
  // units per CTA, so its occupancy (in units) sizes the wave.
  AttendConfig occ = cfg;
  int units_per_cta = 1;
  {
    AttendConfig dcfg{};
    if (kind == kKernelTensorCore && rows_per_block == 8 && page_size == kPageSize &&
        attend_config_dec(head_dim_qk, head_dim_vo, 8, 4, &dcfg)) {
      occ = dcfg;
      units_per_cta = std::max(1, dcfg.units_per_cta);
    }
  }
  int num_sms = opts.num_sms, ctas_per_sm = opts.ctas_per_sm;
  if (num_sms == 0 || ctas_per_sm == 0) {
    int dev = device;
    cudaError_t e = cudaSuccess;
    if (dev < 0) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    // the device's SM count and the kernel's resident CTAs per SM do not
    // change: query them once per (device, kernel) and keep them (a plan is
    // built every serving step)
    static std::mutex mu;
    static std::map<std::pair<int, const void*>, std::pair<int, int>> known;
    std::pair<int, int> sm_occ{0, 0};
    {
      std::lock_guard<std::mutex> lock(mu);
      auto it = known.find({dev, occ.func});
      if (it != known.end()) sm_occ = it->second;
    }
    if (sm_occ.first == 0) {
      e = cudaDeviceGetAttribute(&sm_occ.first, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return cuda_fail(e, "SM count");
      int optin = 0;
      e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
      if (e != cudaSuccess) return cuda_fail(e, "shared-memory opt-in");
      if (occ.smem_bytes > optin)
        return fail(NVFP4KV_ERR_UNSUPPORTED,
                    "kernel needs %d bytes of shared memory, device allows %d per block",
                    occ.smem_bytes, optin);
      int cur = -1;
      e = cudaGetDevice(&cur);
      if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
      if (cur != dev && (e = cudaSetDevice(dev)) != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
      e = prepare_kernel(occ);
      if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&sm_occ.second, occ.func,
                                                          occ.warps * 32, occ.smem_bytes);
      if (cur != dev) cudaSetDevice(cur);
      if (e != cudaSuccess) return cuda_fail(e, "occupancy");
      if (sm_occ.second < 1) sm_occ.second = 1;
      sm_occ.second *= units_per_cta;  // unit slots per SM
      std::lock_guard<std::mutex> lock(mu);
      known[{dev, occ.func}] = sm_occ;
    }
    if (num_sms == 0) num_sms = sm_occ.first;
    if (ctas_per_sm == 0) ctas_per_sm = sm_occ.second;
    info->device = dev;
  } else {
    info->device = device;
  }

  // ---- chunk size (tiles per unit) --------------------------------------
  auto row_blocks_of = [&](int b) { return (nq[b] * G + rows_per_block - 1) / rows_per_block; };
  auto ctas_for = [&](int64_t c) {
    int64_t n = 0;
    for (int b = 0; b < batch; ++b)
      if (nq[b] > 0) n += (int64_t)num_kv_heads * ((nt[b] + c - 1) / c) * row_blocks_of(b);
    return n;
  };
  int64_t chunk = std::max(max_np, 1);
  if (!opts.disable_split) {
    if (opts.force_chunk_tokens > 0) {
      chunk = opts.force_chunk_tokens / kPageSize;
    } else if (max_np > kMinChunkPages) {
      const int64_t slots = (int64_t)num_sms * ctas_per_sm;
      int64_t work = 0;
      for (int b = 0; b < batch; ++b)
        if (nq[b] > 0) work += (int64_t)num_kv_heads * nt[b] * row_blocks_of(b);
      int64_t lo = std::max<int64_t>(kMinChunkPages, (work + slots - 1) / std::max<int64_t>(slots, 1));
      int64_t hi = max_np;
      if (lo >= hi || ctas_for(hi) > slots) {
        chunk = hi;  // already one unit per request suffices / cannot fit one wave
      } else {
        while (lo < hi) {  // smallest chunk whose grid fits one wave
          const int64_t mid = (lo + hi) / 2;
          if (ctas_for(mid) <= slots) hi = mid; else lo = mid + 1;
        }
        chunk = lo;
      }
    }
    // The extend kernel over an E4M3 cache (one CTA an SM, long units): the grid
    // may be several waves, so the chunk is the one whose units, longest first,
    // keep the busiest SM shortest: that of one wave or the longest request in up
    // to 8 pieces.  20 requests of 1000-30000 tokens 290 -> 183 us, 13 of
    // 100-60000 332 -> 246 us; even batches keep their whole requests.
    if (kind == kKernelE4m3 && rows_per_block > 16 && opts.force_chunk_tokens == 0 &&
        opts.max_splits == 0 && max_np > kMinChunkPages) {
      // a heap, the least loaded SM first (a SM past the most units that are
      // looked at stays idle: an option may name any number of them)
      const int bins = std::min<int>(num_sms, kMostModelled);
      std::vector<int64_t> sms(bins);
      std::vector<std::pair<int64_t, int64_t>> rest;  // units that are not whole chunks
      int64_t least = INT64_MAX, best = chunk, mean = 0;
      for (int j : {1, 2, 3, 4, 5, 6, 8, 0}) {  // pieces; 0: one wave's chunk
        int64_t c = j == 0 ? chunk : (max_np + j - 1) / j;
        c = std::min<int64_t>(std::max<int64_t>((c + 7) / 8 * 8, kMinChunkPages), max_np);
        if (ctas_for(c) > kMostModelled) continue;  // (so many even out by themselves)
        auto cost = [](int64_t pages) { return (pages + 7) / 8 + kUnitTiles; };
        int64_t full = 0, work = 0, most = 0;
        rest.clear();
        for (int b = 0; b < batch; ++b) {
          if (nq[b] == 0) continue;
          const int64_t alike = (int64_t)num_kv_heads * row_blocks_of(b);
          full += alike * (nt[b] / c);
          if (nt[b] % c) rest.push_back({cost(nt[b] % c), alike});
        }
        std::sort(rest.begin(), rest.end(), std::greater<>());
        sms.assign(bins, 0);
        auto add = [&](int64_t x, int64_t times) {
          work += x * times;
          for (; times > 0; --times) {
            const int64_t v = sms[0] + x;
            int at = 0;
            for (int k; (k = 2 * at + 1) < bins; at = k) {
              if (k + 1 < bins && sms[k + 1] < sms[k]) ++k;
              if (sms[k] >= v) break;
              sms[at] = sms[k];
            }
            sms[at] = v;
            most = std::max(most, v);
          }
        };
        add(cost(c), full);
        for (const auto& [x, times] : rest) add(x, times);
        if (most < least) {
          least = most;
          best = c;
        }
        // whole requests have the least work: within 3 % of its mean is enough
        if (j == 1) mean = work / num_sms;
        if (least * 32 <= mean * 33) break;
      }
      chunk = best;
    }
    if (opts.max_splits > 0)
      chunk = std::max<int64_t>(chunk, (max_np + opts.max_splits - 1) / opts.max_splits);
    // the tcgen05 kernels stream tiles of 8 pages: whole tiles per unit.  (The E4M3
    // kernel of up to 16 rows streams tiles of one: rounded, its chunks leave part of
    // the wave empty, 16 rows x 4 requests of 32771 tokens 53.5 against 52.7 us, 9 of
    // 1111 tokens 11.9 against 11.1.)
    if ((kind == kKernelTcgen05 || (kind == kKernelE4m3 && rows_per_block > 16)) &&
        opts.force_chunk_tokens == 0 && chunk < max_np)
      chunk = std::min<int64_t>((chunk + 7) / 8 * 8, max_np);
  }
  chunk = std::max<int64_t>(chunk, 1);

  // ---- units, partial bases, merge indptr -------------------------------
  std::vector<WorkUnit> units;
  int32_t max_units = 0;
  bool split = false;
  int64_t n_units = 0;
  for (int b = 0; b < batch; ++b)
    if (nq[b] > 0) {
      if (nt[b] > chunk) split = true;
      n_units += (int64_t)num_kv_heads * ((nt[b] + chunk - 1) / chunk);
    }
  units.reserve(static_cast<size_t>(n_units));
  int64_t partial = 0;
  std::vector<int64_t> pbase(batch, 0);
  std::vector<int32_t> nsplit(batch, 0);
  for (int b = 0; b < batch; ++b) {
    if (nq[b] == 0) continue;
    const int S = static_cast<int>((nt[b] + chunk - 1) / chunk);
    nsplit[b] = S;
    max_units = std::max(max_units, S);
    pbase[b] = partial;
    if (split) partial += (int64_t)nq[b] * num_qo_heads * S;
    const int64_t L = static_cast<int64_t>(np[b] - 1) * page_size + last_page_len_h[b];
    const int64_t cp = chunk * PT;  // pages per unit
    for (int h = 0; h < num_kv_heads; ++h)
      for (int s = 0; s < S; ++s) {
        WorkUnit u{};
        u.b = b;
        u.h_kv = h;
        u.page_begin = kv_indptr_h[b] + static_cast<int32_t>(s * cp);
        u.num_pages = static_cast<int32_t>(std::min<int64_t>(cp, np[b] - s * cp));
        u.tok_begin = static_cast<int32_t>(s * chunk * kPageSize);
        u.kv_len = static_cast<int32_t>(L);
        u.qo_begin = qo_indptr_h[b];
        u.qo_len = nq[b];
        u.split = s;
        u.num_splits = S;
        u.partial_base = static_cast<int32_t>(pbase[b]);
        u.pair = b * num_kv_heads + h;
        units.push_back(u);
      }
  }
  // Longest units first when the grid takes more than one wave: the block
  // scheduler then starts the long units early (longest-processing-time
  // order); partial indices do not depend on the unit order.  A grid of one
  // wave starts every unit at once, and its order is left as built.
  int row_blocks = 0;
  for (int b = 0; b < batch; ++b)
    if (nq[b] > 0) row_blocks = std::max(row_blocks, row_blocks_of(b));
  if ((int64_t)units.size() * row_blocks > (int64_t)num_sms * ctas_per_sm)
    std::stable_sort(units.begin(), units.end(), [](const WorkUnit& a, const WorkUnit& b) {
      return a.num_pages > b.num_pages;
    });
  if (partial > INT32_MAX)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "too many partial states (%lld)", (long long)partial);
  const int64_t entries = split ? (int64_t)total_rows * num_qo_heads : 0;

  // ---- layout ------------------------------------------------------------
  const uint64_t off_flags = 0;
  const uint64_t off_counters = 256;
  const uint64_t n_counters = split ? (uint64_t)batch * num_kv_heads * row_blocks : 0;
  const uint64_t off_units = align_up(off_counters + n_counters * 4, 256);
  const uint64_t off_merge = align_up(off_units + units.size() * sizeof(WorkUnit), 256);
  const uint64_t off_plse = align_up(off_merge + (split ? (entries + 1) * 4 : 0), 256);
  const uint64_t off_po = align_up(off_plse + partial * 4, 256);
  const uint64_t off_rm = align_up(off_po + (uint64_t)partial * head_dim_vo * 4, 256);
  const uint64_t n_row_max = kind == kKernelFp4QP
                                 ? (uint64_t)total_rows * num_qo_heads * std::max(max_units, 1)
                                 : 0;
  const uint64_t ws_bytes = align_up(off_rm + n_row_max * 4, 256);
  const uint64_t host_bytes = off_plse - off_units;

  info->magic = kPlanMagic;
  info->batch = batch;
  info->num_qo_heads = num_qo_heads;
  info->num_kv_heads = num_kv_heads;
  info->head_dim_qk = head_dim_qk;
  info->head_dim_vo = head_dim_vo;
  info->page_size = page_size;
  info->causal = opts.causal ? 1 : 0;
  info->kernel = kind;
  info->num_units = static_cast<int32_t>(units.size());
  info->row_blocks = row_blocks;
  info->rows_per_block = rows_per_block;
  info->warps = cfg.warps;
  info->split = split ? 1 : 0;
  info->chunk_pages = static_cast<int32_t>(std::min<int64_t>(chunk, INT32_MAX));
  info->max_units_per_request = max_units;
  info->total_qo_rows = total_rows;
  info->num_sms = num_sms;
  info->ctas_per_sm = ctas_per_sm;
  info->out_dtype = opts.out_dtype;
  info->smem_bytes = cfg.smem_bytes;
  info->num_partials = partial;
  info->total_kv_pages = total_pages;
  info->workspace_bytes = ws_bytes;
  info->plan_host_bytes = host_bytes;
  info->off_flags = off_flags;
  info->off_units = off_units;
  info->off_merge_indptr = off_merge;
  info->off_partial_lse = off_plse;
  info->off_partial_o = off_po;
  info->off_counters = off_counters;
  info->off_row_max = n_row_max ? off_rm : 0;
  info->device_last_page_len = opts.device_last_page_len;

  if (host_bytes > 0 && (!plan_host || plan_host_bytes < host_bytes))
    return fail(NVFP4KV_ERR_WORKSPACE_TOO_SMALL, "plan_host needs %llu bytes",
                (unsigned long long)host_bytes);
  uint8_t* hb = static_cast<uint8_t*>(plan_host);
  if (host_bytes > 0) std::memset(hb, 0, host_bytes);
  if (!units.empty()) std::memcpy(hb, units.data(), units.size() * sizeof(WorkUnit));
  if (split) {
    int32_t* mi = reinterpret_cast<int32_t*>(hb + (off_merge - off_units));
    for (int b = 0; b < batch; ++b)
      for (int i = 0; i < nq[b]; ++i)
        for (int h = 0; h < num_qo_heads; ++h) {
          const int64_t e = (int64_t)(qo_indptr_h[b] + i) * num_qo_heads + h;
          mi[e] = static_cast<int32_t>(pbase[b] + ((int64_t)i * num_qo_heads + h) * nsplit[b]);
        }
    mi[entries] = static_cast<int32_t>(partial);
  }
  if (!workspace) return ok();
  if (workspace_bytes < ws_bytes)
    return fail(NVFP4KV_ERR_WORKSPACE_TOO_SMALL, "workspace needs %llu bytes",
                (unsigned long long)ws_bytes);
  if (!aligned(workspace, 256))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (host_bytes > 0)
    e = cudaMemcpyAsync(ws + off_units, hb, host_bytes, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return cuda_fail(e, "plan upload");
  e = cudaMemsetAsync(ws + off_flags, 0, off_units - off_flags, stream);  // flags, counters
  if (e != cudaSuccess) return cuda_fail(e, "flag reset");
  return ok();
}

}  // extern "C"

namespace {

// The checks of a run apart from its cache: plan, workspace, device, query.
int check_plan_run(const nvfp4kv_plan_info* info, const void* q, int64_t qst, int64_t qsh,
                   const int32_t* kv_indices, const void* workspace, uint64_t workspace_bytes,
                   const void* out) {
  if (!workspace || workspace_bytes < info->workspace_bytes || !aligned(workspace, 256))
    return fail(NVFP4KV_ERR_WORKSPACE_TOO_SMALL, "workspace needs %llu bytes, 256-aligned",
                (unsigned long long)info->workspace_bytes);
  if (info->device >= 0) {  // the plan's SM count, occupancy and smem sizing
    int cur = -1;
    cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (cur != info->device)
      return fail(NVFP4KV_ERR_PLAN_MISMATCH, "plan made for device %d, current device is %d",
                  info->device, cur);
  }
  if (info->num_units == 0) return NVFP4KV_OK;
  if (!q || !kv_indices || !out)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null q / kv_indices / out");
  if (!aligned(q, 16) || qst % 8 || qsh % 8 || qst < 0 || qsh < 0 || !aligned(out, 4))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "q must be 16-byte aligned with strides multiple of 8 elements");
  return NVFP4KV_OK;
}

int check_run(const nvfp4kv_plan_info* info, const void* q, int64_t qst, int64_t qsh,
              const nvfp4kv_paged_cache* cache, const int32_t* kv_indices,
              const void* workspace, uint64_t workspace_bytes, const void* out) {
  if (!info || info->magic != kPlanMagic)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "info is not a plan");
  if (int st = check_cache(cache, true)) return st;
  if (cache->num_kv_heads != info->num_kv_heads || cache->head_dim_qk != info->head_dim_qk ||
      cache->head_dim_vo != info->head_dim_vo || cache->page_size != info->page_size)
    return fail(NVFP4KV_ERR_PLAN_MISMATCH, "cache dims differ from the plan");
  if (info->kernel == kKernelE4m3)
    return fail(NVFP4KV_ERR_PLAN_MISMATCH, "plan made for the E4M3 cache (kernel 5)");
  return check_plan_run(info, q, qst, qsh, kv_indices, workspace, workspace_bytes, out);
}

// The launch parameters that every attention kernel shares.
AttendParams run_params(const nvfp4kv_plan_info* info, const void* q, int64_t qst, int64_t qsh,
                        const CacheView& view, const int32_t* kv_indices, void* workspace,
                        void* out, float* lse) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttendParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride_tok = qst;
  p.q_stride_head = qsh;
  p.cache = view;
  p.kv_indices = kv_indices;
  p.units = reinterpret_cast<const WorkUnit*>(ws + info->off_units);
  p.num_units = info->num_units;
  p.num_qo_heads = info->num_qo_heads;
  p.group = info->num_qo_heads / info->num_kv_heads;
  p.causal = info->causal;
  p.split = info->split;
  p.page_size = info->page_size;
  p.out_f16 = info->out_dtype == 1;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.partial_o = reinterpret_cast<float*>(ws + info->off_partial_o);
  p.partial_lse = reinterpret_cast<float*>(ws + info->off_partial_lse);
  p.counters = reinterpret_cast<int*>(ws + info->off_counters);
  p.flags = reinterpret_cast<uint32_t*>(ws + info->off_flags);
  p.live_last_page_len = info->device_last_page_len;
  return p;
}

}  // namespace

namespace nvfp4kv {
int check_paged_cache(const nvfp4kv_paged_cache* cache, bool for_attention) {
  return check_cache(cache, for_attention);
}

// The argument checks of nvfp4kv_decode_run, for entry points that must
// validate before they enqueue anything of their own.
int validate_run(const nvfp4kv_plan_info* info, const void* q, int64_t qst, int64_t qsh,
                 const nvfp4kv_paged_cache* cache, const int32_t* kv_indices,
                 const void* workspace, uint64_t workspace_bytes, const void* out) {
  return check_run(info, q, qst, qsh, cache, kv_indices, workspace, workspace_bytes, out);
}
}  // namespace nvfp4kv

namespace {

struct TreeMask {
  const uint32_t* mask;
  int32_t words;
};

struct NewTokens {
  const void* k = nullptr;
  const void* v = nullptr;
  int64_t k_stride_tok = 0, k_stride_head = 0, v_stride_tok = 0, v_stride_head = 0;
};

// How the wide tree kernel runs a plan: in clusters of `ctas` CTAs that share a unit's value
// dims and its tokens, or (whole) those of all units of a pair of request and kv head, which
// the cluster then joins in place of the fold; sorted: in more than one wave, the longest pairs
// first, where the longest would hold the others up.
// Measured, a plan's units / whole pairs, us, 64 rows: one request of one kv head, 300 tokens
// 14.0 / 11.7, 4096 24.8 / 15.9, 32771 64 / 42; of 8 kv heads, 2000 tokens 20 / 14, 8000 22.5 /
// 20, 32771 36 / 44; 4 of 2000 18.5 / 16, of 32771 85 / 78 (145 without clusters); 8 of 4000
// 30.5 / 27; 4 of 500-8000 23 / 26; 512/256 heads, one of 2000 28 / 21.5, 8 of 2048-8192 57 /
// 67.  One wave / sorted: 18 requests of 1000-30000 tokens 210 / 169, 60 of 300-5000, 2 kv heads,
// 52 / 44, 512/256 heads, 30 of 500-8192, 140 / 95, 64/64 heads, 16 of 500-8192, 53 / 45; 16 of
// 512-4096 38 / 42, 12 of 100-8000 44 / 46.
struct TreeClusters {
  int ctas;
  bool whole, sorted;
  int64_t tokens;  // of a CTA, at most
};
constexpr int64_t kTreeTiles = 2;  // tiles of a whole unit that a CTA keeps
constexpr int kTreeSorted = 512;   // units among which a CTA finds its own by rank
TreeClusters tree_clusters(const nvfp4kv_plan_info* info, const TreeConfig& cfg, int blocks) {
  // The CTAs that share the value dims, doubled while the launch's stay one wave: of whole
  // pairs, one of clusters, whose CTAs are neighbours (16 of 8 CTAs are two waves, 38 us for
  // 26).  Among a plan's units are shorter ones, behind which a cluster too many finds room.
  auto grow = [&](int64_t units, int64_t tokens, bool whole) {
    int ctas = cfg.value_parts;
    while (ctas < 8 && units * blocks * ctas * 2 <= info->num_sms &&
           (!whole || units * blocks <= tree_max_clusters(cfg, ctas * 2)) &&
           tokens >= kTreeTiles * cfg.tile_tokens * (2 * ctas / cfg.value_parts))
      ctas *= 2;
    return ctas;
  };
  auto tiles = [&](int64_t tokens, int ctas) {  // of a CTA
    const int64_t share = (int64_t)cfg.tile_tokens * (ctas / cfg.value_parts);
    return (tokens + share - 1) / share;
  };
  const int64_t chunk = (int64_t)info->chunk_pages * kPageSize, splits = info->max_units_per_request;
  const int64_t pairs = (int64_t)info->batch * info->num_kv_heads, longest = chunk * splits;
  TreeClusters best{grow(info->num_units, chunk, false), false, false, chunk};
  if (pairs * blocks * cfg.value_parts > info->num_sms) return best;
  // In eighths of a tile (1.1 us): a CTA starts and ends in 7 tiles, one that finds its pair's
  // units in 8, one of several waves in 14; a fold takes 2.5, and 0.37 for each state of 64
  // rows of 128 dims; the last CTAs of several waves end an eighth late.
  const int64_t rows = std::min<int64_t>(kTreeRows, (int64_t)info->row_blocks * info->rows_per_block);
  const int64_t fold = splits < 2 ? 0 : 20 + 3 * splits * rows * info->head_dim_vo / 8192;
  const int64_t waves = ((int64_t)info->num_units * blocks * best.ctas + info->num_sms - 1) / info->num_sms;
  int64_t least = 8 * waves * (tiles(chunk, best.ctas) + 7) + fold;
  const int ctas = grow(pairs, longest, true);
  const int64_t whole = 8 * (tiles(longest, ctas) + 8);
  if (splits > 1 && whole <= least) {
    least = whole;
    best = {ctas, true, false, tiles(longest, ctas) * cfg.tile_tokens};
  }
  const int64_t mean = info->total_kv_pages * info->page_size / info->batch;
  for (int n = 2 * cfg.value_parts; n <= 8 && info->num_units <= kTreeSorted; n *= 2) {
    const int64_t all = pairs * blocks * n;
    if (all <= info->num_sms) continue;
    const int64_t cost =
        std::max(all * (tiles(mean, n) + 14) * 9 / info->num_sms, 8 * (tiles(longest, n) + 8));
    if (cost < least) {
      least = cost;
      best = {n, true, true, tiles(longest, n) * cfg.tile_tokens};
    }
  }
  return best;
}

// Trees: more than 16 rows a kv head go to the kernel of 128-row blocks (it takes a plan
// of either kernel), up to 16 to the mma.sync kernel's own form; but 9 to 16 rows where a
// cluster takes a whole request of few tokens a CTA (16 rows, 8 kv heads, the former for the
// latter, us: 128/128 heads, one request of 300 tokens 10 / 12, 4096 14 / 21, 4 of 2000 14 /
// 17.5, 8 of 4000 33 / 30; 256/256, 1000 13 / 23; 512/256, 1000 15 / 22; 64/64, 300 9 / 8.5,
// 1000 10 / 9.6).  Other batches, the former / the latter: 16 requests of 512-4096 tokens x 16
// rows 34 / 32, x 20 rows 36 / 61, x 64 39 / 95; 4 x 32771 tokens x 16 rows 71 / 67, x 20 rows
// 72 / 127; 512/256 heads x 32 rows 35 / 61; 64/64 heads x 20 rows 20 / 26, 56 / 66 and 69 /
// 83, two requests of 500 10 / 9.
struct TreeLaunch {
  bool wide;  // the kernel of 128-row blocks, in the form that follows
  TreeConfig cfg;
  TreeClusters clusters;
  int blocks;
};
int tree_launch_of(const nvfp4kv_plan_info* info, TreeLaunch* t) {
  *t = TreeLaunch{};
  const bool large = info->kernel == kKernelTcgen05 || info->row_blocks > 1;
  TreeConfig cfg{};
  if ((!large && info->rows_per_block <= 8) ||
      !attend_config_tree(info->head_dim_qk, info->head_dim_vo, &cfg))
    return NVFP4KV_OK;
  AttendConfig wide{};
  wide.func = cfg.func;
  wide.smem_bytes = cfg.smem_bytes;
  if (cudaError_t e = prepare_kernel(wide)) return cuda_fail(e, "kernel attributes");
  const int blocks = (info->row_blocks * info->rows_per_block + kTreeRows - 1) / kTreeRows;
  const TreeClusters clusters = tree_clusters(info, cfg, blocks);
  const int dk = info->head_dim_qk;
  if (large || (dk >= 128 && clusters.whole && !clusters.sorted &&
                clusters.tokens <= std::min(4 * dk, 1024)))
    *t = TreeLaunch{true, cfg, clusters, blocks};
  return NVFP4KV_OK;
}

// What a tree run asks of its plan.
int check_tree_plan(const nvfp4kv_plan_info* info) {
  if (info->kernel != kKernelTensorCore && info->kernel != kKernelTcgen05)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "trees run in the tensor-core kernels (plan option "
                "kernel 0, 1 or 3)");
  return NVFP4KV_OK;
}

int attend(const nvfp4kv_plan_info* info, const void* q_bf16, int64_t q_stride_tok,
           int64_t q_stride_head, const nvfp4kv_paged_cache* cache, const int32_t* kv_indices,
           float sm_scale, void* workspace, uint64_t workspace_bytes, void* out_bf16,
           float* lse, cudaStream_t stream, const NewTokens* nt, const TreeMask* tree = nullptr) {
  if (int st = check_run(info, q_bf16, q_stride_tok, q_stride_head, cache, kv_indices,
                         workspace, workspace_bytes, out_bf16))
    return st;
  if (tree) {
    if (int st = check_tree_plan(info)) return st;
    if (tree->words < 1 || tree->words > kMaxTreeNodes / 32)
      return fail(NVFP4KV_ERR_UNSUPPORTED, "mask_words %d (1 to %d)", tree->words,
                  kMaxTreeNodes / 32);
    if (info->num_units > 0 && (!tree->mask || !aligned(tree->mask, 4)))
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "tree_mask null or misaligned");
  }
  if (nt) {
    if (info->kernel != kKernelTensorCore && info->kernel != kKernelTcgen05 &&
        info->kernel != kKernelFp4QP)
      return fail(NVFP4KV_ERR_UNSUPPORTED, "the fused append runs in the tensor-core kernels");
    if (info->num_units > 0 &&
        (!nt->k || !nt->v || !aligned(nt->k, 16) || !aligned(nt->v, 16) ||
         nt->k_stride_tok % 8 || nt->k_stride_head % 8 || nt->v_stride_tok % 8 ||
         nt->v_stride_head % 8 || nt->k_stride_tok < 0 || nt->k_stride_head < 0 ||
         nt->v_stride_tok < 0 || nt->v_stride_head < 0))
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                  "new K/V must be 16-byte aligned with strides multiple of 8 elements");
  }
  if (info->num_units == 0) return ok();
  AttendConfig cfg{};
  // a tensor-core plan of one block of <= 8 rows runs the bulk-copy decode
  // kernel when the cache layout allows it (same arithmetic, same occupancy
  // or better: the plan's one-wave grid stays one wave)
  const bool dec = !tree && info->kernel == kKernelTensorCore && info->rows_per_block == 8 &&
                   info->page_size == kPageSize && bulk_decode_layout(cache) &&
                   attend_config_dec(info->head_dim_qk, info->head_dim_vo, 8,
                                     info->num_units <= info->num_sms ? 1 : 4, &cfg);
  TreeLaunch launch{};
  if (tree)
    if (int st = tree_launch_of(info, &launch)) return st;
  if (launch.wide) {
    cfg.func = launch.cfg.func;
    cfg.smem_bytes = launch.cfg.smem_bytes;
  }
  if (!dec && !launch.wide &&
      !lookup_kernel(info->kernel, info->head_dim_qk, info->head_dim_vo, info->page_size,
                     info->rows_per_block, &cfg, tree != nullptr))
    return fail(NVFP4KV_ERR_UNSUPPORTED, "planned kernel not available");
  cudaError_t e = prepare_kernel(cfg);
  if (e != cudaSuccess) return cuda_fail(e, "kernel attributes");
  if (!(sm_scale > 0.f)) sm_scale = 1.0f / std::sqrt(static_cast<float>(info->head_dim_qk));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttendParams p = run_params(info, q_bf16, q_stride_tok, q_stride_head, view_of(cache),
                              kv_indices, workspace, out_bf16, lse);
  p.qk_scale_log2 = static_cast<float>(static_cast<double>(sm_scale) *
                                       cache->k_global_scale * 1.4426950408889634);
  p.v_scale = cache->v_global_scale;
  if (tree) {
    p.tree_mask = tree->mask;
    p.tree_words = tree->words;
    p.row_blocks = info->row_blocks;
  }
  if (nt) {
    p.new_k = static_cast<const uint16_t*>(nt->k);
    p.new_v = static_cast<const uint16_t*>(nt->v);
    p.nk_stride_tok = nt->k_stride_tok;
    p.nk_stride_head = nt->k_stride_head;
    p.nv_stride_tok = nt->v_stride_tok;
    p.nv_stride_head = nt->v_stride_head;
    p.k_global_scale = cache->k_global_scale;
    p.v_global_scale = cache->v_global_scale;
  }
  if (info->kernel == kKernelFp4QP) {
    // FP4 query and probabilities: the row-maximum pass (which also stores
    // the fused append's tokens), then the attention pass with those maxima
    AttendConfig mcfg{};
    if (!attend_config_tc_fp4qp(info->head_dim_qk, info->head_dim_vo, info->rows_per_block, 1,
                                &mcfg))
      return fail(NVFP4KV_ERR_UNSUPPORTED, "planned kernel not available");
    e = prepare_kernel(mcfg);
    if (e != cudaSuccess) return cuda_fail(e, "kernel attributes");
    p.row_max = reinterpret_cast<float*>(ws + info->off_row_max);
    p.row_max_splits = std::max(info->max_units_per_request, 1);
    e = launch_attend(mcfg, p, info->num_units, info->row_blocks, stream);
    if (e != cudaSuccess) return cuda_fail(e, "row-maximum launch");
    p.new_k = nullptr;
    p.new_v = nullptr;
  }
  if (launch.wide) {
    const TreeClusters& c = launch.clusters;
    p.tree_whole = c.whole ? info->num_units : 0;
    p.tree_sorted = c.sorted;
    const int grid = c.whole ? info->batch * info->num_kv_heads : info->num_units;
    e = launch_attend_tree(launch.cfg, p, grid, launch.blocks, c.ctas, stream);
  } else {
    e = launch_attend(cfg, p, info->num_units, info->row_blocks, stream);
  }
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return ok();
}

}  // namespace

namespace nvfp4kv {

int attend_e4m3(const nvfp4kv_plan_info* info, const void* q, int64_t q_stride_tok,
                int64_t q_stride_head, int32_t q_dtype, const CacheView& view, int num_kv_heads,
                int page_size, int head_dim_qk, int head_dim_vo, const int32_t* kv_indices,
                float sm_scale, void* workspace, uint64_t workspace_bytes, void* out, float* lse,
                cudaStream_t stream) {
  if (!info || info->magic != kPlanMagic)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "info is not a plan");
  if (info->kernel != kKernelE4m3)
    return fail(NVFP4KV_ERR_PLAN_MISMATCH, "the E4M3 cache needs a plan with kernel = 5");
  if (num_kv_heads != info->num_kv_heads || head_dim_qk != info->head_dim_qk ||
      head_dim_vo != info->head_dim_vo || page_size != info->page_size)
    return fail(NVFP4KV_ERR_PLAN_MISMATCH, "cache dims differ from the plan");
  if (int st = check_plan_run(info, q, q_stride_tok, q_stride_head, kv_indices, workspace,
                              workspace_bytes, out))
    return st;
  if (info->num_units == 0) return ok();
  if (!aligned(out, 8) || !aligned(lse, 4))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "out must be 8-byte and lse 4-byte aligned");
  AttendConfig cfg{};
  if (!lookup_kernel(kKernelE4m3, info->head_dim_qk, info->head_dim_vo, info->page_size,
                     info->rows_per_block, &cfg))
    return fail(NVFP4KV_ERR_UNSUPPORTED, "planned kernel not available");
  cudaError_t e = prepare_kernel(cfg);
  if (e != cudaSuccess) return cuda_fail(e, "kernel attributes");
  if (!(sm_scale > 0.f)) sm_scale = 1.0f / std::sqrt(static_cast<float>(info->head_dim_qk));
  AttendParams p = run_params(info, q, q_stride_tok, q_stride_head, view, kv_indices, workspace,
                              out, lse);
  p.qk_scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  p.v_scale = 1.f;
  p.q_f16 = q_dtype;
  e = launch_attend(cfg, p, info->num_units, info->row_blocks, stream);
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return ok();
}

}  // namespace nvfp4kv

extern "C" {

int nvfp4kv_decode_attend(const nvfp4kv_plan_info* info, const void* q_bf16,
                          int64_t q_stride_tok, int64_t q_stride_head,
                          const nvfp4kv_paged_cache* cache, const int32_t* kv_indices,
                          float sm_scale, void* workspace, uint64_t workspace_bytes,
                          void* out_bf16, float* lse, cudaStream_t stream) {
  return attend(info, q_bf16, q_stride_tok, q_stride_head, cache, kv_indices, sm_scale,
                workspace, workspace_bytes, out_bf16, lse, stream, nullptr);
}

int nvfp4kv_decode_append_run(const nvfp4kv_plan_info* info, const void* new_k_bf16,
                              int64_t k_stride_tok, int64_t k_stride_head,
                              const void* new_v_bf16, int64_t v_stride_tok,
                              int64_t v_stride_head, const void* q_bf16,
                              int64_t q_stride_tok, int64_t q_stride_head,
                              const nvfp4kv_paged_cache* cache, const int32_t* kv_indices,
                              float sm_scale, void* workspace, uint64_t workspace_bytes,
                              void* out_bf16, float* lse, cudaStream_t stream) {
  NewTokens nt;
  nt.k = new_k_bf16;
  nt.v = new_v_bf16;
  nt.k_stride_tok = k_stride_tok;
  nt.k_stride_head = k_stride_head;
  nt.v_stride_tok = v_stride_tok;
  nt.v_stride_head = v_stride_head;
  return attend(info, q_bf16, q_stride_tok, q_stride_head, cache, kv_indices, sm_scale,
                workspace, workspace_bytes, out_bf16, lse, stream, &nt);
}

int nvfp4kv_tree_run(const nvfp4kv_plan_info* info, const uint32_t* tree_mask, int32_t mask_words,
                     const void* new_k_bf16, int64_t k_stride_tok, int64_t k_stride_head,
                     const void* new_v_bf16, int64_t v_stride_tok, int64_t v_stride_head,
                     const void* q_bf16, int64_t q_stride_tok, int64_t q_stride_head,
                     const nvfp4kv_paged_cache* cache, const int32_t* kv_indices, float sm_scale,
                     void* workspace, uint64_t workspace_bytes, void* out_bf16, float* lse,
                     cudaStream_t stream) {
  if (!new_k_bf16 != !new_v_bf16)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "new_k and new_v: both or neither");
  NewTokens nt;
  nt.k = new_k_bf16;
  nt.v = new_v_bf16;
  nt.k_stride_tok = k_stride_tok;
  nt.k_stride_head = k_stride_head;
  nt.v_stride_tok = v_stride_tok;
  nt.v_stride_head = v_stride_head;
  const TreeMask tree{tree_mask, mask_words};
  return attend(info, q_bf16, q_stride_tok, q_stride_head, cache, kv_indices, sm_scale,
                workspace, workspace_bytes, out_bf16, lse, stream, new_k_bf16 ? &nt : nullptr,
                &tree);
}

int nvfp4kv_tree_form(const nvfp4kv_plan_info* info, nvfp4kv_tree_launch* form) {
  if (!info || info->magic != kPlanMagic)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "info is not a plan");
  if (!form) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "form is null");
  if (int st = check_tree_plan(info)) return st;
  *form = nvfp4kv_tree_launch{};
  if (info->num_units == 0) return ok();
  TreeLaunch t{};
  if (int st = tree_launch_of(info, &t)) return st;
  form->block_rows = t.wide ? kTreeRows : info->rows_per_block;
  form->row_blocks = t.wide ? t.blocks : info->row_blocks;
  form->cluster_ctas = t.wide ? t.clusters.ctas : 1;
  form->value_ctas = t.wide ? t.cfg.value_parts : 1;
  form->whole_requests = t.wide && t.clusters.whole;
  form->longest_first = t.wide && t.clusters.sorted;
  form->folded = info->split && !form->whole_requests;
  return ok();
}

int nvfp4kv_decode_merge(const nvfp4kv_plan_info* info, void* workspace,
                         uint64_t workspace_bytes, void* out_bf16, float* lse,
                         cudaStream_t stream) {
  if (!info || info->magic != kPlanMagic)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "info is not a plan");
  if (!info->split) return ok();
  if (!workspace || workspace_bytes < info->workspace_bytes || !aligned(workspace, 256))
    return fail(NVFP4KV_ERR_WORKSPACE_TOO_SMALL, "workspace needs %llu bytes",
                (unsigned long long)info->workspace_bytes);
  if (!out_bf16) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "out is null");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaError_t e = launch_merge(
      reinterpret_cast<const float*>(ws + info->off_partial_o),
      reinterpret_cast<const float*>(ws + info->off_partial_lse),
      reinterpret_cast<const int32_t*>(ws + info->off_merge_indptr),
      static_cast<int32_t>((int64_t)info->total_qo_rows * info->num_qo_heads),
      info->head_dim_vo, static_cast<uint16_t*>(out_bf16), lse, info->out_dtype == 1, stream);
  if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  return ok();
}

int nvfp4kv_decode_run(const nvfp4kv_plan_info* info, const void* q_bf16,
                       int64_t q_stride_tok, int64_t q_stride_head,
                       const nvfp4kv_paged_cache* cache, const int32_t* kv_indices,
                       float sm_scale, void* workspace, uint64_t workspace_bytes,
                       void* out_bf16, float* lse, cudaStream_t stream) {
  // the split-KV merge is fused into the attention kernel
  return nvfp4kv_decode_attend(info, q_bf16, q_stride_tok, q_stride_head, cache, kv_indices,
                               sm_scale, workspace, workspace_bytes, out_bf16, lse, stream);
}

int nvfp4kv_merge_states(const float* o_partial, const float* lse_partial,
                         const int32_t* merge_indptr, int32_t num_entries,
                         int32_t head_dim_vo, void* out_bf16, float* lse,
                         cudaStream_t stream) {
  if (num_entries < 0) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num_entries < 0");
  if (head_dim_vo <= 0 || head_dim_vo % 32 || head_dim_vo > 512)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "head_dim_vo %d: multiple of 32, at most 512",
                head_dim_vo);
  if (num_entries == 0) return ok();
  if (!o_partial || !lse_partial || !merge_indptr || !out_bf16)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null pointer");
  if (!aligned(o_partial, 16) || !aligned(out_bf16, 2))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "o_partial must be 16-byte aligned");
  cudaError_t e = launch_merge(o_partial, lse_partial, merge_indptr, num_entries, head_dim_vo,
                               static_cast<uint16_t*>(out_bf16), lse, false, stream);
  if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  return ok();
}

int nvfp4kv_workspace_flags(const nvfp4kv_plan_info* info, const void* workspace,
                            uint32_t* flags, int32_t clear, cudaStream_t stream) {
  if (!info || info->magic != kPlanMagic || !workspace || !flags)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "bad arguments");
  const uint8_t* ws = static_cast<const uint8_t*>(workspace);
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, ws + info->off_flags, 4, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "flag read");
  if (clear) {
    e = cudaMemsetAsync(const_cast<uint8_t*>(ws) + info->off_flags, 0, 4, stream);
    if (e != cudaSuccess) return cuda_fail(e, "flag clear");
  }
  *flags = v;
  if (v) return fail(NVFP4KV_ERR_DEVICE_CHECK, "device flags 0x%x", v);
  return ok();
}

}  // extern "C"
