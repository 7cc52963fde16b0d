// api_step.cpp -- host side of the serving-step entry points of
// include/nvfp4kv.h beside the NVFP4 attention: the page table of a step,
// rotary positions and the E4M3 cache (argument validation and dispatch).
#include "nvfp4kv.h"

#include <cmath>

#include <cuda_runtime_api.h>

#include "checks.h"
#include "internal.h"

namespace nvfp4kv {
// The attention of a plan whose kernel is 5, over an E4M3 cache whose
// arguments have been checked (api.cpp).
int attend_e4m3(const nvfp4kv_plan_info* info, const void* q, int64_t q_stride_tok,
                int64_t q_stride_head, int32_t q_dtype, const CacheView& view, int num_kv_heads,
                int page_size, int head_dim_qk, int head_dim_vo, const int32_t* kv_indices,
                float sm_scale, void* workspace, uint64_t workspace_bytes, void* out, float* lse,
                cudaStream_t stream);
}  // namespace nvfp4kv

using namespace nvfp4kv;

namespace {

// ---- sums of two doubles, 106 bits ------------------------------------------
// The frequency table is multiplied by positions up to 2^31 and holds units of
// 2^-64 turns: doubles alone are off by 2^11 units.  Error-free sums and products
// (Dekker 1971, Knuth); products are fused explicitly, so that every machine's
// compiler computes the same.
struct Wide {
  double hi, lo;  // the number hi + lo, |lo| at most half a unit of hi
};
constexpr double kMostTurns = 0x1p40;  // a position: past it 106 bits end above 2^-64

Wide two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Wide add(Wide a, Wide b) {
  const Wide s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const Wide u = two_sum(s.hi, s.lo + t.hi);
  return two_sum(u.hi, u.lo + t.lo);
}
Wide sub(Wide a, Wide b) { return add(a, {-b.hi, -b.lo}); }
Wide mul(Wide a, Wide b) {
  const double p = a.hi * b.hi;
  return two_sum(p, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, std::fma(a.hi, b.hi, -p))));
}
Wide div(Wide a, Wide b) {
  const double q = a.hi / b.hi;
  const Wide r = sub(a, mul(b, {q, 0.0}));
  const double q2 = r.hi / b.hi;
  const Wide r2 = sub(r, mul(b, {q2, 0.0}));
  return add(two_sum(q, q2), {r2.hi / b.hi, 0.0});
}
Wide power(Wide x, int n) {
  Wide y{1.0, 0.0};
  for (; n > 0; n >>= 1) {
    if (n & 1) y = mul(y, x);
    x = mul(x, x);
  }
  return y;
}

}  // namespace

namespace nvfp4kv {
int check_e4m3_cache(const nvfp4kv_e4m3_cache* c) {
  if (!c) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache is null");
  if (!c->k_data || !c->v_data || !c->k_scale || !c->v_scale)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache buffer pointer is null");
  if (c->page_size != kPageSize && c->page_size != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "page_size %d (16 and 1 are supported)", c->page_size);
  if (c->num_pages <= 0 || c->num_kv_heads <= 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num_pages %d / num_kv_heads %d must be > 0",
                c->num_pages, c->num_kv_heads);
  const int64_t dims[2] = {c->head_dim_qk, c->head_dim_vo};
  const int64_t data[2][3] = {{c->k_stride_page, c->k_stride_slot, c->k_stride_head},
                              {c->v_stride_page, c->v_stride_slot, c->v_stride_head}};
  const int64_t scale[2][2] = {{c->k_scale_stride_page, c->k_scale_stride_head},
                               {c->v_scale_stride_page, c->v_scale_stride_head}};
  for (int kv = 0; kv < 2; ++kv) {
    if (dims[kv] <= 0 || dims[kv] % 32 || dims[kv] > 512)
      return fail(NVFP4KV_ERR_UNSUPPORTED,
                  "head dims (%d, %d): each must be a multiple of 32 and at most 512",
                  c->head_dim_qk, c->head_dim_vo);
    for (int i = 0; i < 3; ++i)
      if (data[kv][i] < 0 || data[kv][i] % 16)
        return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                    "data strides must be non-negative multiples of 16 bytes");
    if (!lie_apart(dims[kv], {{c->num_pages, data[kv][0]},
                              {c->page_size, data[kv][1]},
                              {c->num_kv_heads, data[kv][2]}}))
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache strides make rows overlap");
    for (int i = 0; i < 2; ++i)
      if (scale[kv][i] < 0 || scale[kv][i] % 4)
        return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                    "scale strides must be non-negative multiples of 4 bytes");
    if (!lie_apart(4, {{c->num_pages, scale[kv][0]}, {c->num_kv_heads, scale[kv][1]}}))
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "scale strides overlap");
  }
  if (!aligned(c->k_data, 16) || !aligned(c->v_data, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "cache buffer misaligned");
  return NVFP4KV_OK;
}

}  // namespace nvfp4kv

// The checks of nvfp4kv_rope's arguments, and its launch parameters (num_tokens and both
// head counts 0 where there is nothing to do).
static int rope_params(const void* q, int64_t q_stride_tok, int64_t q_stride_head, void* q_out,
                       int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t num_qo_heads,
                       const void* k, int64_t k_stride_tok, int64_t k_stride_head, void* k_out,
                       int64_t k_out_stride_tok, int64_t k_out_stride_head, int32_t num_kv_heads,
                       int32_t num_tokens, const int32_t* positions, int32_t head_dim,
                       int32_t rotary_dim, int32_t interleaved, int32_t dtype,
                       const uint64_t* freq, float attention_factor, RopeParams* p) {
  if (num_tokens < 0 || num_qo_heads < 0 || num_kv_heads < 0 || num_qo_heads > (1 << 20) ||
      num_kv_heads > (1 << 20))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "bad num_tokens or head counts");
  if (dtype != 0 && dtype != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "dtype %d (0 bf16, 1 f16)", dtype);
  if (head_dim < 8 || head_dim % 8 || head_dim > 512)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "head_dim %d (a multiple of 8, at most 512)", head_dim);
  if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "rotary_dim %d (even, 2 to head_dim %d)", rotary_dim,
                head_dim);
  if (!std::isfinite(attention_factor))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "attention_factor is not finite");
  if (num_tokens == 0 || num_qo_heads + num_kv_heads == 0) return NVFP4KV_OK;
  if (!positions || !freq || (num_qo_heads > 0 && (!q || !q_out)) ||
      (num_kv_heads > 0 && (!k || !k_out)))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null pointer");
  if (!aligned(freq, 8)) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "freq misaligned");
  if ((num_qo_heads > 0 && (bad_row_strides(q, q_stride_tok, q_stride_head) ||
                            bad_row_strides(q_out, q_out_stride_tok, q_out_stride_head))) ||
      (num_kv_heads > 0 && (bad_row_strides(k, k_stride_tok, k_stride_head) ||
                            bad_row_strides(k_out, k_out_stride_tok, k_out_stride_head))))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "rows must be 16-byte aligned with strides multiple of 8 elements");
  // outputs hold every row apart; in place means the same rows
  if ((num_qo_heads > 0 && !lie_apart(head_dim, {{num_tokens, q_out_stride_tok},
                                                 {num_qo_heads, q_out_stride_head}})) ||
      (num_kv_heads > 0 && !lie_apart(head_dim, {{num_tokens, k_out_stride_tok},
                                                 {num_kv_heads, k_out_stride_head}})))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "output strides make rows overlap");
  if ((num_qo_heads > 0 && q == q_out &&
       (q_stride_tok != q_out_stride_tok || q_stride_head != q_out_stride_head)) ||
      (num_kv_heads > 0 && k == k_out &&
       (k_stride_tok != k_out_stride_tok || k_stride_head != k_out_stride_head)))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "in place needs the same strides");
  p->q = static_cast<const uint16_t*>(q);
  p->k = static_cast<const uint16_t*>(k);
  p->q_out = static_cast<uint16_t*>(q_out);
  p->k_out = static_cast<uint16_t*>(k_out);
  p->q_st = q_stride_tok; p->q_sh = q_stride_head;
  p->k_st = k_stride_tok; p->k_sh = k_stride_head;
  p->qo_st = q_out_stride_tok; p->qo_sh = q_out_stride_head;
  p->ko_st = k_out_stride_tok; p->ko_sh = k_out_stride_head;
  p->positions = positions;
  p->freq = freq;
  p->num_tokens = num_tokens;
  p->num_qo_heads = num_qo_heads;
  p->num_kv_heads = num_kv_heads;
  p->head_dim = head_dim;
  p->rotary_dim = rotary_dim;
  p->interleaved = interleaved ? 1 : 0;
  p->f16 = dtype;
  p->attention_factor = attention_factor;
  return NVFP4KV_OK;
}

extern "C" {

int nvfp4kv_build_page_table(const int32_t* kv_len, const int32_t* qo_len, int32_t batch,
                             int32_t page_size, int32_t* block_table,
                             int64_t block_table_stride, int32_t max_pages_per_request,
                             const int32_t* free_pages, int32_t num_free,
                             const int32_t* free_head, const nvfp4kv_step_table* out,
                             uint32_t* device_flags, cudaStream_t stream) {
  if (batch < 0 || max_pages_per_request < 0 || num_free < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "batch, max_pages_per_request or num_free < 0");
  if (batch > kMaxPageTableBatch)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "batch %d (at most %d)", batch, kMaxPageTableBatch);
  if (page_size < 1 || page_size > 65536)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "page_size %d (1 to 65536)", page_size);
  if (!out || !out->qo_indptr || !out->kv_indptr || !out->free_head)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null output");
  if (out->max_pages < 0 || out->max_tokens < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "max_pages or max_tokens < 0");
  if (batch > 0 && (!kv_len || !qo_len || !out->last_page_len))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null lengths");
  if (batch > 0 && max_pages_per_request > 0 && !block_table)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "block_table is null");
  if (batch > 1 && block_table_stride < max_pages_per_request)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "block table rows overlap");
  if ((num_free > 0 && !free_pages) || (out->max_pages > 0 && !out->kv_indices) ||
      (out->max_tokens > 0 && (!out->batch_idx || !out->positions)))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null list");
  if (free_head == out->free_head)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "the new free head must not overwrite the one that is read");
  if (!aligned(out->slot_map, 8))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "slot_map must be 8-byte aligned");
  PageTableParams p{};
  p.kv_len = kv_len;
  p.qo_len = qo_len;
  p.block_table = block_table;
  p.table_stride = block_table_stride;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.batch = batch;
  p.page_size = page_size;
  p.table_width = max_pages_per_request;
  p.num_free = num_free;
  p.max_tokens = out->max_tokens;
  p.max_pages = out->max_pages;
  p.qo_indptr = out->qo_indptr;
  p.kv_indptr = out->kv_indptr;
  p.last_page_len = out->last_page_len;
  p.kv_indices = out->kv_indices;
  p.batch_idx = out->batch_idx;
  p.positions = out->positions;
  p.slot_map = out->slot_map;
  p.free_head_out = out->free_head;
  p.flags = device_flags;
  return launched(launch_page_table(p, stream), "page table launch");
}

int nvfp4kv_rope_frequencies(int32_t rotary_dim, const nvfp4kv_rope_options* o,
                             uint64_t* freq_host) {
  if (!o || !freq_host) return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null pointer");
  if (rotary_dim < 2 || rotary_dim > 512 || rotary_dim % 2)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "rotary_dim %d (even, 2 to 512)", rotary_dim);
  if (!(o->base > 1.0) || !std::isfinite(o->base) || !(o->factor > 0.0) ||
      !std::isfinite(o->factor) || o->original_max_position < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "base > 1, factor > 0 and a length are needed");
  if (o->original_max_position > 0 &&
      !(o->high_rotations > o->low_rotations && o->low_rotations >= 0.0 &&
        std::isfinite(o->high_rotations)))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "high_rotations must exceed low_rotations >= 0");
  const int pairs = rotary_dim / 2;
  const Wide two_pi{6.283185307179586, 2.4492935982947064e-16};  // 2 pi to 2^-106
  // x = base^(-1 / pairs) by Newton's steps for base x^pairs = 1
  Wide x{std::pow(o->base, -1.0 / pairs), 0.0};
  for (int step = 0; step < 2 && pairs > 1; ++step) {
    const Wide rest = sub({1.0, 0.0}, mul(power(x, pairs), {o->base, 0.0}));
    x = add(x, mul(x, div(rest, {static_cast<double>(pairs), 0.0})));
  }
  const Wide factor{o->factor, 0.0};
  for (int i = 0; i < pairs; ++i) {
    Wide f = power(x, i);
    if (o->original_max_position > 0) {
      const int64_t n = o->original_max_position;
      const Wide length = two_sum(static_cast<double>(n >> 32) * 0x1p32,
                                  static_cast<double>(n & 0xFFFFFFFF));
      const Wide low{o->low_rotations, 0.0}, high{o->high_rotations, 0.0};
      Wide g = div(sub(div(mul(length, f), two_pi), low), sub(high, low));
      if (g.hi < 0.0) g = {0.0, 0.0};
      if (g.hi >= 1.0) g = {1.0, 0.0};
      f = add(div(mul(f, sub({1.0, 0.0}, g)), factor), mul(f, g));
    } else {
      f = div(f, factor);
    }
    // turns a position, its whole part dropped, in units of 2^-64
    const Wide turns = div(f, two_pi);
    if (!(turns.hi < kMostTurns))
      return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "factor %g: a frequency above 2^40 turns a position",
                  o->factor);
    Wide part = two_sum(turns.hi - std::floor(turns.hi), turns.lo);
    if (part.hi < 0.0) part = add(part, {1.0, 0.0});
    const double units = part.hi * 0x1p64, whole = std::floor(units);  // at most 2^64
    freq_host[i] = static_cast<uint64_t>(static_cast<unsigned __int128>(whole)) +
                   static_cast<uint64_t>(static_cast<int64_t>(
                       std::floor(units - whole + part.lo * 0x1p64 + 0.5)));
  }
  return ok();
}

int nvfp4kv_rope(const void* q, int64_t q_stride_tok, int64_t q_stride_head, void* q_out,
                 int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t num_qo_heads,
                 const void* k, int64_t k_stride_tok, int64_t k_stride_head, void* k_out,
                 int64_t k_out_stride_tok, int64_t k_out_stride_head, int32_t num_kv_heads,
                 int32_t num_tokens, const int32_t* positions, int32_t head_dim,
                 int32_t rotary_dim, int32_t interleaved, int32_t dtype, const uint64_t* freq,
                 float attention_factor, cudaStream_t stream) {
  RopeParams p{};
  if (int st = rope_params(q, q_stride_tok, q_stride_head, q_out, q_out_stride_tok,
                           q_out_stride_head, num_qo_heads, k, k_stride_tok, k_stride_head, k_out,
                           k_out_stride_tok, k_out_stride_head, num_kv_heads, num_tokens,
                           positions, head_dim, rotary_dim, interleaved, dtype, freq,
                           attention_factor, &p))
    return st;
  return launched(launch_rope(p, stream), "rope launch");
}

int nvfp4kv_norm_rope(const void* q, int64_t q_stride_tok, int64_t q_stride_head, void* q_out,
                      int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t num_qo_heads,
                      const void* k, int64_t k_stride_tok, int64_t k_stride_head, void* k_out,
                      int64_t k_out_stride_tok, int64_t k_out_stride_head, int32_t num_kv_heads,
                      int32_t num_tokens, const int32_t* positions, int32_t head_dim,
                      int32_t rotary_dim, int32_t interleaved, int32_t dtype, const uint64_t* freq,
                      float attention_factor, const void* q_weight, const void* k_weight,
                      int32_t weight_dtype, float weight_offset, float eps,
                      cudaStream_t stream) {
  NormRopeParams n{};
  if (int st = rope_params(q, q_stride_tok, q_stride_head, q_out, q_out_stride_tok,
                           q_out_stride_head, num_qo_heads, k, k_stride_tok, k_stride_head, k_out,
                           k_out_stride_tok, k_out_stride_head, num_kv_heads, num_tokens,
                           positions, head_dim, rotary_dim, interleaved, dtype, freq,
                           attention_factor, &n.rope))
    return st;
  if (weight_dtype != dtype && weight_dtype != 2)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "weight_dtype %d (that of the rows, or 2: float32)",
                weight_dtype);
  if (!(eps >= 1e-20f && eps <= 1e20f))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "eps must lie in [1e-20, 1e20]");
  if (!std::isfinite(weight_offset))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "weight_offset is not finite");
  if (n.rope.num_tokens == 0) return ok();
  if ((num_qo_heads > 0 && (!q_weight || !aligned(q_weight, 16))) ||
      (num_kv_heads > 0 && (!k_weight || !aligned(k_weight, 16))))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "weights must be 16-byte aligned");
  n.q_weight = q_weight;
  n.k_weight = k_weight;
  n.weight_f32 = weight_dtype == 2;
  n.weight_offset = weight_offset;
  n.eps = eps;
  return launched(launch_norm_rope(n, stream), "norm_rope launch");
}

int nvfp4kv_e4m3_append(const nvfp4kv_e4m3_cache* cache, const void* k, int64_t k_stride_tok,
                        int64_t k_stride_head, const void* v, int64_t v_stride_tok,
                        int64_t v_stride_head, int32_t dtype, int32_t num_rows,
                        const int32_t* qo_indptr, const int32_t* kv_indptr,
                        const int32_t* kv_indices, const int32_t* last_page_len, int32_t batch,
                        uint32_t* device_flags, cudaStream_t stream) {
  if (int st = check_e4m3_cache(cache)) return st;
  if (num_rows < 0 || batch < 0)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "num_rows %d / batch %d negative", num_rows, batch);
  if (dtype != 0 && dtype != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "dtype %d (0 bf16, 1 f16)", dtype);
  if (num_rows == 0 || batch == 0) return ok();
  if (!k || !v || !qo_indptr || !kv_indptr || !kv_indices || !last_page_len)
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT, "null input pointer");
  if (bad_row_strides(k, k_stride_tok, k_stride_head) ||
      bad_row_strides(v, v_stride_tok, v_stride_head))
    return fail(NVFP4KV_ERR_INVALID_ARGUMENT,
                "inputs must be 16-byte aligned with strides multiple of 8 elements");
  E4m3AppendParams p{};
  p.data[0] = cache->k_data; p.data[1] = cache->v_data;
  p.scale[0] = reinterpret_cast<uint8_t*>(cache->k_scale);
  p.scale[1] = reinterpret_cast<uint8_t*>(cache->v_scale);
  p.sp[0] = cache->k_stride_page; p.ss[0] = cache->k_stride_slot; p.sh[0] = cache->k_stride_head;
  p.sp[1] = cache->v_stride_page; p.ss[1] = cache->v_stride_slot; p.sh[1] = cache->v_stride_head;
  p.scp[0] = cache->k_scale_stride_page; p.sch[0] = cache->k_scale_stride_head;
  p.scp[1] = cache->v_scale_stride_page; p.sch[1] = cache->v_scale_stride_head;
  p.dim[0] = cache->head_dim_qk; p.dim[1] = cache->head_dim_vo;
  p.src[0] = static_cast<const uint16_t*>(k);
  p.src[1] = static_cast<const uint16_t*>(v);
  p.src_tok[0] = k_stride_tok; p.src_head[0] = k_stride_head;
  p.src_tok[1] = v_stride_tok; p.src_head[1] = v_stride_head;
  p.num_pages = cache->num_pages;
  p.page_size = cache->page_size;
  p.num_kv_heads = cache->num_kv_heads;
  p.num_rows = num_rows;
  p.batch = batch;
  p.f16 = dtype;
  p.qo_indptr = qo_indptr;
  p.kv_indptr = kv_indptr;
  p.kv_indices = kv_indices;
  p.last_page_len = last_page_len;
  p.flags = device_flags;
  return launched(launch_e4m3_append(p, stream), "e4m3_append launch");
}

int nvfp4kv_e4m3_decode_run(const nvfp4kv_plan_info* info, const void* q, int64_t q_stride_tok,
                            int64_t q_stride_head, int32_t q_dtype,
                            const nvfp4kv_e4m3_cache* cache, const int32_t* kv_indices,
                            float sm_scale, void* workspace, uint64_t workspace_bytes, void* out,
                            float* lse, cudaStream_t stream) {
  if (int st = check_e4m3_cache(cache)) return st;
  if (q_dtype != 0 && q_dtype != 1)
    return fail(NVFP4KV_ERR_UNSUPPORTED, "q_dtype %d (0 bf16, 1 f16)", q_dtype);
  CacheView v{};
  v.k_data = cache->k_data;
  v.v_data = cache->v_data;
  v.k_sf = reinterpret_cast<const uint8_t*>(cache->k_scale);
  v.v_sf = reinterpret_cast<const uint8_t*>(cache->v_scale);
  v.k_sp = cache->k_stride_page; v.k_ss = cache->k_stride_slot; v.k_sh = cache->k_stride_head;
  v.v_sp = cache->v_stride_page; v.v_ss = cache->v_stride_slot; v.v_sh = cache->v_stride_head;
  v.ksf_sp = cache->k_scale_stride_page; v.ksf_sh = cache->k_scale_stride_head;
  v.vsf_sp = cache->v_scale_stride_page; v.vsf_sh = cache->v_scale_stride_head;
  v.num_pages = cache->num_pages;
  return attend_e4m3(info, q, q_stride_tok, q_stride_head, q_dtype, v, cache->num_kv_heads,
                     cache->page_size, cache->head_dim_qk, cache->head_dim_vo, kv_indices,
                     sm_scale, workspace, workspace_bytes, out, lse, stream);
}

}  // extern "C"
