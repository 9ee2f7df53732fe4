// asv_paged_api.cu -- the extern "C" entry points over the paged key/value cache declared in
// include/asv.h: argument validation and dispatch.
#include <cmath>

#include "asv.h"
#include "asv_internal.h"
#include "asv_paged.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes of the cache and the batch, then the element type.
asv_status check_sizes(const asv_paged_cache& c, const asv_paged_batch& b) {
  if (b.B < 0 || b.N < 0 || b.max_pages < 0 || c.num_pages < 1) return ASV_ERR_SHAPE;
  if (c.page_size < 8 || c.page_size % 8 != 0 || c.kv_heads < 1 || c.kv_heads > 1024) return ASV_ERR_SHAPE;
  if (c.head_dim < 8 || c.head_dim % 8 != 0 || c.head_dim > 128) return ASV_ERR_SHAPE;
  // positions are 32-bit
  if ((long long)b.max_pages * c.page_size > 0x7fff0000LL) return ASV_ERR_SHAPE;
  if (c.dtype != ASV_BF16 && c.dtype != ASV_F16) return ASV_ERR_DTYPE;
  return ASV_OK;
}

// A stride that is used (extent above 1) is a positive multiple of 8 elements, 16 bytes.
bool stride_ok(long long extent, int64_t s) { return extent <= 1 || (s > 0 && s % 8 == 0); }

bool rows_ok(const asv_rows* r, int N, int heads) {
  return !r || (aligned(r->data, 16) && stride_ok(N, r->stride_token) && stride_ok(heads, r->stride_head));
}

bool cache_ok(const asv_paged_cache& c, const asv_paged_batch& b) {
  return aligned(c.k, 16) && aligned(c.v, 16) && stride_ok(c.num_pages, c.k_stride_page) &&
         stride_ok(c.page_size, c.k_stride_slot) && stride_ok(c.kv_heads, c.k_stride_head) &&
         stride_ok(c.num_pages, c.v_stride_page) && stride_ok(c.page_size, c.v_stride_slot) &&
         stride_ok(c.kv_heads, c.v_stride_head) && aligned(b.indptr, 4) && aligned(b.cache_len, 4) &&
         aligned(b.block_table, 4);
}

bool cache_given(const asv_paged_cache& c, const asv_paged_batch& b) {
  return c.k && c.v && b.indptr && b.cache_len && (b.max_pages == 0 || b.block_table);
}

asv::RowsView rows_view(const asv_rows& r, int N, int heads) {
  return {static_cast<uint16_t*>(r.data), N > 1 ? r.stride_token : 0, heads > 1 ? r.stride_head : 0};
}

asv::PagedView paged_view(const asv_paged_cache& c, const asv_paged_batch& b) {
  asv::PagedView v;
  v.k = static_cast<uint16_t*>(c.k);
  v.v = static_cast<uint16_t*>(c.v);
  v.num_pages = c.num_pages;
  v.page_size = c.page_size;
  v.kv_heads = c.kv_heads;
  v.head_dim = c.head_dim;
  v.k_page = c.num_pages > 1 ? c.k_stride_page : 0;
  v.k_slot = c.k_stride_slot;
  v.k_head = c.kv_heads > 1 ? c.k_stride_head : 0;
  v.v_page = c.num_pages > 1 ? c.v_stride_page : 0;
  v.v_slot = c.v_stride_slot;
  v.v_head = c.kv_heads > 1 ? c.v_stride_head : 0;
  v.B = b.B;
  v.N = b.N;
  v.indptr = b.indptr;
  v.cache_len = b.cache_len;
  v.table = b.block_table;
  v.max_pages = b.max_pages;
  v.table_stride = b.block_table_stride;
  return v;
}

}  // namespace

extern "C" {

asv_status paged_kv_append(const asv_paged_cache* cache, const asv_paged_batch* batch, const asv_rows* k,
                           const asv_rows* v, const asv_rows* q, const asv_rows* out_q, int q_heads,
                           const asv_rotary* rotary, uint32_t* out_req_status, cudaStream_t stream) {
  if (!cache || !batch) return ASV_ERR_NULL;
  const asv_paged_cache& c = *cache;
  const asv_paged_batch& b = *batch;
  asv_status st = check_sizes(c, b);
  if (st != ASV_OK) return st;
  if (q && (q_heads < 1 || q_heads > 128 * 1024)) return ASV_ERR_SHAPE;
  if (b.B == 0 || b.N == 0) return ASV_OK;
  if (rotary && (rotary->dim < 2 || rotary->dim % 2 != 0 || rotary->dim > c.head_dim || rotary->max_position < 1 ||
                 (rotary->interleaved != 0 && rotary->interleaved != 1)))
    return ASV_ERR_PARAM;
  if (!cache_ok(c, b) || !rows_ok(k, b.N, c.kv_heads) || !rows_ok(v, b.N, c.kv_heads) || !rows_ok(q, b.N, q_heads) ||
      !rows_ok(out_q, b.N, q_heads) || (rotary && !aligned(rotary->table, 4)) || !aligned(out_req_status, 4))
    return ASV_ERR_ALIGN;
  if (!cache_given(c, b) || !k || !k->data || !v || !v->data || (!q) != (!out_q) || (q && !q->data) ||
      (out_q && !out_q->data) || (rotary && !rotary->table) || !out_req_status)
    return ASV_ERR_NULL;
  asv::AppendArgs a = {};
  a.c = paged_view(c, b);
  a.k = rows_view(*k, b.N, c.kv_heads);
  a.v = rows_view(*v, b.N, c.kv_heads);
  if (q) {
    a.q = rows_view(*q, b.N, q_heads);
    a.out_q = rows_view(*out_q, b.N, q_heads);
    a.q_heads = q_heads;
  }
  if (rotary) {
    a.rotary = rotary->table;
    a.rot_dim = rotary->dim;
    a.max_position = rotary->max_position;
    a.interleaved = rotary->interleaved;
  }
  a.status = out_req_status;
  cudaError_t e = asv::launch_paged_append(a, c.dtype, stream);
  return e == cudaSuccess ? ASV_OK : asv::record_cuda_error(e);
}

size_t asv_paged_workspace_bytes(int q_heads, int kv_heads, int head_dim) {
  if (kv_heads < 1 || q_heads < kv_heads || head_dim < 1 || head_dim > 128) return 0;
  return asv::paged_workspace_bytes(head_dim) + asv::kCheckLogBytes;
}

asv_status paged_attention(const asv_paged_cache* cache, const asv_paged_batch* batch, const asv_rows* q,
                           const asv_rows* out, int q_heads, float scale, int window, float* out_lse,
                           uint32_t* out_req_status, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!cache || !batch) return ASV_ERR_NULL;
  const asv_paged_cache& c = *cache;
  const asv_paged_batch& b = *batch;
  asv_status st = check_sizes(c, b);
  if (st != ASV_OK) return st;
  if (q_heads < 1 || q_heads % c.kv_heads != 0 || q_heads / c.kv_heads > 128) return ASV_ERR_SHAPE;
  if (b.B == 0 || b.N == 0) return ASV_OK;
  if (!std::isfinite(scale) || !(scale > 0.0f) || window < 0) return ASV_ERR_PARAM;
  if (!cache_ok(c, b) || !rows_ok(q, b.N, q_heads) || !rows_ok(out, b.N, q_heads) || !aligned(out_lse, 4) ||
      !aligned(out_req_status, 4) || !aligned(workspace, 256))
    return ASV_ERR_ALIGN;
  if (!cache_given(c, b) || !q || !q->data || !out || !out->data || !out_req_status) return ASV_ERR_NULL;
  if (!workspace || ws_bytes < asv_paged_workspace_bytes(q_heads, c.kv_heads, c.head_dim)) return ASV_ERR_WORKSPACE;
  asv::AttendArgs a = {};
  a.c = paged_view(c, b);
  a.q = rows_view(*q, b.N, q_heads);
  a.out = rows_view(*out, b.N, q_heads);
  a.q_heads = q_heads;
  a.group = q_heads / c.kv_heads;
  a.scale = scale;
  a.window = window;
  a.lse = out_lse;
  a.status = out_req_status;
  a.tickets = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + asv::kPagedTicketBytes);
  if (asv::kCheckLogBytes)
    a.check_log = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + asv::paged_workspace_bytes(c.head_dim));
  cudaError_t e = asv::launch_paged_attention(a, c.dtype, stream);
  return e == cudaSuccess ? ASV_OK : asv::record_cuda_error(e);
}

}  // extern "C"
