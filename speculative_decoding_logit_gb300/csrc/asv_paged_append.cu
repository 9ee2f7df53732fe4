// asv_paged_append.cu -- paged_kv_append: the new tokens' keys (rotated by position) and values into
// the pages of the cache, and the rotated queries.
//
// Per token: R_p turns the pairs of every query and key head by the position's angles, cos and sin from
// the caller's table (fp32); values are copied.  Each element is read once and written once and nothing
// is used twice but the table's row, so the launch is bound by HBM for long batches and by its chain of
// dependent loads (indptr, cache_len, block table and table row, each an L2 or HBM latency) for short
// ones.
//
// One CTA per token.  Its threads first take their vectors of q, k and v (independent of the chain, so
// their latency overlaps it), then find the token's request by counting the requests that end before
// it, one load per thread and 256 requests, and share one copy of the table's row.
#include "asv_paged_device.cuh"

namespace asv {

namespace {

constexpr int kThreads = 256;

// The rotated element of a pair: a cos - b sin for its first element, a cos + b sin for its second (a
// the element, b its partner).
__device__ __forceinline__ float turn(float a, float b, float c, float s, bool second) {
  return second ? fmaf(a, c, b * s) : fmaf(a, c, -(b * s));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a) {
  __shared__ float s_cs[128];  // cos of the position's angles, then their sines
  const PagedView& c = a.c;
  const int token = blockIdx.x, tid = threadIdx.x;
  const int vecs = c.head_dim / 8;
  const int n_rot = (a.q_heads + c.kv_heads) * vecs;
  const int items = n_rot + c.kv_heads * vecs;

  // the request: the first whose rows end after this token
  int before = 0;
  for (int i = 0; i < c.B; i += kThreads) {
    const bool ends = i + tid < c.B && c.indptr[i + tid + 1] <= token;
    before += __syncthreads_count(ends);
  }
  const long long limit = a.rotary != nullptr ? min((long long)a.max_position, table_positions(c)) : table_positions(c);
  if (token == 0)  // one CTA looks every request over
    for (int b = tid; b < c.B; b += kThreads)
      if (!load_request(c, b, limit).ok) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
  if (before >= c.B) return;
  const Request r = load_request(c, before, limit);
  if (!r.ok || token < r.start || token >= r.end) return;
  const int pos = r.past + (token - r.start);
  const int entry = pos / c.page_size, slot = pos % c.page_size;
  const int page = c.table[before * c.table_stride + entry];
  const bool page_ok = page >= 0 && page < c.num_pages;
  if (!page_ok && tid == 0) atomicOr(a.status + before, ASV_REQ_BAD_PAGE);
  if (a.rotary != nullptr && tid < a.rot_dim) s_cs[tid] = a.rotary[(long long)pos * a.rot_dim + tid];
  __syncthreads();
  const int half = a.rot_dim / 2;

  for (int i = tid; i < items; i += kThreads) {
    const int head = i / vecs, d0 = (i - head * vecs) * 8;
    const bool is_q = head < a.q_heads, is_k = !is_q && head < a.q_heads + c.kv_heads;
    const int h = is_q ? head : is_k ? head - a.q_heads : head - a.q_heads - c.kv_heads;
    const RowsView& in = is_q ? a.q : is_k ? a.k : a.v;
    const uint16_t* row = in.p + token * in.tok + h * in.head;
    uint4 x = *reinterpret_cast<const uint4*>(row + d0);
    uint16_t* dst;
    if (is_q) dst = a.out_q.p + token * a.out_q.tok + h * a.out_q.head;
    else if (is_k) dst = c.k + page * c.k_page + slot * c.k_slot + h * c.k_head;
    else dst = c.v + page * c.v_page + slot * c.v_slot + h * c.v_head;
    if (!is_q && !page_ok) continue;
    if ((is_q || is_k) && d0 < a.rot_dim) {
      uint32_t* w = &x.x;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = d0 + e;
        const float2 pair = unpack2<BF16>(w[e / 2]);
        const float self = e % 2 ? pair.y : pair.x;
        y[e] = self;
        if (d < a.rot_dim) {
          const bool second = a.interleaved ? d % 2 : d >= half;
          const int partner = a.interleaved ? d ^ 1 : second ? d - half : d + half;
          const int j = a.interleaved ? d / 2 : second ? d - half : d;
          y[e] = turn(self, unpack1<BF16>(row[partner]), s_cs[j], s_cs[half + j], second);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack2<BF16>(y[2 * e], y[2 * e + 1]);
    }
    *reinterpret_cast<uint4*>(dst + d0) = x;
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int dtype, cudaStream_t s) {
  if (dtype == ASV_BF16) paged_append_kernel<true><<<a.c.N, kThreads, 0, s>>>(a);
  else paged_append_kernel<false><<<a.c.N, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace asv
