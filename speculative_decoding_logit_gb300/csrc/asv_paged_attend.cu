// asv_paged_attend.cu -- paged_attention: attention of a chunk of new tokens over a paged cache.
//
// One warp per (token, query head): the lanes score 32 keys at a time against the query row (held in
// shared memory, fp32), the softmax's maximum and sum run along, and the weighted values accumulate
// with the lanes spread over the head's entries.
#include "asv_paged_device.cuh"

namespace asv {

namespace {

constexpr int kWarps = 4;

template <bool BF16>
__global__ void __launch_bounds__(32 * kWarps) paged_attention_kernel(const AttendArgs a) {
  __shared__ float s_q[kWarps][128];
  const PagedView& c = a.c;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int token = blockIdx.x, head = blockIdx.y * kWarps + warp;
  const int D = c.head_dim;
  int before = 0;
  for (int i = 0; i < c.B; i += 32 * kWarps) {
    const int j = i + int(threadIdx.x);
    before += __syncthreads_count(j < c.B && c.indptr[j + 1] <= token);
  }
  if (token == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < c.B; b += 32 * kWarps)
      if (!load_request(c, b, table_positions(c)).ok) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
  if (before >= c.B || head >= a.q_heads) return;
  const Request r = load_request(c, before, table_positions(c));
  if (token < r.start || token >= r.end) return;
  uint16_t* out = a.out.p + token * a.out.tok + head * a.out.head;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // entries 4 * lane + e
  float top = -INFINITY, sum = 0.0f;
  if (r.ok) {
    for (int d = lane; d < D; d += 32)
      s_q[warp][d] = unpack1<BF16>(a.q.p[token * a.q.tok + head * a.q.head + d]);
    __syncwarp();
    const int last = r.past + (token - r.start);
    const int first = a.window > 0 ? max(0, last - a.window + 1) : 0;
    const long long kh = (head / a.group) * c.k_head, vh = (head / a.group) * c.v_head;
    for (int j0 = first; j0 <= last; j0 += 32) {
      const int j = j0 + lane;
      float s = -INFINITY;
      int page = -1;
      if (j <= last) {
        page = c.table[before * c.table_stride + j / c.page_size];
        if (page < 0 || page >= c.num_pages) {
          atomicOr(a.status + before, ASV_REQ_BAD_PAGE);
          page = -1;
        } else {
          const uint16_t* k = c.k + page * c.k_page + (j % c.page_size) * c.k_slot + kh;
          s = 0.0f;
          for (int d = 0; d < D; d += 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(k + d);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = unpack2<BF16>(w[e]);
              s = fmaf(y.x, s_q[warp][d + 2 * e], s);
              s = fmaf(y.y, s_q[warp][d + 2 * e + 1], s);
            }
          }
          s *= a.scale;
        }
      }
      const float next = fmaxf(top, warp_max(s));
      const float ref = next == -INFINITY ? 0.0f : next;
      const float keep = expf(top - ref);
      const float p = expf(s - ref);
      top = next;
      sum = sum * keep + p;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= keep;
      for (int i = 0; i < 32 && j0 + i <= last; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i);
        const int pg = __shfl_sync(0xffffffffu, page, i);
        if (pg < 0 || 4 * lane >= D) continue;
        const uint16_t* v = c.v + pg * c.v_page + ((j0 + i) % c.page_size) * c.v_slot + vh;
        const uint2 x = *reinterpret_cast<const uint2*>(v + 4 * lane);
        const float2 lo = unpack2<BF16>(x.x), hi = unpack2<BF16>(x.y);
        acc[0] = fmaf(pi, lo.x, acc[0]);
        acc[1] = fmaf(pi, lo.y, acc[1]);
        acc[2] = fmaf(pi, hi.x, acc[2]);
        acc[3] = fmaf(pi, hi.y, acc[3]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  if (4 * lane < D)
    *reinterpret_cast<uint2*>(out + 4 * lane) =
        make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv), pack2<BF16>(acc[2] * inv, acc[3] * inv));
  if (lane == 0 && a.lse != nullptr)
    a.lse[(long long)token * a.q_heads + head] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_paged_attention(const AttendArgs& a, int dtype, cudaStream_t s) {
  const dim3 grid(a.c.N, (a.q_heads + kWarps - 1) / kWarps);
  if (dtype == ASV_BF16) paged_attention_kernel<true><<<grid, 32 * kWarps, 0, s>>>(a);
  else paged_attention_kernel<false><<<grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace asv
