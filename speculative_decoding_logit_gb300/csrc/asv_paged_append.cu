// asv_paged_append.cu -- paged_kv_append: the new tokens' keys (rotated by position) and values into
// the pages of the cache, and the rotated queries.
//
// Per token: R_p turns the pairs of every query and key head by the position's angles, cos and sin from
// the caller's table (fp32); values are copied.  Each element is read once and written once and nothing
// is used twice but the table's row, so the launch is bound by HBM for long batches and by its chain of
// dependent loads (indptr, cache_len, block table and table row, each an L2 or HBM latency) for short
// ones.
//
// A CTA takes kTokens consecutive tokens: its first threads find their requests (all threads count the
// requests that end before the first token, 256 a step; the others are at most a few further), pages and
// slots, and the rows of the table come to shared memory once for all heads.  Then a task is one or two
// 16-byte vectors: where a pair's elements are dim / 2 apart and that is whole vectors, one thread has
// both, so every element is loaded once.
#include <algorithm>

#include "asv_paged_device.cuh"

namespace asv {

namespace {

constexpr int kThreads = 256;

// How a head's vectors are made tasks of.
enum Pairing {
  kPlain,     // a vector a task; pairs lie within it (interleaved), or nothing is rotated
  kHalves,    // vectors j and j + dim / 2 a task, and the vectors from dim on one by one
  kFours,  // a vector a task, its partners fetched by four (dim / 2 a multiple of 4)
  kScattered  // a vector a task, its partners fetched one by one
};

struct TokenPlace {
  int request, pos, page, slot;  // page < 0: not appended; request < 0: no token
};

// The elements of a pair turned: (a cos - b sin, b cos + a sin).
__device__ __forceinline__ float first_of(float a, float b, float c, float s) { return fmaf(a, c, -(b * s)); }
__device__ __forceinline__ float second_of(float a, float b, float c, float s) { return fmaf(b, c, a * s); }

template <bool BF16, int PAIRING, int TOKENS>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ __align__(16) float s_cs[TOKENS][128];  // cos of the positions' angles, then their sines
  __shared__ TokenPlace s_place[TOKENS];
  const PagedView& c = a.c;
  const int tid = threadIdx.x, token0 = blockIdx.x * TOKENS;
  const long long limit = a.rotary != nullptr ? min((long long)a.max_position, table_positions(c)) : table_positions(c);

  // What comes after on the stream may set itself up; what came before is needed from here on.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the tokens' requests and places
  int before = 0;
  for (int i = 0; i < c.B; i += kThreads) before += __syncthreads_count(i + tid < c.B && c.indptr[i + tid + 1] <= token0);
  if (tid < TOKENS) {
    const int token = token0 + tid;
    TokenPlace p = {-1, 0, -1, 0};
    int b = before;
    while (b < c.B && c.indptr[b + 1] <= token) ++b;
    if (token < c.N && b < c.B) {
      const Request r = load_request(c, b, limit);
      if (r.ok && token >= r.start && token < r.end) {
        p.request = b;
        p.pos = r.past + (token - r.start);
        const int entry = p.pos / c.page_size;
        p.slot = p.pos - entry * c.page_size;
        if (ASV_GUARD(a, entry >= 0 && entry < c.max_pages)) p.page = c.table[b * c.table_stride + entry];
        if (p.page < 0 || p.page >= c.num_pages) {
          atomicOr(a.status + b, ASV_REQ_BAD_PAGE);
          p.page = -1;
        }
      }
    }
    s_place[tid] = p;
  }
  if (blockIdx.x == 0)  // one CTA looks every request over
    for (int b = tid; b < c.B; b += kThreads)
      if (!load_request(c, b, limit).ok) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
  __syncthreads();
  if (a.rotary != nullptr) {
    for (int i = tid; i < TOKENS * a.rot_dim; i += kThreads) {
      const int t = i / a.rot_dim, j = i - t * a.rot_dim;
      if (s_place[t].request >= 0 && ASV_GUARD(a, s_place[t].pos >= 0 && s_place[t].pos < a.max_position && j < 128))
        s_cs[t][j] = a.rotary[(long long)s_place[t].pos * a.rot_dim + j];
    }
    __syncthreads();
  }

  // ---- the rows: a thread keeps its place within a head (no division per vector) and goes through the heads of
  // all tokens, kRows rows of the CTA's threads at a time
  const int half = a.rot_dim / 2, vecs = c.head_dim / 8;
  const int pairs = PAIRING == kHalves ? half / 8 : 0;  // tasks of two vectors
  const int tasks = vecs - pairs;
  {
    const int heads = a.q_heads + c.kv_heads;
    const int rows = kThreads / tasks, j = tid % tasks;
    const bool pair = j < pairs;
    const int d = (PAIRING == kHalves && !pair ? j + pairs : j) * 8;  // (the pairs take 2 * pairs vectors)
    int t = 0, h = tid / tasks;
    if (h >= rows) t = TOKENS;
#pragma unroll PAIRING == kHalves ? 2 : 4
    for (;; h += rows) {
      while (h >= heads && t < TOKENS) {
        h -= heads;
        ++t;
      }
      if (t >= TOKENS) break;
      const TokenPlace p = s_place[t];
      const bool is_q = h < a.q_heads;
      if (p.request < 0 || (!is_q && p.page < 0)) continue;
      const long long token = token0 + t;
      // the row, the vector and its partners within it, the slot
      if (!ASV_GUARD(a, token < c.N && p.request < c.B && h < heads && d + 8 <= c.head_dim &&
                            (PAIRING == kHalves && pair ? half + d + 8 <= a.rot_dim : PAIRING == kPlain || a.rot_dim <= c.head_dim) &&
                            (is_q || (p.page < c.num_pages && p.slot >= 0 && p.slot < c.page_size))))
        continue;
      const uint16_t* src = is_q ? a.q.p + token * a.q.tok + h * a.q.head
                                 : a.k.p + token * a.k.tok + (h - a.q_heads) * a.k.head;
      uint16_t* dst = is_q ? a.out_q.p + token * a.out_q.tok + h * a.out_q.head
                           : c.k + p.page * c.k_page + p.slot * c.k_slot + (h - a.q_heads) * c.k_head;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(src + d));
      uint32_t u[4] = {x.x, x.y, x.z, x.w};
      const float* cs = s_cs[t];
      if (PAIRING == kHalves && pair) {
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(src + half + d));
        uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 co = *reinterpret_cast<const float2*>(cs + d + 2 * e);
          const float2 si = *reinterpret_cast<const float2*>(cs + half + d + 2 * e);
          const float2 p0 = unpack2<BF16>(u[e]), p1 = unpack2<BF16>(w[e]);
          u[e] = pack2<BF16>(first_of(p0.x, p1.x, co.x, si.x), first_of(p0.y, p1.y, co.y, si.y));
          w[e] = pack2<BF16>(second_of(p0.x, p1.x, co.x, si.x), second_of(p0.y, p1.y, co.y, si.y));
        }
        *reinterpret_cast<uint4*>(dst + half + d) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (PAIRING == kFours && d < a.rot_dim) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int at = d + 4 * g;
          if (at < a.rot_dim) {
            const bool low = at < half;
            const int q = low ? at : at - half;
            const uint2 y = __ldg(reinterpret_cast<const uint2*>(src + (low ? at + half : q)));
            const float4 co = *reinterpret_cast<const float4*>(cs + q), si = *reinterpret_cast<const float4*>(cs + half + q);
            auto turn = [&](float2 own, float2 other, float c0, float c1, float s0, float s1) {
              return low ? pack2<BF16>(first_of(own.x, other.x, c0, s0), first_of(own.y, other.y, c1, s1))
                         : pack2<BF16>(second_of(other.x, own.x, c0, s0), second_of(other.y, own.y, c1, s1));
            };
            u[2 * g] = turn(unpack2<BF16>(u[2 * g]), unpack2<BF16>(y.x), co.x, co.y, si.x, si.y);
            u[2 * g + 1] = turn(unpack2<BF16>(u[2 * g + 1]), unpack2<BF16>(y.y), co.z, co.w, si.z, si.w);
          }
        }
      } else if (PAIRING != kHalves && d < a.rot_dim) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = unpack2<BF16>(u[e]);
          const int d0 = d + 2 * e;
          float2 z = v;
          if (PAIRING == kPlain) {
            if (d0 < a.rot_dim) {
              const float co = cs[d0 / 2], si = cs[half + d0 / 2];
              z = make_float2(first_of(v.x, v.y, co, si), second_of(v.x, v.y, co, si));
            }
          } else {
            auto turn = [&](int at, float own) {
              if (at >= a.rot_dim) return own;
              const int q = at < half ? at : at - half;
              const float other = unpack1<BF16>(src[at < half ? at + half : q]);
              return at < half ? first_of(own, other, cs[q], cs[half + q]) : second_of(other, own, cs[q], cs[half + q]);
            };
            z = make_float2(turn(d0, v.x), turn(d0 + 1, v.y));
          }
          u[e] = pack2<BF16>(z.x, z.y);
        }
      }
      *reinterpret_cast<uint4*>(dst + d) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  // values
  const int rows = kThreads / vecs, d = (tid % vecs) * 8;
  int t = 0, h = tid / vecs;
  if (h >= rows) return;
#pragma unroll 4
  for (;; h += rows) {
    while (h >= c.kv_heads && t < TOKENS) {
      h -= c.kv_heads;
      ++t;
    }
    if (t >= TOKENS) break;
    const TokenPlace p = s_place[t];
    if (p.request < 0 || p.page < 0) continue;
    if (!ASV_GUARD(a, token0 + t < c.N && h < c.kv_heads && d + 8 <= c.head_dim && p.page < c.num_pages && p.slot >= 0 &&
                          p.slot < c.page_size))
      continue;
    *reinterpret_cast<uint4*>(c.v + p.page * c.v_page + p.slot * c.v_slot + h * c.v_head + d) =
        __ldg(reinterpret_cast<const uint4*>(a.v.p + (long long)(token0 + t) * a.v.tok + h * a.v.head + d));
  }
}

template <bool BF16, int PAIRING>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  // a programmatic launch: the CTAs start while the launch before it ends
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // More tokens to a CTA share the search and the chain of loads, fewer have more loads in flight: doubled up to eight
  // while there are more than 13 CTAs to an SM, and up to sixteen while there are more than 8 and a CTA's threads have
  // less than four vectors each (9216 tokens of 576 vectors: 44 us at one token to a CTA, 34 at eight; 3995 of 525: 21,
  // 18.6 at two, 26 at eight; 15,713 of 60: 70, 17.8 at eight, 14.2 at sixteen).
  const long long vectors = (long long)(a.q_heads + 2 * a.c.kv_heads) * (a.c.head_dim / 8);
  int tokens = 1;
  auto ctas = [&]() { return (a.c.N + tokens - 1) / tokens; };
  while ((tokens < 8 && ctas() > 2048) || (tokens < 16 && ctas() > 1216 && tokens * vectors < 4 * kThreads)) tokens *= 2;
  cfg.gridDim = dim3(unsigned(ctas()), 1, 1);
  switch (tokens) {
    case 1: return cudaLaunchKernelEx(&cfg, paged_append_kernel<BF16, PAIRING, 1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, paged_append_kernel<BF16, PAIRING, 2>, a);
    case 4: return cudaLaunchKernelEx(&cfg, paged_append_kernel<BF16, PAIRING, 4>, a);
    case 8: return cudaLaunchKernelEx(&cfg, paged_append_kernel<BF16, PAIRING, 8>, a);
    default: return cudaLaunchKernelEx(&cfg, paged_append_kernel<BF16, PAIRING, 16>, a);
  }
}

#ifdef ASV_CHECKED
__device__ uint32_t g_check_log[2];  // the append has no workspace to keep a log in
#endif

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& args, int dtype, cudaStream_t s) {
#ifdef ASV_CHECKED
  AppendArgs a = args;
  void* log = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&log, g_check_log);
  if (e != cudaSuccess) return e;
  a.check_log = static_cast<uint32_t*>(log);
#else
  const AppendArgs& a = args;
#endif
  const int pairing = a.rotary == nullptr || a.interleaved ? kPlain
                      : a.rot_dim % 16 == 0                ? kHalves
                      : a.rot_dim % 8 == 0                 ? kFours
                                                           : kScattered;
  const bool bf16 = dtype == ASV_BF16;
  switch (pairing) {
    case kPlain: return bf16 ? launch<true, kPlain>(a, s) : launch<false, kPlain>(a, s);
    case kHalves: return bf16 ? launch<true, kHalves>(a, s) : launch<false, kHalves>(a, s);
    case kFours: return bf16 ? launch<true, kFours>(a, s) : launch<false, kFours>(a, s);
    default: return bf16 ? launch<true, kScattered>(a, s) : launch<false, kScattered>(a, s);
  }
}

}  // namespace asv

#ifdef ASV_CHECKED
// The append's check log (the count and the line of the first failure), when the device's work is done.  Returns a
// cudaError.
extern "C" int asv_paged_append_check_log(uint32_t* out) {
  const cudaError_t e = cudaDeviceSynchronize();
  return int(e != cudaSuccess ? e : cudaMemcpyFromSymbol(out, asv::g_check_log, sizeof(asv::g_check_log)));
}
#endif
