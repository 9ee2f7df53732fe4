// asv_paged_device.cuh -- what the paged-cache kernels share: 16-bit element conversions and the
// reading of a request's place in the batch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "asv_device.cuh"
#include "asv_paged.h"

namespace asv {

// Two 16-bit elements of a 32-bit word, widened (exact).
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(bf16_lo(w), bf16_hi(w));
  } else {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
  }
}

// Two fp32 values rounded to nearest into one word, `lo` in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t w;
  if constexpr (BF16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  } else {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  }
  return w;
}

template <bool BF16>
__device__ __forceinline__ float unpack1(uint16_t x) {
  return unpack2<BF16>(uint32_t(x)).x;
}

// Rows [start, end) of request b and the tokens before them.  `ok` is false when the entries are not
// 0 <= start <= end <= N, the length is negative, or the tokens go past position `limit`.
struct Request {
  int start, end, past;
  bool ok;
};

__device__ __forceinline__ Request load_request(const PagedView& c, int b, long long limit) {
  Request r;
  r.start = c.indptr[b];
  r.end = c.indptr[b + 1];
  r.past = c.cache_len[b];
  r.ok = r.start >= 0 && r.start <= r.end && r.end <= c.N && r.past >= 0 &&
         (long long)r.past + (r.end - r.start) <= limit;
  return r;
}

// Positions the block table has pages for.
__device__ __forceinline__ long long table_positions(const PagedView& c) {
  return (long long)c.max_pages * c.page_size;
}

}  // namespace asv
