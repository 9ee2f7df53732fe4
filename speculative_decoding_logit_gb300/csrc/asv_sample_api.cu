// asv_sample_api.cu -- the extern "C" entry point of the token sampling declared in include/asv.h: argument validation
// and dispatch.
#include "asv.h"
#include "asv_internal.h"
#include "asv_paged.h"
#include "asv_sample.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows that are written must not overlap: strides of extents above 1 are positive, and with both the outer one at least
// covers the inner ones.
bool apart(int B, int n, int64_t stride_b, int64_t stride_n, int64_t row) {
  if (n > 1 && stride_n < row) return false;
  return B <= 1 || stride_b >= (n > 1 ? (n - 1) * stride_n + row : row) ||
         (n > 1 && stride_b >= row && stride_n >= (B - 1) * stride_b + row);
}

}  // namespace

extern "C" asv_status sample_tokens(const asv_logits* logits, const asv_field* u, const asv_sampling* params,
                                    const asv_sampling_each* each, const asv_field* out_tokens,
                                    const asv_field* out_logprobs, const asv_field* out_probs, uint32_t* out_req_status,
                                    cudaStream_t stream) {
  if (!logits || !params) return ASV_ERR_NULL;
  const asv_logits& x = *logits;
  const int B = x.B, n = x.n, V = x.V;
  if (B < 0 || n < 0 || V < 1 || V > asv::kSampleMaxVocab || (long long)B * n > 0x7fffffff / 8) return ASV_ERR_SHAPE;
  if ((B > 1 && x.stride_request < 0) || (n > 1 && x.stride_position < 0) || (u && B > 1 && u->stride_request < 0) ||
      (u && n > 1 && u->stride_position < 0))
    return ASV_ERR_SHAPE;
  if ((out_tokens && !apart(B, n, out_tokens->stride_request, out_tokens->stride_position, 1)) ||
      (out_logprobs && !apart(B, n, out_logprobs->stride_request, out_logprobs->stride_position, 1)) ||
      (out_probs && !apart(B, n, out_probs->stride_request, out_probs->stride_position, V)))
    return ASV_ERR_SHAPE;
  if (x.dtype != ASV_F32 && x.dtype != ASV_BF16) return ASV_ERR_DTYPE;
  if (B == 0 || n == 0) return ASV_OK;
  const asv_sampling_each none = {};
  const asv_sampling_each& e = each ? *each : none;
  const asv_sampling& p = *params;
  if (!asv::sampling_ok(e.temperature ? 1.0f : p.temperature, e.top_k ? 0 : p.top_k, e.top_p ? 1.0f : p.top_p,
                        e.min_p ? 0.0f : p.min_p))
    return ASV_ERR_PARAM;
  if (!aligned(x.data, x.dtype == ASV_BF16 ? 2 : 4) || (u && !aligned(u->data, 4)) || !aligned(e.temperature, 4) ||
      !aligned(e.top_k, 4) || !aligned(e.top_p, 4) || !aligned(e.min_p, 4) || (out_tokens && !aligned(out_tokens->data, 4)) ||
      (out_logprobs && !aligned(out_logprobs->data, 4)) || (out_probs && !aligned(out_probs->data, 4)) ||
      !aligned(out_req_status, 4))
    return ASV_ERR_ALIGN;
  if (!x.data || !u || !u->data || !out_tokens || !out_tokens->data || (out_logprobs && !out_logprobs->data) ||
      (out_probs && !out_probs->data) || !out_req_status)
    return ASV_ERR_NULL;
  asv::SampleArgs a = {};
  // (strides of extent 1 may be anything)
  auto by = [](int extent, int64_t stride) { return extent > 1 ? (long long)stride : 0ll; };
  a.x = x.data;
  a.x_b = by(B, x.stride_request);
  a.x_n = by(n, x.stride_position);
  a.B = B;
  a.n = n;
  a.V = V;
  a.u = static_cast<const float*>(u->data);
  a.u_b = by(B, u->stride_request);
  a.u_n = by(n, u->stride_position);
  a.one = p;
  a.temperature = e.temperature;
  a.top_k = e.top_k;
  a.top_p = e.top_p;
  a.min_p = e.min_p;
  a.tokens = static_cast<int32_t*>(out_tokens->data);
  a.tokens_b = by(B, out_tokens->stride_request);
  a.tokens_n = by(n, out_tokens->stride_position);
  if (out_logprobs) {
    a.logprobs = static_cast<float*>(out_logprobs->data);
    a.logprobs_b = by(B, out_logprobs->stride_request);
    a.logprobs_n = by(n, out_logprobs->stride_position);
  }
  if (out_probs) {
    a.probs = static_cast<float*>(out_probs->data);
    a.probs_b = by(B, out_probs->stride_request);
    a.probs_n = by(n, out_probs->stride_position);
  }
  a.status = out_req_status;
  const cudaError_t err = asv::launch_sample(a, x.dtype, stream);
  return err == cudaSuccess ? ASV_OK : asv::record_cuda_error(err);
}
