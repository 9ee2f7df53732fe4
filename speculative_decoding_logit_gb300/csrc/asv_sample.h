// asv_sample.h -- host-side declarations of the token sampling.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "asv.h"
#include "asv_internal.h"

namespace asv {

struct SampleArgs {
  const void* x;
  long long x_b, x_n;  // strides in elements, here and below
  int B, n, V;
  const float* u;
  long long u_b, u_n;
  asv_sampling one;          // the parameters of every request that has none of its own
  const float* temperature;  // [B] each; nullptr: `one`'s
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  long long tokens_b, tokens_n;
  float* logprobs;  // nullptr: not wanted, and so probs
  long long logprobs_b, logprobs_n;
  float* probs;
  long long probs_b, probs_n;
  uint32_t* status;
  uint32_t* check_log;  // of the checked build: there is no workspace, its log is the library's
};

// Weights are whole numbers of 2^-44, the largest 1, so a row of 2^19 has a sum below 2^63.
constexpr int kSampleUnitBits = 44;
constexpr int kSampleMaxVocab = 1 << 19;

// What a request's parameters may be (NaN fails every test).
__host__ __device__ inline bool sampling_ok(float temperature, int top_k, float top_p, float min_p) {
  return (temperature == 0.0f || (temperature >= 5.42101086e-20f && temperature <= 1.84467441e19f)) && top_k >= 0 &&
         top_p >= 0.0f && top_p <= 1.0f && min_p >= 0.0f && min_p <= 1.0f;
}

cudaError_t launch_sample(const SampleArgs& a, int dtype, cudaStream_t s);

}  // namespace asv
