// Internal structures of include/step.h's operators.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_internal.h"
#include "paged_internal.h"
#include "step.h"

namespace moe {

// ---- RMS norm (norm.cu)
struct NormParams {
  const void *x, *r, *w;
  void *sum, *y;
  float* scales;
  int T, H, d;
  long long x_ts, x_hs, r_ts, r_hs, s_ts, s_hs, y_ts, y_hs;
  int dtype, w_dtype, y_dtype;
  int group;      // of an 8-bit y
  FastDiv div, div_h;  // by group, by H
  float eps, offset, inv_d;
};
constexpr int kNormMaxD = 32768;
cudaError_t launch_norm(const NormParams& p, cudaStream_t st);

// ---- products with 4-bit weights (linear4.cu)
struct Linear4Params {
  const void* x;
  const float* xs;          // 8-bit x: [T][K / xg]
  const uint8_t* codes;
  const uint16_t *scale, *bias;
  void* y;
  long long x_ts, y_ts;
  int x_dtype, y_dtype, bf_scale;
  int T, K, O, group, xg;
};
constexpr int kLinear4MaxK = 36864, kLinear4MaxT = 8 * 65535;
cudaError_t launch_linear4(const Linear4Params& p, cudaStream_t st);

// ---- sampling (sample.cu)
struct SampleParams {
  const void* logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  float all_temperature, all_top_p, all_min_p;  // where there is no array
  int all_top_k;
  int32_t* token;
  float* logprob;
  long long stride;
  int dtype, B, V;
};
constexpr int kSampleMaxV = 360448;
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st);

}  // namespace moe
