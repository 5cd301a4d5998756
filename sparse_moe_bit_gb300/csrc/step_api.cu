// C ABI of include/step.h: argument checks, launches on the caller's stream.
#include <cmath>

#include "paged_internal.h"
#include "step_internal.h"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define STEP_CK(call, what)                                                \
  do {                                                                     \
    const cudaError_t e_ = (call);                                         \
    if (e_ != cudaSuccess)                                                 \
      return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_));   \
  } while (0)

int size_of(int dtype) {
  switch (dtype) {
    case STEP_BF16: case STEP_F16: return 2;
    case STEP_F32: return 4;
    case STEP_E4M3: case STEP_I8: return 1;
  }
  return 0;
}
bool is8(int dtype) { return dtype == STEP_E4M3 || dtype == STEP_I8; }
bool is_float(int dtype) { return dtype >= STEP_BF16 && dtype <= STEP_F32; }
// whether n rows of `width` elements, `stride` apart, write over one another
bool overlap(int n, int64_t stride, int width) { return n > 1 && stride < width && stride > -(int64_t)width; }

}  // namespace

extern "C" {

moe_status rms_norm(const void* x, int dtype, int T, int H, int d, int64_t x_ts, int64_t x_hs,
                    const void* residual, int64_t r_ts, int64_t r_hs, void* sum, int64_t s_ts,
                    int64_t s_hs, const void* weight, int weight_dtype, int unit_offset, float eps,
                    void* y, int y_dtype, int64_t y_ts, int64_t y_hs, float* scales, int group,
                    void* stream) {
  if (!is_float(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype %d", dtype);
  if (!size_of(y_dtype)) return fail(MOE_ERR_INVALID_ARG, "y_dtype %d", y_dtype);
  if (weight && weight_dtype != dtype && weight_dtype != STEP_F32)
    return fail(MOE_ERR_INVALID_ARG, "weight_dtype %d", weight_dtype);
  if (!weight && unit_offset) return fail(MOE_ERR_INVALID_ARG, "unit_offset without a weight");
  if (T < 0 || H < 1 || d < 1) return fail(MOE_ERR_INVALID_ARG, "bad size (T=%d H=%d d=%d)", T, H, d);
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (is8(y_dtype) ? group < 0 || (group > 0 && d % group) : group != 0)
    return fail(MOE_ERR_INVALID_ARG, "group of %d in rows of %d", group, d);
  if (!residual != !sum) return fail(MOE_ERR_INVALID_ARG, "residual and sum come together");
  if (d > kNormMaxD) return fail(MOE_ERR_UNSUPPORTED, "d above %d", kNormMaxD);
  if ((long long)T * H >= (1ll << 31) - 4) return fail(MOE_ERR_UNSUPPORTED, "T * H = %lld", (long long)T * H);
  if (T == 0) return MOE_OK;
  if (!x || !y || (is8(y_dtype) != (scales != nullptr)))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor, or scales without an 8-bit y");
  const int es = size_of(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(sum, es) || !aligned(y, size_of(y_dtype)) ||
      !aligned(scales, 4) || (weight && !aligned(weight, size_of(weight_dtype))))
    return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (y == x && (y_dtype != dtype || y_ts != x_ts || y_hs != x_hs || sum == x))
    return fail(MOE_ERR_INVALID_ARG, "y in place with another type or strides, or beside sum");
  if (sum && (y == sum || y == residual || (sum == x && (s_ts != x_ts || s_hs != x_hs)) ||
              (sum == residual && (s_ts != r_ts || s_hs != r_hs))))
    return fail(MOE_ERR_INVALID_ARG, "sum in place with other strides, or y over it");
  if (overlap(T, y_ts, d) || overlap(H, y_hs, d) || (sum && (overlap(T, s_ts, d) || overlap(H, s_hs, d))))
    return fail(MOE_ERR_INVALID_ARG, "rows of y or sum overlap");
  NormParams p{};
  p.x = x;
  p.r = residual;
  p.w = weight;
  p.sum = sum;
  p.y = y;
  p.scales = scales;
  p.T = T;
  p.H = H;
  p.d = d;
  p.x_ts = x_ts, p.x_hs = x_hs, p.r_ts = r_ts, p.r_hs = r_hs;
  p.s_ts = s_ts, p.s_hs = s_hs, p.y_ts = y_ts, p.y_hs = y_hs;
  p.dtype = dtype;
  p.w_dtype = weight_dtype;
  p.y_dtype = y_dtype;
  p.group = group ? group : d;
  p.div = make_fastdiv(p.group);
  p.div_h = make_fastdiv(H);
  p.eps = eps;
  p.offset = unit_offset ? 1.f : 0.f;
  p.inv_d = 1.f / (float)d;
  STEP_CK(launch_norm(p, static_cast<cudaStream_t>(stream)), "rms_norm launch");
  return MOE_OK;
}

moe_status linear4(const void* x, int x_dtype, int T, int K, int64_t x_ts, const float* x_scale,
                   int x_group, const void* codes, const void* scale, const void* bias,
                   int scale_dtype, int O, int group, void* y, int y_dtype, int64_t y_ts,
                   void* stream) {
  if (x_dtype != STEP_BF16 && x_dtype != STEP_F16 && !is8(x_dtype))
    return fail(MOE_ERR_INVALID_ARG, "x_dtype %d", x_dtype);
  if (!is_float(y_dtype)) return fail(MOE_ERR_INVALID_ARG, "y_dtype %d", y_dtype);
  if (scale_dtype != MOE_SCALE_F16 && scale_dtype != MOE_SCALE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "scale_dtype %d", scale_dtype);
  if (T < 0 || K < 1 || O < 1) return fail(MOE_ERR_INVALID_ARG, "bad size (T=%d K=%d O=%d)", T, K, O);
  if (group < 1 || K % group) return fail(MOE_ERR_INVALID_ARG, "group of %d in K=%d", group, K);
  if (x_group < 0 || (x_group > 0 && K % x_group) || (!is8(x_dtype) && x_group != 0))
    return fail(MOE_ERR_INVALID_ARG, "x_group of %d in K=%d", x_group, K);
  if (group % 64) return fail(MOE_ERR_UNSUPPORTED, "group of %d (a multiple of 64 is supported)", group);
  if (x_group > 0 && x_group != K && x_group % 64)
    return fail(MOE_ERR_UNSUPPORTED, "x_group of %d (a multiple of 64 is supported)", x_group);
  if (K > kLinear4MaxK) return fail(MOE_ERR_UNSUPPORTED, "K above %d", kLinear4MaxK);
  if (O > (1 << 30) || T > kLinear4MaxT)
    return fail(MOE_ERR_UNSUPPORTED, "O above 2^30 or T above %d", kLinear4MaxT);
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scale || !bias || !y || is8(x_dtype) != (x_scale != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor, or x_scale without an 8-bit x");
  if (!aligned(x, 16) || x_ts * size_of(x_dtype) % 16)
    return fail(MOE_ERR_INVALID_ARG, "rows of x must be 16-byte aligned");
  if (!aligned(codes, 16) || !aligned(scale, 16) || !aligned(bias, 16) || !aligned(x_scale, 4) ||
      !aligned(y, size_of(y_dtype)))
    return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (overlap(T, y_ts, O)) return fail(MOE_ERR_INVALID_ARG, "rows of y overlap");
  Linear4Params p{};
  p.x = x;
  p.xs = x_scale;
  p.codes = static_cast<const uint8_t*>(codes);
  p.scale = static_cast<const uint16_t*>(scale);
  p.bias = static_cast<const uint16_t*>(bias);
  p.y = y;
  p.x_ts = x_ts;
  p.y_ts = y_ts;
  p.x_dtype = x_dtype;
  p.y_dtype = y_dtype;
  p.bf_scale = scale_dtype == MOE_SCALE_BF16;
  p.T = T;
  p.K = K;
  p.O = O;
  p.group = group;
  p.xg = x_group ? x_group : K;
  STEP_CK(launch_linear4(p, static_cast<cudaStream_t>(stream)), "linear4 launch");
  return MOE_OK;
}

moe_status sample(const void* logits, int dtype, int B, int V, int64_t stride, const float* u,
                  const float* temperature, const int32_t* top_k, const float* top_p,
                  const float* min_p, float all_temperature, int all_top_k, float all_top_p,
                  float all_min_p, int32_t* token, float* logprob, void* cuda_stream) {
  if (!is_float(dtype)) return fail(MOE_ERR_INVALID_ARG, "dtype %d", dtype);
  if (B < 0 || V < 1) return fail(MOE_ERR_INVALID_ARG, "bad size (B=%d V=%d)", B, V);
  if (V > kSampleMaxV || B > (1 << 27)) return fail(MOE_ERR_UNSUPPORTED, "B=%d, V=%d (V up to %d)", B, V, kSampleMaxV);
  if (B == 0) return MOE_OK;
  if (!logits || !u || !token) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned(logits, size_of(dtype)) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 4) || !aligned(logprob, 4))
    return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
  SampleParams p{};
  p.logits = logits;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.all_temperature = all_temperature;
  p.all_top_k = all_top_k;
  p.all_top_p = all_top_p;
  p.all_min_p = all_min_p;
  p.token = token;
  p.logprob = logprob;
  p.stride = stride;
  p.dtype = dtype;
  p.B = B;
  p.V = V;
  STEP_CK(launch_sample(p, static_cast<cudaStream_t>(cuda_stream)), "sample launch");
  return MOE_OK;
}

}  // extern "C"
