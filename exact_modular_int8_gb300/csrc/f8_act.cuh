// f8_act.cuh -- activations of the epilogue, and their slopes, in fp32.
//
//   relu(x) = x where x > 0, else 0            slope 1 where x > 0, else 0
//   silu(x) = x / (1 + exp(-x))                s (1 + x (1 - s)), s = 1 / (1 + exp(-x))
//   gelu(x) = x (1 + erf(x / sqrt 2)) / 2      (1 + erf(x / sqrt 2)) / 2 + x exp(-x^2 / 2) / sqrt(2 pi)
//   gelu_tanh(x) = x (1 + tanh u) / 2          s + 2 u' x s (1 - s)
//                = x s, s = 1 / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3)
//
// tanh enters as the logistic function, which loses nothing where 1 + tanh u is
// small.  1 + erf loses there: gelu is off by up to |x| 2^-23 in absolute terms.
// NaN stays NaN; an infinity gives what the formula gives.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rg_common.cuh"

namespace rg {
namespace {

// The quotient to 2 ulp; 0 for a denominator above 2^126, where these quotients are below 2^-100 |x|.
__device__ __forceinline__ float logistic_times(float x, float e) { return __fdividef(x, 1.0f + e); }

constexpr float kSqrt2OverPi = 0.7978845608028654f;

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == RG_ACT_RELU) return x <= 0.0f ? 0.0f : x;
  if constexpr (ACT == RG_ACT_SILU) return logistic_times(x, expf(-x));
  if constexpr (ACT == RG_ACT_GELU) return 0.5f * x * (1.0f + erff(x * 0.7071067811865476f));
  if constexpr (ACT == RG_ACT_GELU_TANH)
    return logistic_times(x, expf(-2.0f * kSqrt2OverPi * fmaf(0.044715f * x * x, x, x)));
  return x;
}
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case RG_ACT_RELU: return activate<RG_ACT_RELU>(x);
    case RG_ACT_SILU: return activate<RG_ACT_SILU>(x);
    case RG_ACT_GELU: return activate<RG_ACT_GELU>(x);
    case RG_ACT_GELU_TANH: return activate<RG_ACT_GELU_TANH>(x);
    default: return x;
  }
}

__device__ __forceinline__ float slope(float x, int act) {
  switch (act) {
    case RG_ACT_RELU: return x <= 0.0f ? 0.0f : x > 0.0f ? 1.0f : x;
    case RG_ACT_SILU: {
      const float s = logistic_times(1.0f, expf(-x));
      return s * fmaf(x, 1.0f - s, 1.0f);
    }
    case RG_ACT_GELU:
      return fmaf(x * 0.3989422804014327f, expf(-0.5f * x * x), 0.5f + 0.5f * erff(x * 0.7071067811865476f));
    case RG_ACT_GELU_TANH: {
      // beyond 30 s is 0 or 1 and the second term 0, which x^2 overflowing would hide
      const float v = x > 30.0f ? 30.0f : x < -30.0f ? -30.0f : x, q = 0.044715f * v * v;
      const float s = logistic_times(1.0f, expf(-2.0f * kSqrt2OverPi * fmaf(q, v, v)));
      return fmaf(2.0f * kSqrt2OverPi * fmaf(3.0f, q, 1.0f) * v, s * (1.0f - s), s);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float load_real(const void* p, int type, long long at) {
  if (type == RG_TYPE_F32) return static_cast<const float*>(p)[at];
  if (type == RG_TYPE_F16) return __half2float(static_cast<const __half*>(p)[at]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void store_real(void* p, int type, long long at, float v) {
  if (type == RG_TYPE_F32) static_cast<float*>(p)[at] = v;
  else if (type == RG_TYPE_F16) static_cast<__half*>(p)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

}  // namespace
}  // namespace rg
