// f8_act.cuh -- activations of the epilogue, and their slopes, in fp32.
//
//   relu(x) = x where x > 0, else 0            slope 1 where x > 0, else 0
//   silu(x) = x / (1 + exp(-x))                s (1 + x (1 - s)), s = 1 / (1 + exp(-x))
//   gelu(x) = x (1 + erf(x / sqrt 2)) / 2      (1 + erf(x / sqrt 2)) / 2 + x exp(-x^2 / 2) / sqrt(2 pi)
//   gelu_tanh(x) = x (1 + tanh u) / 2          s + 2 u' x s (1 - s)
//                = x s, s = 1 / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3)
//
// A few operations each, since a tile's epilogue and the quantisation of a gradient
// are bound by their instructions and the code of an activation stands 128 times in
// the pair kernel.  tanh enters as the logistic function, which loses nothing where 1
// + tanh u is small.  Exponentials and reciprocals are the hardware's approximations
// (2^-22 and 2^-23 of themselves; an exponential another |argument| 2^-24 for the
// rounding of its argument, where it hardly counts).  erf is Abramowitz and
// Stegun's 7.1.26, off by 1.5 10^-7, with its exp(-x^2 / 2) shared by the slope.  These
// bounds add up to at most |x| 2^-20 in absolute terms; measured over [-30, 30], gelu
// is off by up to |x| 2^-21.5, silu and gelu_tanh by |x| 2^-22.5.  NaN stays NaN; an
// infinity gives what the formula gives, and to a slope its limit (0 or 1).
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rg_common.cuh"

namespace rg {
namespace {

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kSqrt2OverPi = 0.7978845608028654f;

// 1 / (1 + 2^a)
__device__ __forceinline__ float logistic2(float a) { return rcp_fast(1.0f + exp2_fast(a)); }
// gelu_tanh's 1 / (1 + exp(-2 u)), and u' over sqrt(2 / pi)
__device__ __forceinline__ float tanh_logistic(float x, float x2) {
  return logistic2(x * fmaf(x2, -2.0f * kLog2E * kSqrt2OverPi * 0.044715f, -2.0f * kLog2E * kSqrt2OverPi));
}

// (1 + erf(x / sqrt 2)) / 2, given e = exp(-x^2 / 2).
__device__ __forceinline__ float normal_cdf(float x, float e) {
  const float t = rcp_fast(fmaf(fabsf(x), 0.3275911f * 0.7071067811865476f, 1.0f));
  float q = fmaf(t, 0.5f * 1.061405429f, -0.5f * 1.453152027f);
  q = fmaf(q, t, 0.5f * 1.421413741f);
  q = fmaf(q, t, -0.5f * 0.284496736f);
  q = fmaf(q, t, 0.5f * 0.254829592f);
  // (a choice of the sign by comparison spilled registers in the pair kernel's epilogue)
  return 0.5f + copysignf(fmaf(-q * t, e, 0.5f), x);
}
__device__ __forceinline__ float exp_half_square(float x) { return exp2_fast(x * (-0.5f * kLog2E * x)); }

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == RG_ACT_RELU) return x <= 0.0f ? 0.0f : x;
  if constexpr (ACT == RG_ACT_SILU) return x * logistic2(-kLog2E * x);
  if constexpr (ACT == RG_ACT_GELU) return x * normal_cdf(x, exp_half_square(x));
  if constexpr (ACT == RG_ACT_GELU_TANH) return x * tanh_logistic(x, x * x);
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

// x held to [-top, top]; a NaN stays one.
__device__ __forceinline__ float held(float x, float top) { return x > top ? top : x < -top ? -top : x; }

// Far out a slope is 0 or 1, and the product of x with what is 0 there exactly is
// taken at a finite x: an infinity is an ordinary value here, since what is kept for
// the slope is rounded to 16 bits (fp16: beyond 65504).
template <int ACT>
__device__ __forceinline__ float slope(float x) {
  if constexpr (ACT == RG_ACT_RELU) return x <= 0.0f ? 0.0f : x > 0.0f ? 1.0f : x;
  if constexpr (ACT == RG_ACT_SILU) {
    // beyond 128: 1 + exp(x) overflows and s is 0, or exp(-x) is below 2^-126 and s is 1
    const float v = held(x, 128.0f), s = logistic2(-kLog2E * v);
    return s * fmaf(v, 1.0f - s, 1.0f);
  }
  if constexpr (ACT == RG_ACT_GELU) {
    // beyond 16 e is 0: exp(-128) is below 2^-126
    const float v = held(x, 16.0f), e = exp_half_square(v);
    return fmaf(v * 0.3989422804014327f, e, normal_cdf(v, e));
  }
  if constexpr (ACT == RG_ACT_GELU_TANH) {
    // beyond 30 s is 0 or 1 and the second term 0, which x^2 overflowing would hide
    const float v = held(x, 30.0f), v2 = v * v;
    const float s = tanh_logistic(v, v2);
    return fmaf(v * fmaf(v2, 6.0f * kSqrt2OverPi * 0.044715f, 2.0f * kSqrt2OverPi), s * (1.0f - s), s);
  }
  return 1.0f;
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
