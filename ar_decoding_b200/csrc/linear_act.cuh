// linear_act.cuh -- the activations of tidar_linear_fused, shared by its kernels.
#pragma once

#include "../../include/tidar.h"
#include "sm100.cuh"

namespace tidar {

// v Phi(v), Phi the normal distribution function (0.5 (1 + erf(v / sqrt 2)), without
// that sum's cancellation in the negative tail: 1 + erff has one digit left at v = -5 and
// none below -5.6).  Phi(-t) = exp(-t^2 / 2) G(t) for t >= 0, and G(t) = erfcx(t / sqrt 2)
// / 2 falls slowly, like 1 / t: a polynomial in s = 1 / (1 + t / 3.4), fitted by least
// squares to the smallest relative error on 0 <= t <= 13.6 (3.6e-8; Phi(-13.6) is below
// bf16's range).  The result is off by 5e-7 of itself for |v| < 1, 3e-6 down to -8 and
// 8e-6 to -13 (the exponent's rounding).  1024 x 4096 x 4096: 33.0 us with erff, 32.4 with
// this, 35.6 with erfcf.
__device__ __forceinline__ float lin_gelu(float v) {
  const float t = fabsf(v), s = __fdividef(1.f, fmaf(t, 1.f / 3.4f, 1.f));
  float g = 0.039509729f;
  g = fmaf(g, s, -0.185585514f);
  g = fmaf(g, s, 0.278201669f);
  g = fmaf(g, s, -0.124241441f);
  g = fmaf(g, s, 0.170618534f);
  g = fmaf(g, s, 0.0828891173f);
  g = fmaf(g, s, 0.121692568f);
  g = fmaf(g, s, 0.116896264f);
  g = fmaf(g, s, 1.90702776e-5f);
  const float q = g * __expf(-0.5f * t * t);
  return v * (v < 0.f ? q : 1.f - q);
}

// v / (1 + 2^z), as 2^-16 v / (2^-16 + 2^(z - 16)): __fdividef is 0 past a denominator of
// 2^126, and v 2^-z is a bf16 number up to z = 140 (below |v| = 2^-110 the product's own
// rounding adds 2^-134).
__device__ __forceinline__ float lin_sigmoid(float v, float z16) {
  return __fdividef(v * 0x1p-16f, 0x1p-16f + ex2(z16));
}

// On the fp32 sum (bias added); a NaN stays a NaN.
__device__ __forceinline__ float lin_act(float v, int act) {
  switch (act) {
    case TIDAR_ACT_RELU: return v < 0.f ? 0.f : v;
    case TIDAR_ACT_GELU: return lin_gelu(v);
    // 0.5 v (1 + tanh u) = v / (1 + exp(-2u)): no cancellation in the negative tail
    case TIDAR_ACT_GELU_TANH:
      return lin_sigmoid(v, fmaf(fmaf(0.044715f * v * v, v, v), -2.3022082f, -16.f));   // sqrt(8 / pi) log2 e
    case TIDAR_ACT_SILU: return lin_sigmoid(v, fmaf(v, -1.4426950408889634f, -16.f));
  }
  return v;
}

// Four of them, as a call, where a thread's epilogue is short: code that an SM
// fetches for the first time costs about a nanosecond an instruction (272 x 4096 x
// 4096 17.6 us with the activations inlined, 16.8 with calls; over the hundreds of
// values a thread of the paired tiles has, inlined 15.2 and called 18.9 us).
static __device__ __noinline__ float4 lin_act4(float4 v, int act) {
  return make_float4(lin_act(v.x, act), lin_act(v.y, act), lin_act(v.z, act), lin_act(v.w, act));
}

}  // namespace tidar
