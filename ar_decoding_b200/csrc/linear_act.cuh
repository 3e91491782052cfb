// linear_act.cuh -- the activations of tidar_linear_fused, shared by its kernels.
#pragma once

#include "../../include/tidar.h"

namespace tidar {

// On the fp32 sum (bias added).  v / (1 + exp(-u)) is 0 once exp overflows, v
// once it vanishes; a NaN stays a NaN.
__device__ __forceinline__ float lin_act(float v, int act) {
  switch (act) {
    case TIDAR_ACT_RELU: return v < 0.f ? 0.f : v;
    case TIDAR_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    // 0.5 v (1 + tanh u) = v / (1 + exp(-2u)): no cancellation in the negative tail
    case TIDAR_ACT_GELU_TANH: {
      const float u2 = 1.5957691216057308f * fmaf(0.044715f * v * v, v, v);
      return __fdividef(v, 1.f + __expf(-u2));
    }
    case TIDAR_ACT_SILU: return __fdividef(v, 1.f + __expf(-v));
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
