// The activations of a feed-forward block and their derivatives.
#pragma once

#include "device_common.h"

namespace bitnet {

//   silu:  act(g) = g / (1 + e^-g),  act'(g) = t (1 + g (1 - t)), t = 1 / (1 + e^-g)
//   relu2: act(g) = max(g, 0)^2,     act'(g) = 2 max(g, 0)
// The quotient is a reciprocal refined by nothing: v_rcp_f32 is within 1 ulp,
// far below the bf16 rounding of the outputs. It gives 0 where its result would
// be subnormal, and e^-g overflows soon after; so the sum is taken times 2^-8
// and the quotient, which a product may leave subnormal, with it: act(g) is
// right to 2^-17 down to where it is subnormal itself (g = -91.7; without the
// factor everything below -87.3 became 0).

struct ActSilu {
  static __device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(0x1p-8f + __builtin_amdgcn_exp2f(fmaf(g, -1.44269504f, -8.0f))) * 0x1p-8f;
  }
  static __device__ __forceinline__ float f(float g) { return g * sigmoid(g); }
  static __device__ __forceinline__ void fd(float g, float& a, float& da) {
    const float t = sigmoid(g);
    a = g * t;
    da = t + a * (1.0f - t);
  }
};
struct ActRelu2 {
  static __device__ __forceinline__ float f(float g) {
    const float r = g > 0.0f ? g : (g == g ? 0.0f : g);  // a NaN stays one
    return r * r;
  }
  static __device__ __forceinline__ void fd(float g, float& a, float& da) {
    const float r = g > 0.0f ? g : (g == g ? 0.0f : g);
    a = r * r;
    da = 2.0f * r;
  }
};

}  // namespace bitnet
