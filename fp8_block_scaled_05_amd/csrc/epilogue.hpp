// Activations of the linear layer's epilogue, and their derivatives.
//
//   relu  max(z, 0)
//   silu  z sigma(z)
//   gelu  z sigma(2 u), u = c (z + 0.044715 z^3), c = sqrt(2 / pi): the tanh
//         form 0.5 z (1 + tanh u), since 1 + tanh u = 2 sigma(2 u)
// with sigma(x) = 1 / (1 + e^-x).  Derivatives (0 at z = 0 for relu):
//   silu  s + z s (1 - s), s = sigma(z)
//   gelu  s + z s (1 - s) 2 u', s = sigma(2 u), u' = c (1 + 3 * 0.044715 z^2)
#pragma once

#include "device.hpp"
#include "internal.hpp"

namespace fp8bs {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
// |z| past which sigma(2 u) is 0 or 1 in FP32: z is clamped to it inside u, so
// that z^3 stays finite
constexpr float kGeluTop = 20.0f;

// sigma(x) by the hardware exponential and reciprocal (each within 1 ulp; the
// argument's rounding to |x| 2^-24 is what e^-x loses most): below bf16's
// rounding by far for the epilogue's outputs.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == kActRelu) {
    return z > 0.0f || z != z ? z : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    return z * sigmoid_fast(z);
  } else if constexpr (ACT == kActGelu) {
    // e^(-2 u) = 2^(c (k1 + k1 a c^2))
    constexpr float k1 = -2.0f * kGeluC * kLog2e, k3 = k1 * kGeluA;
    const float c = __builtin_amdgcn_fmed3f(z, -kGeluTop, kGeluTop);
    const float e = __builtin_amdgcn_exp2f(c * __builtin_fmaf(c * c, k3, k1));
    return z * __builtin_amdgcn_rcpf(1.0f + e);
  } else {
    return z;
  }
}

// z within [-top, top], NaN as it is (the median of three would drop it).
__device__ __forceinline__ float clamped(float z, float top) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -top), top);
}

// The derivative, in the same arithmetic.  1 - s is taken as e s, with s = 1 / (1
// + e): the difference itself, off by 2^-25 whatever its size, cost the largest
// derivatives two more units of FP32.  z is clamped so that e stays finite, where
// s is below 2^-124 or 1 and the derivative 0 or 1.
template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (ACT == kActRelu) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float c = clamped(z, 87.0f);
    const float e = __builtin_amdgcn_exp2f(c * -kLog2e);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    return __builtin_fmaf(c * s, e * s, s);
  } else if constexpr (ACT == kActGelu) {
    constexpr float k1 = -2.0f * kGeluC * kLog2e, k3 = k1 * kGeluA;
    constexpr float d1 = 2.0f * kGeluC, d3 = 3.0f * d1 * kGeluA;  // 2 u' = d1 + d3 z^2
    const float c = clamped(z, 10.0f);
    const float c2 = c * c;
    const float e = __builtin_amdgcn_exp2f(c * __builtin_fmaf(c2, k3, k1));
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    return __builtin_fmaf(c * s * (e * s), __builtin_fmaf(c2, d3, d1), s);
  } else {
    return 1.0f;
  }
}

// f(std::integral_constant<int, act>) for the runtime act (wave-uniform).
template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default: break;
  }
}

}  // namespace fp8bs
