// The gate of a feed-forward block, silu(g) * u with silu(g) = g / (1 + e^-g),
// and its derivatives.
#pragma once

#include <hip/hip_runtime.h>

namespace qnf4 {

// 1 / (1 + e^-g) in fp32. The exponential and the reciprocal are the
// hardware's, within 1 ulp; e^-g past the largest fp32 makes the result the
// zero that it is next to.
__device__ __forceinline__ float gate_sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

__device__ __forceinline__ float gate_value(float g, float u) { return g * gate_sigmoid(g) * u; }

// (dg, du) from the gradient of h = silu(g) u.
__device__ __forceinline__ void gate_backward(float dh, float g, float u, float &dg, float &du) {
  const float s = gate_sigmoid(g);
  du = dh * (g * s);
  dg = dh * u * (s * (1.0f + g * (1.0f - s)));
}

}  // namespace qnf4
