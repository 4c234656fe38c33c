// The gated product h = act(gate) up, shared by the kernels that form it (gfx950).
//
//   silu         act(g) = g sigma(g)
//   gelu (tanh)  act(g) = g (1 + tanh(k (g + c g^3))) / 2 = g sigma(2 k (g + c g^3)),  k = sqrt(2 / pi), c = 0.044715
//
// Both are g sigma(z) with z odd in g, so sigma comes from e = exp(-|z|): 1 / (1 + e) on the side of
// its sign and e / (1 + e) on the other, neither of which loses digits or overflows anywhere.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504f;
constexpr float kGeluTwoK = 1.59576912f, kGeluC = 0.044715f;

// sigma(z(g)) and 1 - sigma
__device__ __forceinline__ void gate_sigma(float g, Activation act, float &s, float &t) {
  float z = g;
  if (act == Activation::kGeluTanh) z = kGeluTwoK * g * __builtin_fmaf(kGeluC * g, g, 1.0f);
  const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(z) * kLog2e), q = __builtin_amdgcn_rcpf(1.0f + e);
  s = z < 0.f ? e * q : q;
  t = z < 0.f ? q : e * q;
}

// act(g); a gate of -inf gives the limit, 0 (the clamp drops a NaN, s carries it)
__device__ __forceinline__ float gate_act(float g, Activation act) {
  float s, t;
  gate_sigma(g, act, s, t);
  return __builtin_fmaxf(g, -0x1.fffffep127f) * s;
}

// act(g) and act'(g) = s + g s (1 - s) z'(g); past |g| = 128 s is 0 or 1 - s is, in fp32, and with it the
// second term, so g is clamped there and z' cannot overflow
__device__ __forceinline__ void gate_act_slope(float g, Activation act, float &value, float &slope) {
  float s, t;
  gate_sigma(g, act, s, t);
  value = __builtin_fmaxf(g, -0x1.fffffep127f) * s;
  const float c = __builtin_fminf(__builtin_fmaxf(g, -128.f), 128.f);
  float dz = 1.0f;
  if (act == Activation::kGeluTanh) dz = kGeluTwoK * __builtin_fmaf(3.0f * kGeluC * c, c, 1.0f);
  slope = __builtin_fmaf(c * t * dz, s, s);
}

}  // namespace
}  // namespace qlora
