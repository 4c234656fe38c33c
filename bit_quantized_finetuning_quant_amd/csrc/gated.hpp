// The gated product h = act(gate) up, shared by the kernels that form it (gfx950).
//
//   silu         act(g) = g sigma(g)
//   gelu (tanh)  act(g) = g (1 + tanh(k (g + c g^3))) / 2 = g sigma(2 k (g + c g^3)),  k = sqrt(2 / pi), c = 0.044715
//
// Both are g sigma(z) with z odd in g.  sigma = 1 / (1 + e^-z) keeps its relative precision on both sides
// (e^-z overflows, and sigma is 0, only where it is below 2^-127); 1 - sigma is the same of -z.
#pragma once

#include <type_traits>

#include "act8.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504f;
constexpr float kGeluTwoK = 1.59576912f, kGeluC = 0.044715f;

template <Activation kAct>
__device__ __forceinline__ float gate_z(float g) {
  return kAct == Activation::kSilu ? g : kGeluTwoK * g * __builtin_fmaf(kGeluC * g, g, 1.0f);
}
__device__ __forceinline__ float sigma(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// act(g); a gate of -inf gives the limit, 0 (the clamp drops a NaN, sigma carries it)
template <Activation kAct>
__device__ __forceinline__ float gate_act(float g) {
  return __builtin_fmaxf(g, -0x1.fffffep127f) * sigma(gate_z<kAct>(g));
}

// act(g) and act'(g) = s + g s (1 - s) z'(g); past |g| = 128 s is 0 or 1 - s is, in fp32, and with it the
// second term, so g is clamped there and z' cannot overflow
template <Activation kAct>
__device__ __forceinline__ void gate_act_slope(float g, float &value, float &slope) {
  const float z = gate_z<kAct>(g), s = sigma(z), t = sigma(-z);
  value = __builtin_fmaxf(g, -0x1.fffffep127f) * s;
  const float c = __builtin_fminf(__builtin_fmaxf(g, -128.f), 128.f);
  const float dz = kAct == Activation::kSilu ? 1.0f : kGeluTwoK * __builtin_fmaf(3.0f * kGeluC * c, c, 1.0f);
  slope = __builtin_fmaf(c * t * dz, s, s);
}

// f(activation) with the activation as a constant
template <typename F>
__host__ __device__ __forceinline__ void with_activation(Activation act, const F &f) {
  if (act == Activation::kSilu)
    f(std::integral_constant<Activation, Activation::kSilu>());
  else
    f(std::integral_constant<Activation, Activation::kGeluTanh>());
}

// Eight neighbouring values of h, gate and up (bf16 pairs) at element `to`; 8 lanes that call this together hold a
// block of the codes.
__device__ __forceinline__ void store_gated(const GatedOut &out, int64_t to, const u32x4 &h, const u32x4 &gate,
                                            const u32x4 &up) {
  if (out.h) *(u32x4 *)(out.h + to) = h;
  if (out.codes) {
    float block;
    const act8_u32x2 c = encode_block(h, block);
    *(act8_u32x2 *)(out.codes + to) = c;
    if ((to & 63) == 0) out.scale[to >> 6] = block;
  }
  if (out.gate) {
    *(u32x4 *)(out.gate + to) = gate;
    *(u32x4 *)(out.up + to) = up;
  }
}

}  // namespace
}  // namespace qlora
