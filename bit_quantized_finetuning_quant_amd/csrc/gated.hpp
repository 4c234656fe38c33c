// The gated product h = act(gate) up, shared by the kernels that form it (gfx950).
//
//   silu         act(g) = g sigma(g)
//   gelu (tanh)  act(g) = g (1 + tanh(k (g + c g^3))) / 2 = g sigma(2 k (g + c g^3)),  k = sqrt(2 / pi), c = 0.044715
//
// Both are g sigma(z) with z odd in g.  Of a gate that is given in bf16 (the product alone, its backward pass), with t = e^-|z|
// and r = 1 / (1 + t), sigma and 1 - sigma are r and t r, or t r and r where z < 0: both keep their relative precision on
// both sides (silu: 9 half steps of fp32 with the products; tanh-gelu as much and those of its z, which weigh |z| times).
// A gate that is an fp32 sum is itself off by half a step and more, which moves sigma by |z| of them.  There
// sigma = 1 / (1 + exp2(-z log2 e)), whose rounded argument does as much, in 4 instructions in place of 13: with the others 2048
// tokens of two 11008 x 4096 weights take 356 us for 350, 512 with their codes 129 for 127.5.
#pragma once

#include <type_traits>

#include "act8.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f;  // their sum is log2 e to 2^-50
constexpr float kGeluTwoK = 1.59576912f, kGeluC = 0.044715f;

template <Activation kAct>
__device__ __forceinline__ float gate_z(float g) {
  return kAct == Activation::kSilu ? g : kGeluTwoK * g * __builtin_fmaf(kGeluC * g, g, 1.0f);
}

// sigma(z) and 1 - sigma(z).  v_exp takes the remainder of |z| log2 e, at most 1/2 (of the product itself it would lose |z|
// half steps); past the bound on n, t is 0.
__device__ __forceinline__ void sigma(float z, float &s, float &other) {
  const float a = __builtin_fabsf(z), n = __builtin_fmaxf(__builtin_rintf(a * -kLog2e), -240.f);
  const float f = __builtin_fmaf(a, -kLog2eLow, __builtin_fmaf(a, -kLog2e, -n));
  const float t = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  const float r = __builtin_amdgcn_rcpf(1.0f + t), q = t * r;
  s = z < 0.f ? q : r;
  other = z < 0.f ? r : q;
}

// The same of a gate that is a sum; 0 below 2^-126 (e^-z overflows, or the reciprocal is subnormal).
__device__ __forceinline__ float sigma_of_sum(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// act(g); a gate of -inf gives the limit, 0 (the bound drops a NaN, sigma carries it)
template <Activation kAct>
__device__ __forceinline__ float gate_act(float g) {
  float s, other;
  sigma(gate_z<kAct>(g), s, other);
  return __builtin_fmaxf(g, -0x1.fffffep127f) * s;
}

// The same of a sum.
template <Activation kAct>
__device__ __forceinline__ float gate_act_of_sum(float g) {
  return __builtin_fmaxf(g, -0x1.fffffep127f) * sigma_of_sum(gate_z<kAct>(g));
}

// act(g) and act'(g) = s + g s (1 - s) z'(g); past |g| = 128 s is 0 or 1 - s is, in fp32, and with it the
// second term, so g is clamped there and z' cannot overflow
template <Activation kAct>
__device__ __forceinline__ void gate_act_slope(float g, float &value, float &slope) {
  float s, other;
  sigma(gate_z<kAct>(g), s, other);
  value = __builtin_fmaxf(g, -0x1.fffffep127f) * s;
  const float c = __builtin_fminf(__builtin_fmaxf(g, -128.f), 128.f);
  const float dz = kAct == Activation::kSilu ? 1.0f : kGeluTwoK * __builtin_fmaf(3.0f * kGeluC * c, c, 1.0f);
  slope = __builtin_fmaf(c * other * dz, s, s);
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
