// Encoding of 8-bit activation checkpoints (gfx950), shared by the kernels that
// write one: the codec itself and the operators whose result is kept in 8 bits.
#pragma once

#include "common.hpp"

namespace qlora {
namespace {

typedef unsigned short act8_u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t act8_u32x2 __attribute__((ext_vector_type(2)));

// max over the 8 lanes of a block
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));      // lane ^ 1
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));      // lane ^ 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // 7 - lane
}

// The codes of 8 values of a block with the largest magnitude c1 (finite, > 0): the quotients Q = 127 x / c1
// rounded to the nearest integer, ties to the even one.  x and c1 have 8 significant bits, so Q either is
// a multiple of 1/2 or differs from every odd one by at least Q / (127 255), 259 units of its last place.
// q = x (127 / c1) is within 4 of them; rounded to 18 significant bits (by up to 32) it is a tie where Q is
// one, and on Q's side otherwise.  Adding 1.5 2^23 rounds that to the integer, which is then the low byte.
__device__ __forceinline__ act8_u32x2 encode(u32x4 x, float c1) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = x[i];
    v[2 * i] = bf16_lo(pair);
    v[2 * i + 1] = bf16_hi(pair);
  }
  if (c1 < 0x1p-100f || c1 > 0x1p100f) {  // 127 / c1 or 1 / c1 would leave the range
    const float lift = c1 < 1.0f ? 0x1p64f : 0x1p-64f;
    c1 *= lift;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= lift;
  }
  const float inv = 127.0f * __builtin_amdgcn_rcpf(c1);
  uint32_t n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t q = (__float_as_uint(v[i] * inv) + 32u) & ~63u;
    n[i] = __float_as_uint(__uint_as_float(q) + 12582912.0f);
  }
  act8_u32x2 out;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t lo = __builtin_amdgcn_perm(n[4 * w + 1], n[4 * w], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(n[4 * w + 3], n[4 * w + 2], 0x04000C0Cu);
    out[w] = lo | hi;
  }
  return out;
}

// fl32(c1 / 127) of a bf16 c1 >= 0: the product with fl32(1 / 127), corrected by its remainder (right for all 128
// significands; below 2^-100, where the remainder would be subnormal, the division itself).
__device__ __forceinline__ float block_scale(float c1) {
  if (c1 < 0x1p-100f) return c1 / 127.0f;
  const float r = 1.0f / 127.0f, q = c1 * r;
  return __builtin_fmaf(__builtin_fmaf(-q, 127.0f, c1), r, q);
}

// One lane's eighth of a block: the codes of its 8 values, and the block's scale (the same in its 8 lanes,
// which all call this together).  A block with a NaN or Inf has codes 0 and a NaN scale.
__device__ __forceinline__ act8_u32x2 encode_block(u32x4 v, float &scale) {
  act8_u16x2 m = {0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t a = v[w] & 0x7FFF7FFFu;
    m = __builtin_elementwise_max(m, __builtin_bit_cast(act8_u16x2, a));
  }
  const uint32_t top = block_max(max((uint32_t)m[0], (uint32_t)m[1]));
  const float c1 = __uint_as_float(top << 16);
  const bool finite = top < 0x7F80u;
  act8_u32x2 c = {0u, 0u};
  if (finite && top != 0u) c = encode(v, c1);
  scale = finite ? block_scale(c1) : __uint_as_float(0x7FC00000u);
  return c;
}

}  // namespace
}  // namespace qlora
