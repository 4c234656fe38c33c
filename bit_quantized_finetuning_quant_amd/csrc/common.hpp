// Shared device helpers of the gfx950 QLoRA kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

constexpr int kBlock = 64;   // elements per NF4 block (one absmax constant each)
constexpr int kGroup = 256;  // block constants per FP8 double-quantization group
constexpr uint32_t kZeroCode = 7;

// Kernel-argument copy of the 16 NF4 levels (held in SGPRs by the kernels that
// take it, copied to LDS where a per-lane lookup is needed).
struct Codebook {
  float v[16];
};

// Exact midpoints between adjacent NF4 levels (each needs at most 26
// significant bits, so it is exact in fp64).  Used by the quantizer to build
// its per-block thresholds.
struct Midpoints {
  double m[15];
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// e4m3 ("fn") byte -> its exact value (bias 7, 3 mantissa bits, exponent
// field 0 = subnormal m * 2^-9; 0x7F and 0xFF are NaN, which stored data
// never holds).  gfx950's v_cvt_f32_fp8 reads the OCP e4m3 format; every
// e4m3 value is an fp32 value, so the conversion is exact.
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) { return __builtin_amdgcn_cvt_f32_fp8((int)b, 0); }

// Block constant decode: fl32(fl32(e4m3(q) * s2) + mu), two roundings.  The
// multiply and the add must not be contracted into one fused multiply-add
// (HIP's __fmul_rn / __fadd_rn are plain operators, so the pragma is what
// keeps them apart; the library is also built with -ffp-contract=off).
__device__ __forceinline__ float decode_constant(uint32_t q, float s2, float mu) {
#pragma clang fp contract(off)
  const float p = e4m3_to_f32(q) * s2;
  return p + mu;
}

// One decoded weight before the bf16 rounding: fl32(CB[code] * c1hat).
__device__ __forceinline__ float decode_product(float level, float c1hat) {
#pragma clang fp contract(off)
  return level * c1hat;
}

// Two fp32 -> packed bf16 pair (round to nearest even; gfx950 v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// Decode without a memory lookup.  The 16 decoded values of one block,
// t[k] = bf16_rne(fl32(CB[k] * c1hat)), are held in registers as byte
// tables: lo[j] holds the low bytes of t[4j .. 4j+3], hi[j] the high bytes.
// A code then selects its two bytes with v_perm_b32 (which picks bytes 0..7
// of the 64-bit pair {S0, S1}, S1 the low word): one permute over each half
// of a table and a per-byte select on the code's bit 3.  Every decoded value
// is computed exactly as in the lookup form, so the two are bit-identical.
struct DecodeTable {
  uint32_t lo[4], hi[4];
};

// lo[j] and hi[j] of 8 consecutive levels from their 4 packed bf16 pairs
// p[m] = t[2m] | t[2m+1] << 16.
__device__ __forceinline__ void table_half(const uint32_t (&p)[4], uint32_t (&lo)[2], uint32_t (&hi)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    lo[j] = __builtin_amdgcn_perm(p[2 * j + 1], p[2 * j], 0x06040200u);
    hi[j] = __builtin_amdgcn_perm(p[2 * j + 1], p[2 * j], 0x07050301u);
  }
}

// Byte b of the result is byte (code_b) of a 16-byte table, for four codes
// given as the bytes of sel (low 3 bits) and mask (0xFF where the code's bit 3
// is set).
__device__ __forceinline__ uint32_t table_bytes(const uint32_t (&tb)[4], uint32_t sel, uint32_t mask) {
  const uint32_t a = __builtin_amdgcn_perm(tb[1], tb[0], sel), b = __builtin_amdgcn_perm(tb[3], tb[2], sel);
  return (b & mask) | (a & ~mask);
}

// One word of 8 codes (low nibble first) -> 4 words of bf16 pairs; word d
// holds element 2d in its low half and element 2d + 1 in its high half.
__device__ __forceinline__ void decode_word(uint32_t c, const DecodeTable &t, uint32_t (&o)[4]) {
  const uint32_t c4 = c >> 4;
  // bytes of c: even codes n0, n2, n4, n6 in bits 0..3; bytes of c4: odd codes
  const uint32_t se = c & 0x07070707u, so = c4 & 0x07070707u;
  // 0xFF in byte b where bit 3 of code b is set: v_perm selectors 8..11 give 0xFF or 0x00 from the
  // top bit of bytes 1, 3, 5, 7 of {S0, S1}; the shifts bring bit 3 (even codes) or bit 7 (odd
  // codes) of byte b there
  const uint32_t me = __builtin_amdgcn_perm(c << 4, c << 12, 0x0B090A08u);
  const uint32_t mo = __builtin_amdgcn_perm(c, c << 8, 0x0B090A08u);
  const uint32_t le = table_bytes(t.lo, se, me), he = table_bytes(t.hi, se, me);
  const uint32_t lq = table_bytes(t.lo, so, mo), hq = table_bytes(t.hi, so, mo);
  const uint32_t x0 = __builtin_amdgcn_perm(he, le, 0x05010400u);  // t[n0] | t[n2] << 16
  const uint32_t y0 = __builtin_amdgcn_perm(hq, lq, 0x05010400u);  // t[n1] | t[n3] << 16
  const uint32_t x1 = __builtin_amdgcn_perm(he, le, 0x07030602u);  // t[n4] | t[n6] << 16
  const uint32_t y1 = __builtin_amdgcn_perm(hq, lq, 0x07030602u);  // t[n5] | t[n7] << 16
  o[0] = __builtin_amdgcn_perm(y0, x0, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(y0, x0, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(y1, x1, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(y1, x1, 0x07060302u);
}

__device__ __forceinline__ float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// Eight codes of an 8-bit activation checkpoint (two words, low byte first) -> x_hat = bf16(fl32(code
// scale)), four words of bf16 pairs.  A code is read as an unsigned byte 128 above it (v_cvt_f32_ubyte).
__device__ __forceinline__ u32x4 act8_values(uint32_t c0, uint32_t c1, float scale) {
  u32x4 out;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t u = (w ? c1 : c0) ^ 0x80808080u;
    const float f0 = ((float)(u & 255u) - 128.0f) * scale, f1 = ((float)((u >> 8) & 255u) - 128.0f) * scale;
    const float f2 = ((float)((u >> 16) & 255u) - 128.0f) * scale, f3 = ((float)(u >> 24) - 128.0f) * scale;
    out[2 * w] = pack_bf16x2(f0, f1);
    out[2 * w + 1] = pack_bf16x2(f2, f3);
  }
  return out;
}

// Eight 16-bit values from any 2-byte aligned address in one 16-byte load.
__device__ __forceinline__ u32x4 load8(const uint16_t *p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Eight aligned 16-bit values; kStream: past the caches, for data that is read once and is not in them.
template <bool kStream>
__device__ __forceinline__ u32x4 load_run(const uint16_t *p) {
  if constexpr (kStream) return __builtin_nontemporal_load((const u32x4 *)p);
  return *(const u32x4 *)p;
}

// Inputs of this many bytes are read so: less may still lie in the 256 MB last-level cache, where the kernel before
// has just written it.  (Root-mean-square norm backward, 201 MB read: 57.5 -> 45.3 us, 50 MB: 12.3 -> 12.7; gated product
// of 361 MB: 100.6 -> 80.6 us, of 90 MB even.)
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

// s_waitcnt immediate (gfx9 encoding): vmcnt in bits 3:0 and 15:14, expcnt in
// 6:4 (left at its maximum), lgkmcnt in 11:8.
constexpr int waitcnt_imm(int vm, int lgkm) { return (vm & 15) | (7 << 4) | ((lgkm & 15) << 8) | ((vm >> 4) << 14); }

typedef __attribute__((address_space(3))) void lds_void_t;

// The LDS byte address of a pointer into LDS.
__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)(lds_void_t *)p; }

// One 16-byte-per-lane LDS-DMA: lane l reads 16 bytes at sbase + voff and
// writes them at LDS byte address lds + 16 l.  Written as inline asm so that
// the compiler does not treat the whole LDS as possibly being written by it:
// the builtin makes every later LDS read of the wave wait for all outstanding
// loads, including stages that are meant to stay in flight.  The instruction
// has no register result; its waits are issued explicitly by the caller, and
// voff must stay unmodified until they have been.
// m0 is named as clobbered: nothing else in these kernels uses it (checked in
// the generated code), and every DMA sets it right before use.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const char *sbase, uint32_t voff, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(voff), "s"(sbase), "s"(lds)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// Sums over lanes without LDS.
// Lanes 0..31 (or even rows of 16) the sum of a and its other half (row), the others that of b.
template <int kLanes>
__device__ __forceinline__ float fold(float a, float b) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  const auto r = kLanes == 32 ? __builtin_amdgcn_permlane32_swap(x, y, false, false)
                              : __builtin_amdgcn_permlane16_swap(x, y, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The value kBy lanes away in the row of 16.
template <int kBy>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + kBy, 0xF, 0xF, true));
}

// The sum of the row of 16, in all of its lanes.
__device__ __forceinline__ float row16_sum(float v) {
  v += rotated<8>(v);
  v += rotated<4>(v);
  v += rotated<2>(v);
  return v + rotated<1>(v);
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

}  // namespace qlora
