// Matrix products of bf16 operands on 256 x 256 tiles (many tokens) and on
// per-wave 64-row streams (up to 64 tokens), shared by the kernels of the head's
// loss and of the ragged backward pass (gfx950).
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace qlora {
namespace {

constexpr int kTileV = 256;    // rows or columns of the left operand of a workgroup's tile
constexpr int kTileT = 256;    // tokens of a workgroup's tile
constexpr int kStep = 64;      // contraction step
constexpr int kThreads = 512;  // eight waves: 2 along the words or columns, 4 along the tokens
constexpr int kUnit = 16384;   // bytes of half an operand tile of a step: 128 rows of 128 bytes
constexpr int kStage = 4 * kUnit;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));

#define TILE_WAIT_VM(n) asm volatile("s_waitcnt vmcnt(" #n ")" ::: "memory")
#define TILE_WAIT_LDS() asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory")

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// A pointer that is the same in every lane, moved to scalar registers.
__device__ __forceinline__ const char *uniform(const void *p) {
  const uint64_t a = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return (const char *)(((uint64_t)hi << 32) | lo);
}

// LDS layout of an operand tile: rows of 128 bytes, eight 16-byte chunks each, chunk c of row r at
// position c ^ swizzle(r).  The LDS serves 16-byte reads of 16 lanes at a time from 64 banks (two
// rows), so row pairs shift the chunks; the transpose reads take 32-byte pieces of rows r..r+3 and
// r + 8..r + 11 (or + 16), which then fall on different banks too.
__device__ __forceinline__ int swizzle_rows(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int swizzle_cols(int r) { return (((r >> 1) & 1) | ((((r >> 3) ^ (r >> 4)) & 1) << 1)) << 1; }

// The product shared by both matrix kernels: acc[m][t] over a contraction of `steps` steps of 64.
// Left operand: 256 rows of a row-major matrix whose contraction index is contiguous (kTrans =
// false), or 256 columns of one whose rows are the contraction (kTrans = true).  Right operand: 256 rows (tokens).
//
// Two groups of four waves (one wave of each per SIMD) run half a phase apart: while one group
// multiplies (16 MFMAs a wave), the other reads its next fragments from LDS and starts the copies
// that refill it.  A step has four phases, (rows 0..63 of the wave's 128, contraction 0..31), (0..63,
// 32..63), (64..127, 0..31), (64..127, 32..63); the tokens' fragments are read in the first two.  A
// stage's tokens and first rows are free after phase 1, its other rows after phase 3, so each is
// refilled for step k + 2 at once, five to six phases before it is read: two stages (128 KB) are
// enough to hide the memory's latency.
//
// Every wave reads its LDS data completely (lgkmcnt(0)) before the barrier that ends a read phase, so
// a refill started after that barrier cannot overtake a read; each wave waits for its own copies
// (vmcnt, in order of issue) before the barrier after which any wave reads them.
struct Operands {
  const char *left;    // uniform: the tile's first row (kTrans: first column)
  const char *right;   // uniform
  uint32_t left_pitch; // kTrans: bytes between rows of the contraction
  uint32_t left_off[4];   // per lane: copies of rows 0..63 (0, 1) and 64..127 (2, 3) of both row halves
  uint32_t right_off[4];
  int64_t left_step, right_step;  // bytes per contraction step
  int left_rows;       // kTrans: rows of the contraction that exist (the last one stands for those beyond)
};

template <bool kTrans>
__device__ __forceinline__ void copy_left(const Operands &o, int half, int k, int steps, char *stage, int wave,
                                          int lane) {
  const int kc = min(k, steps - 1);  // past the end: any valid rows, never read
  const char *base = o.left + kc * o.left_step;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t off = o.left_off[2 * half + j];
    if (kTrans) {
      // row (2 wave + j) * 8 + lane / 8 of the unit: contraction row of a 64-row sub-tile
      const int row = ((2 * wave + j) * 8 + (lane >> 3)) & 63;
      off += (uint32_t)__mul24(min(row, o.left_rows - 1 - kc * kStep), (int)o.left_pitch);
    }
    dma16(base, off, lds_addr(stage + half * kUnit + (2 * wave + j) * 1024));
  }
}

__device__ __forceinline__ void copy_right(const Operands &o, int k, int steps, char *stage, int wave) {
  const int kc = min(k, steps - 1);
  const char *base = o.right + kc * o.right_step;
#pragma unroll
  for (int j = 0; j < 4; ++j) dma16(base, o.right_off[j], lds_addr(stage + 2 * kUnit + (4 * wave + j) * 1024));
}

template <bool kTrans>
__device__ __forceinline__ void read_left(const char *stage, int half, int kk, int wm, int lane, u32x4 (&a)[4]) {
  const char *unit = stage + half * kUnit + wm * 8192;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    if (!kTrans) {
      const int r = 16 * f + (lane & 15), c = 4 * kk + (lane >> 4);
      a[f] = *(const u32x4 *)(unit + r * 128 + ((c ^ swizzle_rows(r)) << 4));
    } else {
      // lane s of a 16-lane group points at contraction row .. + s/4 and columns 4 (s%4); it
      // receives four consecutive contraction rows of column s
      const int s = lane & 15;
      uint2 part[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 32 * kk + 8 * (lane >> 4) + 4 * h + (s >> 2);
        const int c = 2 * f + ((s & 3) >> 1);
        const char *p = unit + r * 128 + ((c ^ swizzle_cols(r)) << 4) + (s & 1) * 8;
        part[h] = __builtin_bit_cast(
            uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((v4s __attribute__((address_space(3))) *)(lds_void_t *)p));
      }
      a[f] = u32x4{part[0].x, part[0].y, part[1].x, part[1].y};
    }
  }
}

__device__ __forceinline__ void read_right(const char *stage, int kk, int wn, int lane, u32x4 (&b)[4]) {
  const char *unit = stage + 2 * kUnit + wn * 8192;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int r = 16 * f + (lane & 15), c = 4 * kk + (lane >> 4);
    b[f] = *(const u32x4 *)(unit + r * 128 + ((c ^ swizzle_rows(r)) << 4));
  }
}

// Subtracts a power of two from the exponents of eight bf16 values >= 0 (0 where it falls below).
__device__ __forceinline__ void scale_down(u32x4 &v, uint32_t shift) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = v[i];  // a value of its own: a bit cast of a vector's element takes element 0
    const u16x2 less = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, word),
                                                     __builtin_bit_cast(u16x2, shift));
    v[i] = __builtin_bit_cast(uint32_t, less);
  }
}

__device__ __forceinline__ void multiply(const u32x4 (&a)[4], const u32x4 (&b)[4], f32x4 (*acc)[4]) {
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n)
      acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[m]), as_bf16x8(b[n]), acc[m][n], 0, 0, 0);
  __builtin_amdgcn_s_setprio(0);
}

// The 256 tokens' rows of a stage times 2^(-64 d), a token a thread (the first 256); d: two bits a token.
__device__ __forceinline__ void scale_tokens(char *stage, const uint8_t *distances) {
  const int r = threadIdx.x;
  const uint32_t d = (distances[r >> 2] >> (2 * (r & 3))) & 3u;
  if (d == 0) return;
  u32x4 *row = (u32x4 *)(stage + 2 * kUnit + r * 128);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    u32x4 v = row[c];
    scale_down(v, d * 0x20002000u);
    row[c] = v;
  }
}

// acc[m][n][q] of lane l: left row 128 wm + 16 m + 4 (l/16) + q, token 64 wn + 16 n + l%16.
// kScale: the tokens' operand holds values >= 0, multiplied by 2^(-64 d); shifts: d of 0 to 3 per token and two steps,
// four neighbouring tokens a byte, [steps / 2][64]; scaled: whether any of them is not 0.  (Scaled in the
// fragments' registers, every step paid for it: 859 against 820 us for 2048 tokens by 4096 by 32000.)
template <bool kTrans, bool kScale>
__device__ __forceinline__ void product(const Operands &o, int steps, char *lds, const uint8_t *shifts, bool scaled,
                                        f32x4 (&acc)[8][4]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) & 1, wn = (wave & 1) + 2 * (wave >> 2);
  const bool late = wave >= 4;
  copy_right(o, 0, steps, lds, wave);
  copy_left<kTrans>(o, 0, 0, steps, lds, wave, lane);
  copy_left<kTrans>(o, 1, 0, steps, lds, wave, lane);
  copy_right(o, 1, steps, lds + kStage, wave);
  copy_left<kTrans>(o, 0, 1, steps, lds + kStage, wave, lane);
  TILE_WAIT_VM(8);
  barrier();
  if (late) barrier();
  u32x4 a0[4], a1[4], b0[4], b1[4];
  for (int k = 0; k < steps; ++k) {
    char *stage = lds + (k & 1) * kStage, *next = lds + ((k + 1) & 1) * kStage;
    if (kScale && scaled) {  // a phase of its own, rarely taken: the first group scales the tokens' tile in place
      if (!late) scale_tokens(stage, shifts + (k >> 1) * (kTileT / 4));
      TILE_WAIT_LDS();
      barrier();
    }
    // phase 0: rows 0..63
    read_right(stage, 0, wn, lane, b0);
    read_left<kTrans>(stage, 0, 0, wm, lane, a0);
    read_right(stage, 1, wn, lane, b1);
    read_left<kTrans>(stage, 0, 1, wm, lane, a1);
    copy_left<kTrans>(o, 1, k + 1, steps, next, wave, lane);
    TILE_WAIT_LDS();
    TILE_WAIT_VM(8);
    barrier();
    multiply(a0, b0, acc);
    multiply(a1, b1, acc);
    barrier();
    // phase 1: rows 64..127
    read_left<kTrans>(stage, 1, 0, wm, lane, a0);
    read_left<kTrans>(stage, 1, 1, wm, lane, a1);
    copy_right(o, k + 2, steps, stage, wave);
    copy_left<kTrans>(o, 0, k + 2, steps, stage, wave, lane);
    TILE_WAIT_LDS();
    TILE_WAIT_VM(8);
    barrier();
    multiply(a0, b0, acc + 4);
    multiply(a1, b1, acc + 4);
    barrier();
  }
  if (!late) barrier();
  TILE_WAIT_VM(0);  // no copy may outlive the loop: the LDS is reused or given up
  barrier();
}

// A value that is the same in every lane, moved to a scalar register (a division leaves it in a vector
// register, and the products have none to spare).
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Place of a workgroup among `total`.  Workgroup ids go round the eight XCDs, so id / 8 counts within
// one: each XCD takes a contiguous run of places.
__device__ __forceinline__ int place_of(int id, int total) {
  const int per = total >> 3, rest = total & 7, x = id & 7;
  return x * per + min(x, rest) + (id >> 3);  // XCDs below `rest` take one more
}

// The tile at a place: token tiles in groups of eight, every left tile of a group before the next
// group, tokens fastest, so that 32 neighbours (one per CU of an XCD) cover about 8 token by 4 left
// tiles, whose operands its L2 then serves.
struct Tile {
  int left, token;
};
__device__ __forceinline__ Tile tile_at(int place, int nleft, int ntoken) {
  const int group = place / (8 * nleft), first = group * 8;
  const int width = min(8, ntoken - first), in = place - group * 8 * nleft;
  const int left = in / width;
  return Tile{scalar(left), scalar(first + in - left * width)};
}
__device__ __forceinline__ int place_at(const Tile &tile, int nleft, int ntoken) {
  const int group = tile.token / 8;
  return group * 8 * nleft + tile.left * min(8, ntoken - 8 * group) + tile.token - 8 * group;
}

// Splits of the contraction (`length` long, in ranges of whole 128s) of `tiles` output tiles: the count
// with the least rounds of 256 workgroups times range, where a range costs about 512 more (its first
// copies and its result: 12 us against 1.4 us a step) and every partial tile about 2 (256 KB written and
// read again).  At most kMaxSlots workgroups unless the tiles alone are more.
constexpr int kMaxSplits = 64, kMaxSlots = 512;
struct Split {
  int count, range;
};
// The cost of `s` splits, 2^40 and more where they are not possible; their count without empty ranges and the range.
__host__ __device__ inline int64_t split_cost(int tiles, int length, int s, Split &out) {
  const int range = ((length + s - 1) / s + 127) / 128 * 128;
  const int n = (length + range - 1) / range;
  out = Split{n, range};
  if (s > 1 && (tiles * n > kMaxSlots || range < 256)) return (int64_t)1 << 40;
  return (int64_t)((tiles * n + 255) / 256) * (range + 512) + 2 * tiles * n;
}
inline Split choose_split(int tiles, int length) {
  Split best{}, one{};
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= kMaxSplits; ++s) {
    const int64_t c = split_cost(tiles, length, s, one);
    if (c >= (int64_t)1 << 40) break;  // nor are more splits possible
    if (c < cost) {
      cost = c;
      best = one;
    }
  }
  return best;
}
// The same on the device, one count a lane.
__device__ __forceinline__ Split split_of(int tiles, int length) {
  Split mine;
  const int lane = threadIdx.x & 63;
  int64_t key = split_cost(tiles, length, lane + 1, mine) * 64 + lane;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t other = ((int64_t)__shfl_xor((int)(key >> 32), d) << 32) | (uint32_t)__shfl_xor((int)key, d);
    key = other < key ? other : key;
  }
  const int s = (int)(key & 63);
  return Split{scalar(__shfl(mine.count, s)), scalar(__shfl(mine.range, s))};
}

// Workgroups (and partial tiles) that `nleft` by up to `ntoken` tiles need at most.
inline int split_slots(int nleft, int ntoken, int length) {
  int slots = 0;
  for (int t = 1; t <= ntoken; ++t) {
    const int n = nleft * t * choose_split(nleft * t, length).count;
    slots = n > slots ? n : slots;
  }
  return slots;
}

// ---- up to 64 tokens --------------------------------------------------------
// A workgroup takes 64 rows or columns of the left operand and its four waves every fourth contraction
// step each, with no barrier until their sums are added: a wave copies its own 64 x 64 tile (8 KB) and
// the tokens' piece of the step into LDS, one or two steps ahead.  The tokens fill NT tiles of 16.
constexpr int kFewThreads = 256;
constexpr int kFewTokens = 64;

template <int NT>
constexpr int few_stage() {
  return 8192 + NT * 2048;
}
// Stages of a wave.  The logits of 16 tokens fit two workgroups of two stages on a CU; otherwise one
// workgroup has the CU to itself and takes three where they fit.
template <bool kTrans, int NT>
constexpr int few_stages() {
  return NT == 4 || (!kTrans && NT == 1) ? 2 : 3;
}

template <int n>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(n) : "memory");
}

// acc[m][n][q] of lane l: left row (or column) 16 m + 4 (l/16) + q, token 16 n + l%16, added up over the
// wave's steps first, first + 4, ..  mine: the wave's stages.  right_off: per lane, the rows of the
// tokens.  left_rows: rows that exist, of the tile or (kTrans) of the whole contraction.  kScale as
// above, shifts [steps][16 NT].
template <bool kTrans, bool kScale, int NT>
__device__ __forceinline__ void few_product(const char *left, uint32_t left_pitch, int left_rows, int64_t left_step,
                                            const char *right, const uint32_t (&right_off)[2 * NT], int first,
                                            int steps, char *mine, const uint8_t *shifts, f32x4 (&acc)[4][NT]) {
  constexpr int kStages = few_stages<kTrans, NT>(), kBytes = few_stage<NT>(), kCopies = 8 + 2 * NT;
  const int lane = threadIdx.x & 63;
  if (first >= steps) return;
  auto copy = [&](int step, char *stage) {
    const int s = min(step, steps - 1);  // past the end: never read
    const char *lb = left + s * left_step, *rb = right + (int64_t)s * (2 * kStep);
    const int rows = kTrans ? left_rows - s * kStep : left_rows;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = 8 * j + (lane >> 3);
      const int sw = kTrans ? swizzle_cols(r) : swizzle_rows(r);
      dma16(lb, (uint32_t)__mul24(min(r, rows - 1), (int)left_pitch) + (((lane & 7) ^ sw) << 4),
            lds_addr(stage + 1024 * j));
    }
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) dma16(rb, right_off[j], lds_addr(stage + 8192 + 1024 * j));
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) copy(first + 4 * i, mine + i * kBytes);
  char *stage = mine;
  for (int s = first; s < steps; s += 4) {
    wait_copies<(kStages - 1) * kCopies>();
    u32x4 a[2][4], b[2][NT];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      read_left<kTrans>(stage, 0, kk, 0, lane, a[kk]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 16 * n + (lane & 15), c = 4 * kk + (lane >> 4);
        b[kk][n] = *(const u32x4 *)(stage + 8192 + r * 128 + ((c ^ swizzle_rows(r)) << 4));
      }
    }
    uint32_t shift[NT];
    if (kScale) {
#pragma unroll
      for (int n = 0; n < NT; ++n) shift[n] = (uint32_t)shifts[s * (16 * NT) + 16 * n + (lane & 15)] * 0x00800080u;
    }
    TILE_WAIT_LDS();
    copy(s + 4 * kStages, stage);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (kScale) scale_down(b[kk][n], shift[n]);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[kk][m]), as_bf16x8(b[kk][n]), acc[m][n], 0,
                                                             0, 0);
      }
    stage = stage == mine + (kStages - 1) * kBytes ? mine : stage + kBytes;
  }
  wait_copies<0>();
}

// The same with a packed left operand, decoded on its way into LDS: a lane takes one row of the tile, which is one NF4
// block (32 bytes of codes, one constant), builds the block's 16 values in registers and selects them by code, about
// 270 vector instructions a step.  These issue in 63% of the busy cycles of one token's logits (two waves a SIMD) and in
// 45% of its gradient's (one wave a SIMD; both products of 64 tokens: 45 and 47%); the rest is a wave's chain of
// decode, LDS write, wait, LDS read and multiply.  The codes of a step are loaded two steps ahead.  Against
// decoded rows in the workspace, W of 32000 x 4096: one token's loss 114 -> 32 us, with the gradient (each product
// decodes) 165 -> 72 us; 64 tokens 119 -> 54 and 181 -> 109 us.
struct PackedRow {
  u32x4 codes[2];
  uint32_t q;
  float s2;
};

// row0: the tile's first row (kTrans: the contraction's); rows: rows that exist from there; slice: kTrans: the tile's
// block of 64 columns.
template <bool kTrans, bool kScale, int NT>
__device__ __forceinline__ void few_product_packed(const QWeight &q, const Codebook &cb, int64_t row0, int rows,
                                                   int row_blocks, int slice, const char *right,
                                                   const uint32_t (&right_off)[2 * NT], int first, int steps,
                                                   char *mine, const uint8_t *shifts, f32x4 (&acc)[4][NT]) {
  constexpr int kBytes = few_stage<NT>(), kCopies = 2 * NT;
  const int lane = threadIdx.x & 63;
  if (first >= steps) return;
  const float mu = q.dq ? *q.mu : 0.f;
  auto load = [&](int step, PackedRow &p) {
    const int s = min(step, steps - 1);  // past the end: never used
    const int64_t row = row0 + (kTrans ? min(s * kStep + lane, rows - 1) : min(lane, rows - 1));
    const int64_t block = row * row_blocks + (kTrans ? slice : s);
    const u32x4 *c = (const u32x4 *)(q.codes + block * (kBlock / 2));
    p.codes[0] = c[0];
    p.codes[1] = c[1];
    p.s2 = q.s2[q.dq ? block / kGroup : block];
    p.q = *(q.dq ? q.fp8 + block : q.codes);  // a load in any case: a branch here would make the loop wait for all
  };
  auto copy = [&](int step, char *stage) {
    const char *rb = right + (int64_t)min(step, steps - 1) * (2 * kStep);
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) dma16(rb, right_off[j], lds_addr(stage + 8192 + 1024 * j));
  };
  auto turn = [&](int s, PackedRow &p, char *stage) {
    {
      const float c1 = q.dq ? decode_constant(p.q, p.s2, mu) : p.s2;
      DecodeTable t;
      uint32_t pair[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        pair[i] = pack_bf16x2(decode_product(cb.v[2 * i], c1), decode_product(cb.v[2 * i + 1], c1));
      uint32_t lo[2], hi[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t four[4] = {pair[4 * h], pair[4 * h + 1], pair[4 * h + 2], pair[4 * h + 3]};
        table_half(four, lo, hi);
        t.lo[2 * h] = lo[0];
        t.lo[2 * h + 1] = lo[1];
        t.hi[2 * h] = hi[0];
        t.hi[2 * h + 1] = hi[1];
      }
      const int sw = kTrans ? swizzle_cols(lane) : swizzle_rows(lane);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t o[4];
        const uint32_t codes = p.codes[c >> 2][c & 3];
        decode_word(codes, t, o);
        *(u32x4 *)(stage + lane * 128 + ((c ^ sw) << 4)) = u32x4{o[0], o[1], o[2], o[3]};
      }
    }
    // the step's copies are older than its four loads, the next step's copies (and loads) younger
    wait_copies<kCopies + 3>();
    TILE_WAIT_LDS();
    u32x4 a[2][4], b[2][NT];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      read_left<kTrans>(stage, 0, kk, 0, lane, a[kk]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 16 * n + (lane & 15), c = 4 * kk + (lane >> 4);
        b[kk][n] = *(const u32x4 *)(stage + 8192 + r * 128 + ((c ^ swizzle_rows(r)) << 4));
      }
    }
    uint32_t shift[NT];
    if (kScale) {
#pragma unroll
      for (int n = 0; n < NT; ++n) shift[n] = (uint32_t)shifts[s * (16 * NT) + 16 * n + (lane & 15)] * 0x00800080u;
    }
    TILE_WAIT_LDS();
    copy(s + 8, stage);
    load(s + 8, p);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (kScale) scale_down(b[kk][n], shift[n]);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[kk][m]), as_bf16x8(b[kk][n]), acc[m][n], 0,
                                                             0, 0);
      }
  };
  PackedRow even, odd;
  copy(first, mine);
  load(first, even);
  copy(first + 4, mine + kBytes);
  load(first + 4, odd);
  for (int s = first; s < steps; s += 8) {
    turn(s, even, mine);
    if (s + 4 < steps) turn(s + 4, odd, mine + kBytes);
  }
  wait_copies<0>();
}

// The four waves' sums side by side in LDS: [wave][token][68], 64 left rows a token.
constexpr int kFewPad = 68;
template <int NT>
__device__ __forceinline__ void few_put(const f32x4 (&acc)[4][NT], float *red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();  // every wave is done with its stages
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(f32x4 *)&red[((wave * NT + n) * 16 + (lane & 15)) * kFewPad + 16 * m + 4 * (lane >> 4)] = acc[m][n];
  __syncthreads();
}

// The sum over the waves of four left rows of a token.
template <int NT>
__device__ __forceinline__ f32x4 few_sum(const float *red, int token, int row) {
  f32x4 s = *(const f32x4 *)&red[token * kFewPad + row];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const f32x4 x = *(const f32x4 *)&red[(w * 16 * NT + token) * kFewPad + row];
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += x[q];
  }
  return s;
}

template <int NT>
__device__ __forceinline__ void few_zero(f32x4 (&acc)[4][NT]) {
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
}

__device__ __forceinline__ void tile_zero(f32x4 (&acc)[8][4]) {
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace
}  // namespace qlora
