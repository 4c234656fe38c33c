// The gated product behind its projections for up to 128 tokens (gfx950).
//
// Reading and decoding the 4-bit weights is the work here, so every code is read once, decoded once in the
// registers of the lane that multiplies it, and used for all tokens.
//
//   gated_few_prep   u = x A_set^T (bf16), and x laid out as the products take it
//   gated_few        16 columns of gate and of up a workgroup, its waves every fourth chunk of 256 of n_in each; their
//                    sums meet in LDS and the workgroup writes its columns of h (gate, up)
//   gated_split      more than 64 tokens, or 16 of large weights: 64 columns of each a workgroup, 16 a wave, over a range
//                    of the chunks; x comes through LDS, once for the four waves, and the ranges' fp32 results are
//                    added by a launch more
//
// What bounds them: the decode's vector instructions and, next to them, HBM.  Two 11008 x 4096 weights (46.5 MB), 1 token:
// prep 3.6 us, gated_few 16.9 (2.7 TB/s; 4 less with the decode's lookups left out), two 22016 x 8192 (186 MB) 54 at best, 60
// in the mean (3.1 to 3.4 TB/s; 13 less); the decode is 23 instructions for 8 codes of a lane and 5 for their share of the
// table, 38 us of the 54 on all SIMDs.  Codes or x a chunk further ahead cost a wave a SIMD and more than they gain (with
// prep 62 -> 65 us).  gated_split, 64 tokens of 22016 x 8192: 82 us at best, 92 in the mean, of which 43 are the decode's
// instructions and 21 the products.  The adapter's operands are all asked for at once and before the first codes (one after
// the other they were 6 us of 33 tokens of 11008 x 4096).
//
// v_mfma_f32_16x16x32_bf16: A lane l holds A[l % 16][8 (l / 16) + 0..7], B lane l holds B[8 (l / 16) + 0..7][l % 16],
// D register i of lane l is D[4 (l / 16) + i][l % 16].  Which 32 values of the contraction a product takes, and in what
// order, is free as long as A and B agree.  Here lane (n, g) = (l % 16, l / 16) decodes one whole NF4 block of row
// n a chunk, block 4 s + g of chunk s: one constant and one table for 64 codes.  Product j of the chunk takes the j-th
// eight codes of the four blocks, in the order 0 2 4 6 1 3 5 7 in which the decode leaves them.  x is laid out
// accordingly, [chunk][j][g][token][8]: an operand of 16 tokens is 1 KB in the order of its lanes.

#include <algorithm>

#include "common.hpp"
#include "gated.hpp"
#include "launch.hpp"
#include "tile.hpp"

namespace qlora {

namespace {

constexpr int kChunkBlocks = 4;            // NF4 blocks of a row in a chunk
constexpr int kChunk = 64 * kChunkBlocks;  // n_in of a chunk
constexpr int kWaves = 4;                  // waves of a workgroup
constexpr int kPrepWaves = 8, kPrepRows = 4, kPrepTokens = 4;
static_assert(kPrepRows * kPrepTokens == 16, "the lanes' exchange holds 16 sums");

__device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// Ranks [j, j + 8) of a row of r values, zero past r.
__device__ __forceinline__ u32x4 ranks8(const uint16_t *row, int j, int r) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (j + 8 <= r) {
    v = load8(row + j);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < r) v[i >> 1] |= (uint32_t)row[j + i] << (16 * (i & 1));
  }
  return v;
}

__device__ __forceinline__ float dot8(const u32x4 &a, const u32x4 &b, float c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = a[i], y = b[i];
    c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), __builtin_bit_cast(bf16x2, y), c, false);
  }
  return c;
}

// Workgroups below `utiles`: kPrepRows rows of A_set by kPrepTokens tokens of u, the lanes along n_in (a matrix
// instruction's operand would take rows from neighbouring lanes: 64 accesses a load).  The others: x [T][K] into xp, 8
// values a thread, zero past n_in.
__global__ __launch_bounds__(64 * kPrepWaves) void gated_few_prep(const uint16_t *__restrict__ x,
                                                                  const uint16_t *__restrict__ A, int T, int K,
                                                                  int ld, int rows, int utiles, uint16_t *__restrict__ u,
                                                                  uint16_t *__restrict__ xp) {
  __shared__ __attribute__((aligned(16))) float red[kPrepWaves][kPrepRows * kPrepTokens];
  if ((int)blockIdx.x >= utiles) {
    const uint32_t i = ((uint32_t)blockIdx.x - utiles) * (64 * kPrepWaves) + threadIdx.x;
    const uint32_t runs = (uint32_t)((K + kChunk - 1) / kChunk) * (kChunk / 8) * T;
    if (i >= runs) return;
    const uint32_t rest = i / T, t = i - rest * T, sj = rest >> 2, g = rest & 3;
    const int k = 64 * (kChunkBlocks * (int)(sj >> 3) + (int)g) + 8 * (int)(sj & 7);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < K) v = *(const u32x4 *)(x + (int64_t)t * K + k);
    // 0 2 | 4 6 | 1 3 | 5 7
    *(u32x4 *)(xp + 8 * ((int64_t)rest * ld + t)) =
        u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
              __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
    return;
  }
  const int row_tiles = (rows + kPrepRows - 1) / kPrepRows;
  const int r0 = kPrepRows * ((int)blockIdx.x % row_tiles), t0 = kPrepTokens * ((int)blockIdx.x / row_tiles);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint16_t *xr[kPrepTokens], *ar[kPrepRows];
#pragma unroll
  for (int i = 0; i < kPrepTokens; ++i) xr[i] = x + (int64_t)min(t0 + i, T - 1) * K;
#pragma unroll
  for (int i = 0; i < kPrepRows; ++i) ar[i] = A + (int64_t)min(r0 + i, rows - 1) * K;
  float acc[kPrepRows][kPrepTokens] = {};
  for (int k0 = 512 * wave; k0 < K; k0 += 512 * kPrepWaves) {
    const int k = k0 + 8 * lane;
    const bool in = k < K;
    const u32x4 none = {0u, 0u, 0u, 0u};
    u32x4 av[kPrepRows], xv[kPrepTokens];
#pragma unroll
    for (int i = 0; i < kPrepRows; ++i) av[i] = in ? *(const u32x4 *)(ar[i] + k) : none;
#pragma unroll
    for (int i = 0; i < kPrepTokens; ++i) xv[i] = in ? *(const u32x4 *)(xr[i] + k) : none;
#pragma unroll
    for (int i = 0; i < kPrepRows; ++i)
#pragma unroll
      for (int h = 0; h < kPrepTokens; ++h) acc[i][h] = dot8(av[i], xv[h], acc[i][h]);
  }
  // The 16 sums over the lanes.  A swap of two registers' halves (odd rows of 16 with even ones) and an addition fold two
  // values into one register; the rows' sums are rotations.  Row p of 16 lanes holds values 4 p + 0..3.
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = acc[i / kPrepTokens][i % kPrepTokens];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fold<32>(v[i], v[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = fold<16>(v[i], v[i + 4]);
    v[i] = row16_sum(v[i]);
  }
  if ((lane & 15) == 0) *(f32x4 *)&red[wave][4 * (lane >> 4)] = f32x4{v[0], v[1], v[2], v[3]};
  __syncthreads();
  const int i = threadIdx.x / kPrepTokens, h = threadIdx.x % kPrepTokens;
  if (i >= kPrepRows || t0 + h >= T || r0 + i >= rows) return;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kPrepWaves; ++w) s += red[w][threadIdx.x];
  u[(int64_t)(t0 + h) * rows + r0 + i] = __builtin_bit_cast(uint16_t, (__bf16)s);
}

// Four of the bytes that a table of 16 holds, for four codes given by their low 3 bits (sel) and by the place of each
// in the lookups of the two halves, byte i of the lower or (bit 3) of the upper one (pick).
__device__ __forceinline__ uint32_t four_bytes(const uint32_t (&tb)[4], uint32_t sel, uint32_t pick) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(tb[3], tb[2], sel), __builtin_amdgcn_perm(tb[1], tb[0], sel), pick);
}

// Eight codes (low nibble first) -> four bf16 pairs, (0, 2), (4, 6), (1, 3), (5, 7).
__device__ __forceinline__ u32x4 decode_split(uint32_t c, const DecodeTable &t) {
  uint32_t own = 0x03020100u, upper = 0x04040404u;
  asm("" : "+v"(own), "+s"(upper));  // in registers: as literals they would keep the and and the or apart
  const uint32_t se = c & 0x07070707u, so = (c >> 4) & 0x07070707u;
  const uint32_t pe = ((c >> 1) & upper) | own, po = ((c >> 5) & upper) | own;
  const uint32_t le = four_bytes(t.lo, se, pe), he = four_bytes(t.hi, se, pe);
  const uint32_t lq = four_bytes(t.lo, so, po), hq = four_bytes(t.hi, so, po);
  return u32x4{__builtin_amdgcn_perm(he, le, 0x05010400u), __builtin_amdgcn_perm(he, le, 0x07030602u),
               __builtin_amdgcn_perm(hq, lq, 0x05010400u), __builtin_amdgcn_perm(hq, lq, 0x07030602u)};
}

// A chunk of one member's 16 rows as it is loaded: 8 lanes take the 128 bytes of a row, so that a load is whole
// cache lines (a lane's own block, 16 rows apart from its neighbours', is 64 accesses a load: the 90 M codes of two
// 11008 x 4096 weights then take 23 us whatever is done with them).  Lane l holds 16 bytes, piece l % 8, of rows l / 8 and
// 8 + l / 8, and the constant of the block that it decodes.
struct Pieces {
  u32x4 codes[2];
  uint32_t q;
  float s2;
};

// Through the wave's own 2 KB of LDS to the lanes that decode: piece c of row r at position c ^ (r / 2 % 8), so that
// the 16 rows of a read fall on different banks.
__device__ __forceinline__ int piece_at(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

template <bool kDQ>
__device__ __forceinline__ void build_table(const Pieces &b, float mu, const Codebook &cb, DecodeTable &t) {
  const float c1 = kDQ ? decode_constant(b.q, b.s2, mu) : b.s2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4], lo[2], hi[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = pack_bf16x2(decode_product(cb.v[8 * h + 2 * i], c1), decode_product(cb.v[8 * h + 2 * i + 1], c1));
    table_half(p, lo, hi);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t.lo[2 * h + i] = lo[i];
      t.hi[2 * h + i] = hi[i];
    }
  }
}

// The operands of 32 ranks from j on: a lane's eight of a row of each B and of each of its tokens' u.
template <int TT>
struct Ranks {
  u32x4 b[2], u[2][TT];
};

struct GatedFewArgs {
  const uint16_t *xp, *u;
  QWeight w[2];
  const uint16_t *B[2];
  int T, ld, N, K, r;  // ld: tokens from one eight of xp to the next
  float scale;
};

// All loads are on their way before one is waited for (with ranks of whole eights; otherwise value by value).
template <int TT>
__device__ __forceinline__ void load_ranks(const GatedFewArgs &a, int64_t row, const int (&token)[TT], int j,
                                           Ranks<TT> &o) {
  if ((a.r & 7) == 0) {
    const int at = min(j, a.r - 8);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      o.b[m] = load8(a.B[m] + row * a.r + at);
#pragma unroll
      for (int h = 0; h < TT; ++h) o.u[m][h] = load8(a.u + (int64_t)token[h] * (2 * a.r) + m * a.r + at);
    }
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      o.b[m] = ranks8(a.B[m] + row * a.r, j, a.r);
#pragma unroll
      for (int h = 0; h < TT; ++h) o.u[m][h] = ranks8(a.u + (int64_t)token[h] * (2 * a.r) + m * a.r, j, a.r);
    }
  }
}

// acc += u B^T of them, D's rows the tokens', or with kSwap the weight's.
template <bool kSwap, int TT>
__device__ __forceinline__ void add_ranks(const GatedFewArgs &a, int j, Ranks<TT> &o, f32x4 (&acc)[2][TT]) {
  const u32x4 none = {0u, 0u, 0u, 0u};
  const bool in = j < a.r;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const u32x4 b = in ? o.b[m] : none;
#pragma unroll
    for (int h = 0; h < TT; ++h) {
      const u32x4 u = in ? o.u[m][h] : none;
      acc[m][h] = kSwap ? mfma16(b, u, acc[m][h]) : mfma16(u, b, acc[m][h]);
    }
  }
}

// TT tiles of 16 tokens.  Four of them are held to three waves a SIMD, so that the 2.7 that 11008 x 4096 has run at once
// (64 tokens: 37.3 -> 34.9 us); with three the compiler's own choice is faster (33 tokens of 5504 x 2048: 16.4 against 18.8).
template <int TT, bool kDQ>
__global__ __launch_bounds__(64 * kWaves, TT == 4 ? 3 : 0) void gated_few(GatedFewArgs a, Codebook cb, GatedOut out) {
  __shared__ float red[kWaves][16 * TT][17];
  __shared__ __attribute__((aligned(16))) char turn[kWaves][2][2048];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t row = 16 * (int64_t)blockIdx.x + n;
  const int blocks = a.K / kBlock, chunks = (blocks + kChunkBlocks - 1) / kChunkBlocks;
  // Uniform bases and 32-bit lane offsets: the tile's rows of each weight (fewer than 2^31 blocks in all).
  const uint32_t pitch = (uint32_t)a.K / 2, tile0 = blockIdx.x * 16u * (uint32_t)blocks;
  const uint32_t code_row = (uint32_t)(lane >> 3) * pitch, block_row = (uint32_t)n * (uint32_t)blocks;
  auto load = [&](int s, Pieces (&b)[2]) {  // past the row's end: any of it, x is 0 there
    const int c = min(s, chunks - 1);
    const uint32_t code = code_row + min(128u * (uint32_t)c + 16u * (lane & 7), pitch - 16u);
    const uint32_t block = block_row + min((uint32_t)(kChunkBlocks * c + g), (uint32_t)blocks - 1u);
    const uint32_t constant = kDQ ? (tile0 + block) >> 8 : tile0 + block;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint8_t *codes = a.w[m].codes + (int64_t)blockIdx.x * 16 * pitch;
      b[m].codes[0] = *(const u32x4 *)(codes + code);
      b[m].codes[1] = *(const u32x4 *)(codes + (code + 8u * pitch));
      if (kDQ) b[m].q = *(a.w[m].fp8 + tile0 + block);
      b[m].s2 = a.w[m].s2[constant];
    }
  };
  int token[TT];
#pragma unroll
  for (int h = 0; h < TT; ++h) token[h] = min(16 * h + n, a.T - 1);

  // the adapter term first, 32 ranks a product, the waves in turn; its first loads go out before those of the codes
  Ranks<TT> ranks;
  if (32 * wave < a.r) load_ranks(a, row, token, 32 * wave + 8 * g, ranks);
  Pieces next[2];
  load(wave, next);
  const float mu0 = kDQ ? *a.w[0].mu : 0.f, mu1 = kDQ ? *a.w[1].mu : 0.f;
  f32x4 acc[2][TT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < TT; ++h) acc[m][h] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int j = 32 * wave; j < a.r; j += 32 * kWaves) {
    if (j > 32 * wave) load_ranks(a, row, token, j + 8 * g, ranks);
    add_ranks<false>(a, j + 8 * g, ranks, acc);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < TT; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][h][i] *= a.scale;

  const u32x4 *xp = (const u32x4 *)a.xp;
  char *mine = turn[wave][0];
  for (int s = wave; s < chunks; s += kWaves) {
    u32x4 xf[8][TT];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int h = 0; h < TT; ++h) xf[j][h] = (xp + (int64_t)(8 * s + j) * 4 * a.ld)[(uint32_t)(g * a.ld + token[h])];
    DecodeTable t[2];
    u32x4 codes[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *(u32x4 *)(mine + 2048 * m + piece_at(8 * i + (lane >> 3), lane & 7)) = next[m].codes[i];
#pragma unroll
    for (int m = 0; m < 2; ++m) build_table<kDQ>(next[m], m ? mu1 : mu0, cb, t[m]);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) codes[m][i] = *(const u32x4 *)(mine + 2048 * m + piece_at(n, 2 * g + i));
    load(s + kWaves, next);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const u32x4 wg = decode_split(codes[0][j >> 2][j & 3], t[0]), wu = decode_split(codes[1][j >> 2][j & 3], t[1]);
#pragma unroll
      for (int h = 0; h < TT; ++h) {
        acc[0][h] = mfma16(xf[j][h], wg, acc[0][h]);
        acc[1][h] = mfma16(xf[j][h], wu, acc[1][h]);
      }
    }
  }

  // the waves' sums, gate's and then up's; TT values a thread
  float gate[TT];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    if (m) __syncthreads();
#pragma unroll
    for (int h = 0; h < TT; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][16 * h + 4 * g + i][n] = acc[m][h][i];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < TT; ++h) {
      const int t = 16 * h + (threadIdx.x >> 4), c = threadIdx.x & 15;
      float sum = red[0][t][c];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += red[w][t][c];
      if (m == 0) {
        gate[h] = sum;
      } else if (t < a.T) {
        const int64_t to = (int64_t)t * a.N + 16 * (int64_t)blockIdx.x + c;
        with_activation(out.act, [&](auto act) {
          out.h[to] = __builtin_bit_cast(uint16_t, (__bf16)(gate_act_of_sum<act()>(gate[h]) * sum));
        });
        if (out.gate) {
          out.gate[to] = __builtin_bit_cast(uint16_t, (__bf16)gate[h]);
          out.up[to] = __builtin_bit_cast(uint16_t, (__bf16)sum);
        }
      }
    }
  }
}

// TT tiles of 16 tokens, `range` chunks of n_in, z-th of them: part[z][T][2 N].  With x in registers more than two tiles
// leave a SIMD two waves, and each operand comes from L2 once for 32 columns; here it comes once for 128, half a chunk
// (four products) ahead, and the codes a chunk ahead, all by copies into LDS that no register holds.
//   xs   half chunks [4 j][g][token] of 16 bytes as they lie in xp, two in turn
//   cs   a wave's codes of a chunk, in the places that piece_at gives: read to registers at the chunk's start, then
//        refilled
// A wave's waits: at a chunk's start for all of its copies, in its middle for those of x, all but the four copies of
// codes issued after them; each before the barrier behind which other waves read what it has copied, and with
// lgkmcnt(0), so that what it has read is in registers before others overwrite it.  They are asm, which the compiler
// neither drops nor counts; the builtin beside the first tells it that nothing is on its way, or its own wait for what
// is loaded before the loop stands behind every chunk's copies.
template <int TT, bool kDQ>
__global__ __launch_bounds__(64 * kWaves, TT <= 4 ? 3 : 2) void gated_split(GatedFewArgs a, Codebook cb, int range,
                                                                            float *__restrict__ part) {
  __shared__ __attribute__((aligned(1024))) char xs[2][TT * 4096];
  __shared__ __attribute__((aligned(1024))) char cs[kWaves][2][2048];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int tiles = a.N / 64, tile = (int)blockIdx.x % tiles, z = (int)blockIdx.x / tiles;
  const int blocks = a.K / kBlock, chunks = (blocks + kChunkBlocks - 1) / kChunkBlocks;
  const int c0 = z * range, c1 = min(c0 + range, chunks);
  const int64_t row0 = 64 * (int64_t)tile + 16 * wave;
  const uint32_t pitch = (uint32_t)a.K / 2, block0 = (uint32_t)row0 * (uint32_t)blocks;
  const uint32_t block_row = (uint32_t)n * (uint32_t)blocks;
  const char *codes[2] = {uniform(a.w[0].codes + row0 * pitch), uniform(a.w[1].codes + row0 * pitch)};
  // the lane's pieces of a chunk from the scalar base; in the last chunk none past its row's end (x is 0 there)
  uint32_t from[2];
  const uint32_t x_from = 16u * lane;
  auto place = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * i + (lane >> 3);
      from[i] = (uint32_t)r * pitch + min(16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7)), pitch - 16u - 128u * (uint32_t)c);
    }
  };
  uint32_t q[2] = {};
  float s2[2];
  auto load = [&](int c) {  // `from` may change: nothing that it addresses is in flight
    const uint32_t block = block_row + min((uint32_t)(kChunkBlocks * c + g), (uint32_t)blocks - 1u);
    const uint32_t constant = kDQ ? (block0 + block) >> 8 : block0 + block;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (kDQ) q[m] = *(a.w[m].fp8 + block0 + block);
      s2[m] = a.w[m].s2[constant];
    }
    if (c == chunks - 1) place(c);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) dma16(codes[m] + 128 * (int64_t)c, from[i], lds_addr(cs[wave][m] + 1024 * i));
  };
  const char *xp = uniform(a.xp);
  auto load_x = [&](int h, int buf) {  // half chunk h: ld / 4 KB, the waves in turn
    const char *src = xp + (int64_t)h * 256 * a.ld;
    for (int p = wave; p < a.ld / 4; p += kWaves) dma16(src + 1024 * p, x_from, lds_addr(xs[buf] + 1024 * p));
  };
  int token[TT];
#pragma unroll
  for (int h = 0; h < TT; ++h) token[h] = min(16 * h + n, a.T - 1);
  const int splits = (int)gridDim.x / tiles;
  Ranks<TT> ranks;
  if (32 * z < a.r) load_ranks(a, row0 + n, token, 32 * z + 8 * g, ranks);
  place(0);
  load(c0);
  load_x(2 * c0, 0);
  const float mu0 = kDQ ? *a.w[0].mu : 0.f, mu1 = kDQ ? *a.w[1].mu : 0.f;
  // the adapter term, 32 ranks a product, the ranges in turn (its first loads are out already); D's rows are the weight's
  // here: a lane holds four neighbouring columns of one token
  f32x4 acc[2][TT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < TT; ++h) acc[m][h] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int j = 32 * z; j < a.r; j += 32 * splits) {
    if (j > 32 * z) load_ranks(a, row0 + n, token, j + 8 * g, ranks);
    add_ranks<true>(a, j + 8 * g, ranks, acc);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < TT; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][h][i] *= a.scale;

  for (int c = c0; c < c1; ++c) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::"v"(from[0]), "v"(from[1]), "v"(x_from) : "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    barrier();
    load_x(2 * c + 1, 1);
    u32x4 w[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) w[m][i] = *(const u32x4 *)(cs[wave][m] + piece_at(n, 2 * g + i));
    DecodeTable t[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) build_table<kDQ>(Pieces{{}, q[m], s2[m]}, m ? mu1 : mu0, cb, t[m]);
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(w[0][0]), "+v"(w[0][1]), "+v"(w[1][0]), "+v"(w[1][1])::"memory");
    const bool more = c + 1 < c1;
    if (more) load(c + 1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half) {
        if (more)
          asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)" ::: "memory");
        else
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        barrier();
        if (more) load_x(2 * c + 2, 0);
      }
      const char *xh = xs[half] + 16 * (g * a.ld + n);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 wg = decode_split(w[0][half][j], t[0]), wu = decode_split(w[1][half][j], t[1]);
#pragma unroll
        for (int h = 0; h < TT; ++h) {
          const u32x4 xf = *(const u32x4 *)(xh + 64 * j * a.ld + 256 * h);
          acc[0][h] = mfma16(wg, xf, acc[0][h]);
          acc[1][h] = mfma16(wu, xf, acc[1][h]);
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < TT; ++h) {
    const int t = 16 * h + n;
    if (t < a.T)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        *(f32x4 *)(part + ((int64_t)z * a.T + t) * (2 * (int64_t)a.N) + m * a.N + row0 + 4 * g) = acc[m][h];
  }
}

}  // namespace

static int64_t chunk_count(int64_t K) { return (K + kChunk - 1) / kChunk; }
// About two workgroups a CU, which holds three of them up to 64 tokens and two of more: with one the copies' latency shows
// (64 tokens of two 22016 x 8192 weights: 131 us, with two 96), with four the results cost more than they gain (103).  Past 64
// tokens the results are longer, so from 384 tiles on there is one range (128 tokens of 28672 x 4096: two 109 us, one 101;
// 22016 x 8192, 344 tiles: two 161, one 174).
static int64_t range_chunks(int64_t T, int64_t N, int64_t K) {
  const int64_t tiles = N / 64, want = T <= 64 ? (512 + tiles - 1) / tiles : std::max<int64_t>(512 / tiles, tiles < 384 ? 2 : 1);
  const int64_t splits = std::min(want, chunk_count(K));
  return (chunk_count(K) + splits - 1) / splits;
}

// In ranges where x in registers costs more than the launch that adds them.  One pass against ranges, us: 17 tokens of
// two 11008 x 4096 weights 23 and 30, 64 tokens 35 and 37; 33 tokens of 14336 x 4096 34 both, 64 tokens 43 and 40; 33 tokens of
// 13824 x 5120 42 and 41, of 22016 x 8192 95 and 81.
int gated_few_parts(int64_t T, int64_t N, int64_t K) {
  if (T <= 16 || (T <= 64 && N * K < (int64_t)(T <= 48 ? 64 : 48) << 20)) return 0;
  const int64_t range = range_chunks(T, N, K);
  return (int)((chunk_count(K) + range - 1) / range);
}

// Tiles of u, each of which reads its rows of A_set and its tokens whole.
static int64_t u_tiles(int64_t T, int r) {
  return (2 * r + kPrepRows - 1) / kPrepRows * ((T + kPrepTokens - 1) / kPrepTokens);
}
// So from some number of values on the two launches of the adapters' product are faster.  In the launch that lays out x,
// past 2^24: 128 tokens of two 8192 x 8192 weights at rank 64 (2^23) 65 us against 69 with them, at rank 128 75 both, at rank
// 200 85 against 81.  By itself, past 128 tokens, from 5 2^20: 256 tokens of 11008 x 4096 at rank 16 (2^21) 64.5 against 68.3, 129
// at rank 64 (2^22) 65 and 67, 1024 at rank 16 (2^23) 207 and 205.
bool gated_own_u(int64_t T, int64_t K, int r) {
  return u_tiles(T, r) * K <= (T <= kGatedFewTokens ? (int64_t)1 << 24 : (int64_t)5 << 20);
}

size_t gated_few_xp_values(int64_t T, int64_t K) { return (size_t)(chunk_count(K) * kChunk * ((T + 3) / 4 * 4)); }

hipError_t launch_gated_u(int64_t T, const uint16_t *x, const uint16_t *A_set, int64_t K, int r, uint16_t *u,
                          hipStream_t st) {
  const int utiles = (int)u_tiles(T, r);
  gated_few_prep<<<(unsigned)utiles, 64 * kPrepWaves, 0, st>>>(x, A_set, (int)T, (int)K, 0, 2 * r, utiles, u, nullptr);
  return hipGetLastError();
}

hipError_t launch_gated_few(int64_t T, const uint16_t *x, const QWeight *w, const uint16_t *A_set,
                            const uint16_t *const *B, int r, float scale, const GatedOut &out, uint16_t *u, uint16_t *xp,
                            float *part, const Codebook &cb, hipStream_t st) {
  const int64_t N = w[0].n_out, K = w[0].n_in;
  const int utiles = gated_own_u(T, K, r) ? (int)u_tiles(T, r) : 0;
  const int ld = (int)(T + 3) / 4 * 4;
  const int64_t runs = chunk_count(K) * (kChunk / 8) * T;
  gated_few_prep<<<(unsigned)(utiles + (runs + 64 * kPrepWaves - 1) / (64 * kPrepWaves)), 64 * kPrepWaves, 0, st>>>(
      x, A_set, (int)T, (int)K, ld, 2 * r, utiles, u, xp);
  const GatedFewArgs a{xp, u, {w[0], w[1]}, {B[0], B[1]}, (int)T, ld, (int)N, (int)K, r, scale};
  const int parts = gated_few_parts(T, N, K), range = (int)range_chunks(T, N, K);
  auto run = [&](auto tiles, auto dq) {
    if constexpr (tiles() > 1)
      if (parts) {
        gated_split<tiles(), dq()><<<(unsigned)(N / 64 * parts), 64 * kWaves, 0, st>>>(a, cb, range, part);
        return;
      }
    if constexpr (tiles() <= 4) gated_few<tiles(), dq()><<<(unsigned)(N / 16), 64 * kWaves, 0, st>>>(a, cb, out);
  };
  auto with_tiles = [&](auto dq) {
    if (T <= 16)
      run(std::integral_constant<int, 1>(), dq);
    else if (T <= 32)
      run(std::integral_constant<int, 2>(), dq);
    else if (T <= 48)
      run(std::integral_constant<int, 3>(), dq);
    else if (T <= 64)
      run(std::integral_constant<int, 4>(), dq);
    else if (T <= 96)
      run(std::integral_constant<int, 6>(), dq);
    else
      run(std::integral_constant<int, 8>(), dq);
  };
  TimedLaunch tl;
  const bool timed = timing_begin(st, tl, kTimedGemvFwd);
  if (w[0].dq)
    with_tiles(std::true_type());
  else
    with_tiles(std::false_type());
  if (timed) timing_end(st, tl);
  return hipGetLastError();
}

}  // namespace qlora
