// The gated product behind its projections for up to 128 tokens (gfx950).
//
// Reading and decoding the 4-bit weights is the work here, so every code is read once, decoded once in the
// registers of the lane that multiplies it, and used for all tokens; nothing of W goes through LDS.
//
//   gated_few_prep   u = x A_set^T (bf16), and x laid out as the products take it
//   gated_few        16 columns of gate and of up a workgroup, its waves every KS-th chunk of 256 of n_in each;
//                    their sums meet in LDS and the workgroup writes its columns of h (gate, up)
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

namespace qlora {

namespace {

constexpr int kChunkBlocks = 4;            // NF4 blocks of a row in a chunk
constexpr int kChunk = 64 * kChunkBlocks;  // n_in of a chunk
constexpr int kWaves = 4;                  // waves of a workgroup
constexpr int kPrepWaves = 16;

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

// Workgroups below `utiles`: 16 rows of A_set by 16 tokens of u, the waves every 16th step of 32 each.  The others: x
// [T][K] into xp, 8 values a thread, zero past n_in.
__global__ __launch_bounds__(64 * kPrepWaves) void gated_few_prep(const uint16_t *__restrict__ x,
                                                                  const uint16_t *__restrict__ A, int T, int K,
                                                                  int rows, int utiles, uint16_t *__restrict__ u,
                                                                  uint16_t *__restrict__ xp) {
  __shared__ float red[kPrepWaves][16][17];
  if ((int)blockIdx.x >= utiles) {
    const int64_t i = (int64_t)((int)blockIdx.x - utiles) * (64 * kPrepWaves) + threadIdx.x;
    const int64_t runs = (int64_t)((K + kChunk - 1) / kChunk) * (kChunk / 8) * T;
    if (i >= runs) return;
    const int64_t rest = i / T, t = i - rest * T, sj = rest >> 2;
    const int g = (int)(rest & 3);
    const int k = 64 * (kChunkBlocks * (int)(sj >> 3) + g) + 8 * (int)(sj & 7);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < K) v = *(const u32x4 *)(x + t * K + k);
    // 0 2 | 4 6 | 1 3 | 5 7
    *(u32x4 *)(xp + 8 * i) =
        u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
              __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
    return;
  }
  const int row_tiles = (rows + 15) / 16;
  const int r0 = 16 * ((int)blockIdx.x % row_tiles), t0 = 16 * ((int)blockIdx.x / row_tiles);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const uint16_t *xr = x + (int64_t)min(t0 + n, T - 1) * K + 8 * g, *ar = A + (int64_t)min(r0 + n, rows - 1) * K + 8 * g;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 32 * wave; k < K; k += 32 * kPrepWaves)
    acc = mfma16(*(const u32x4 *)(xr + k), *(const u32x4 *)(ar + k), acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][4 * g + i][n] = acc[i];
  __syncthreads();
  const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (threadIdx.x >= 256 || t0 + t >= T || r0 + c >= rows) return;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kPrepWaves; ++w) s += red[w][t][c];
  u[(int64_t)(t0 + t) * rows + r0 + c] = __builtin_bit_cast(uint16_t, (__bf16)s);
}

// Eight codes (low nibble first) -> four bf16 pairs, (0, 2), (4, 6), (1, 3), (5, 7): decode_word without its last
// step.
__device__ __forceinline__ u32x4 decode_split(uint32_t c, const DecodeTable &t) {
  const uint32_t c4 = c >> 4;
  const uint32_t se = c & 0x07070707u, so = c4 & 0x07070707u;
  const uint32_t me = __builtin_amdgcn_perm(c << 4, c << 12, 0x0B090A08u);
  const uint32_t mo = __builtin_amdgcn_perm(c, c << 8, 0x0B090A08u);
  const uint32_t le = table_bytes(t.lo, se, me), he = table_bytes(t.hi, se, me);
  const uint32_t lq = table_bytes(t.lo, so, mo), hq = table_bytes(t.hi, so, mo);
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

struct GatedFewArgs {
  const uint16_t *xp, *u;
  QWeight w[2];
  const uint16_t *B[2];
  int T, N, K, r;
  float scale;
};

// TT tiles of 16 tokens.
template <int TT, bool kDQ>
__global__ __launch_bounds__(64 * kWaves) void gated_few(GatedFewArgs a, Codebook cb, GatedOut out) {
  __shared__ float red[kWaves][16 * TT][17];
  __shared__ __attribute__((aligned(16))) char turn[kWaves][2][2048];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t row = 16 * (int64_t)blockIdx.x + n;
  const int blocks = a.K / kBlock, chunks = (blocks + kChunkBlocks - 1) / kChunkBlocks;
  const int pieces = a.K / 32;  // of a row
  const int64_t row0 = 16 * (int64_t)blockIdx.x;
  auto load = [&](int s, Pieces (&b)[2]) {  // past the row's end: any of it, x is 0 there
    const int c = min(s, chunks - 1);
    const int piece = min(2 * kChunkBlocks * c + (lane & 7), pieces - 1);
    const int64_t block = row * blocks + min(kChunkBlocks * c + g, blocks - 1);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        b[m].codes[i] = *(const u32x4 *)(a.w[m].codes + ((row0 + 8 * i + (lane >> 3)) * pieces + piece) * 16);
      if (kDQ) {
        b[m].q = a.w[m].fp8[block];
        b[m].s2 = a.w[m].s2[block >> 8];
      } else {
        b[m].s2 = a.w[m].s2[block];
      }
    }
  };
  Pieces next[2];
  load(wave, next);
  const float mu0 = kDQ ? *a.w[0].mu : 0.f, mu1 = kDQ ? *a.w[1].mu : 0.f;
  int token[TT];
#pragma unroll
  for (int h = 0; h < TT; ++h) token[h] = min(16 * h + n, a.T - 1);

  // the adapter term first: 32 ranks a product, the waves in turn
  f32x4 acc[2][TT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < TT; ++h) acc[m][h] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int j = 32 * wave; j < a.r; j += 32 * kWaves)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const u32x4 b = ranks8(a.B[m] + row * a.r, j + 8 * g, a.r);
#pragma unroll
      for (int h = 0; h < TT; ++h)
        acc[m][h] = mfma16(ranks8(a.u + (int64_t)token[h] * (2 * a.r) + m * a.r, j + 8 * g, a.r), b, acc[m][h]);
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
      for (int h = 0; h < TT; ++h) xf[j][h] = xp[((8 * s + j) * 4 + g) * a.T + token[h]];
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
          out.h[to] = __builtin_bit_cast(uint16_t, (__bf16)(gate_act<act()>(gate[h]) * sum));
        });
        if (out.gate) {
          out.gate[to] = __builtin_bit_cast(uint16_t, (__bf16)gate[h]);
          out.up[to] = __builtin_bit_cast(uint16_t, (__bf16)sum);
        }
      }
    }
  }
}

}  // namespace

bool gated_few_applies(int64_t T, int64_t N, int64_t K) { return T <= kGatedFewTokens && N <= INT32_MAX && K <= 65536; }

size_t gated_few_xp_values(int64_t T, int64_t K) { return (size_t)((K + kChunk - 1) / kChunk * kChunk * T); }

hipError_t launch_gated_few(int64_t T, const uint16_t *x, const QWeight *w, const uint16_t *A_set,
                            const uint16_t *const *B, int r, float scale, const GatedOut &out, uint16_t *u, uint16_t *xp,
                            const Codebook &cb, hipStream_t st) {
  const int64_t N = w[0].n_out, K = w[0].n_in;
  const int utiles = (int)((2 * r + 15) / 16 * ((T + 15) / 16));
  const int64_t runs = (int64_t)gated_few_xp_values(T, K) / 8;
  gated_few_prep<<<(unsigned)(utiles + (runs + 64 * kPrepWaves - 1) / (64 * kPrepWaves)), 64 * kPrepWaves, 0, st>>>(
      x, A_set, (int)T, (int)K, 2 * r, utiles, u, xp);
  const GatedFewArgs a{xp, u, {w[0], w[1]}, {B[0], B[1]}, (int)T, (int)N, (int)K, r, scale};
  auto run = [&](auto tiles) {
    if (w[0].dq)
      gated_few<tiles(), true><<<(unsigned)(N / 16), 64 * kWaves, 0, st>>>(a, cb, out);
    else
      gated_few<tiles(), false><<<(unsigned)(N / 16), 64 * kWaves, 0, st>>>(a, cb, out);
  };
  if (T <= 16)
    run(std::integral_constant<int, 1>());
  else if (T <= 32)
    run(std::integral_constant<int, 2>());
  else if (T <= 48)
    run(std::integral_constant<int, 3>());
  else if (T <= 64)
    run(std::integral_constant<int, 4>());
  else if (T <= 96)
    run(std::integral_constant<int, 6>());
  else
    run(std::integral_constant<int, 8>());
  return hipGetLastError();
}

}  // namespace qlora
