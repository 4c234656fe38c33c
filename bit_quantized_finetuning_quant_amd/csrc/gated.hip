// The gated product of a feed-forward block (gfx950): h = act(gate) up behind
// the projections of a gate and an up weight, the product alone, and its
// backward pass.
//
//   gate = x Wg^T + s u_g Bg^T,   up = x Wu^T + s u_u Bu^T,   h = bf16(act(gate) up)
//   dgate = bf16(dh up act'(gate)),   dup = bf16(dh act(gate))
//
// Behind the projections the product takes gate and up in fp32; the bf16 copies
// of both are what the backward pass reads, and need not be written.
//
// The product alone and its backward pass are bound by HBM: 2048 x 11008 with h and its codes written (158 MB) 28 us
// with inputs in turn, 5.6 TB/s (24 at best, part of it from the last-level cache); the gradients of 4096 x 22016 (902 MB) 152
// us, 5.9 TB/s.
//
// Behind the projections there are three forms.  Up to 128 tokens the decode is the work (gated_few.hip).  Then the fused
// GEMM (qgemm.hip) decodes a weight tile for 256 tokens beside the matrix instructions: 509 tokens of two 11008 x 4096
// weights 123 us, 0.75 PFLOP/s, bound by the two roles of its waves.  From where that costs less (the forms' times are
// estimated in plan_linear_gated) the weights are decoded first.

#include <algorithm>

#include "act8.hpp"
#include "common.hpp"
#include "gated.hpp"
#include "launch.hpp"
#include "tile.hpp"

namespace qlora {

namespace {

constexpr int kWide = 256;  // threads of the elementwise kernels
constexpr int kRuns = 2;    // runs of 8 values a thread takes, a workgroup's stride apart

template <Activation kAct>
__device__ __forceinline__ u32x4 product8(const u32x4 &g, const u32x4 &u) {
  u32x4 h;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t gp = g[j], up = u[j];
    h[j] = pack_bf16x2(gate_act<kAct>(bf16_lo(gp)) * bf16_lo(up), gate_act<kAct>(bf16_hi(gp)) * bf16_hi(up));
  }
  return h;
}

// 8 consecutive lanes share a block of the codes (N is a multiple of 64, so no block crosses a row).
template <Activation kAct, bool kStream>
__global__ __launch_bounds__(kWide) void gated_act_fwd(const uint16_t *gate, const uint16_t *up, int64_t runs,
                                                         uint16_t *h, int8_t *codes, float *scale) {
  const int64_t step = (int64_t)gridDim.x * (kWide * kRuns);
  for (int64_t first = (int64_t)blockIdx.x * (kWide * kRuns) + threadIdx.x; first < runs; first += step) {
    u32x4 g[kRuns], u[kRuns];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kWide;
      g[j] = i < runs ? load_run<kStream>(gate + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      u[j] = i < runs ? load_run<kStream>(up + 8 * i) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kWide;
      if (i >= runs) continue;
      const u32x4 v = product8<kAct>(g[j], u[j]);
      if (h) *(u32x4 *)(h + 8 * i) = v;
      if (codes) {
        float block;
        const act8_u32x2 c = encode_block(v, block);
        *(act8_u32x2 *)(codes + 8 * i) = c;
        if ((i & 7) == 0) scale[i >> 3] = block;
      }
    }
  }
}

template <Activation kAct, bool kStream>
__global__ __launch_bounds__(kWide) void gated_act_bwd(const uint16_t *dh, const uint16_t *gate, const uint16_t *up,
                                                         int64_t runs, uint16_t *dgate, uint16_t *dup) {
  const int64_t step = (int64_t)gridDim.x * (kWide * kRuns);
  for (int64_t first = (int64_t)blockIdx.x * (kWide * kRuns) + threadIdx.x; first < runs; first += step) {
    u32x4 d[kRuns], g[kRuns], u[kRuns];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kWide;
      d[j] = i < runs ? load_run<kStream>(dh + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      g[j] = i < runs ? load_run<kStream>(gate + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      u[j] = i < runs ? load_run<kStream>(up + 8 * i) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kWide;
      if (i >= runs) continue;
      u32x4 dg, du;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t dp = d[j][w], gp = g[j][w], up2 = u[j][w];
        float v0, v1, s0, s1;
        gate_act_slope<kAct>(bf16_lo(gp), v0, s0);
        gate_act_slope<kAct>(bf16_hi(gp), v1, s1);
        dg[w] = pack_bf16x2(bf16_lo(dp) * bf16_lo(up2) * s0, bf16_hi(dp) * bf16_hi(up2) * s1);
        du[w] = pack_bf16x2(bf16_lo(dp) * v0, bf16_hi(dp) * v1);
      }
      *(u32x4 *)(dgate + 8 * i) = dg;
      *(u32x4 *)(dup + 8 * i) = du;
    }
  }
}

// Eight values of gate (v[0], v[1]) and of up (v[2], v[3]) to `out`.
template <Activation kAct>
__device__ __forceinline__ void finish8(const GatedOut &out, int64_t to, const f32x4 (&v)[4]) {
  u32x4 h, g, u;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float g0 = v[k][2 * q], g1 = v[k][2 * q + 1], u0 = v[2 + k][2 * q], u1 = v[2 + k][2 * q + 1];
      h[2 * k + q] = pack_bf16x2(gate_act_of_sum<kAct>(g0) * u0, gate_act_of_sum<kAct>(g1) * u1);
      g[2 * k + q] = pack_bf16x2(g0, g1);
      u[2 * k + q] = pack_bf16x2(u0, u1);
    }
  store_gated(out, to, h, g, u);
}

// The same from the few-token form's fp32 results part[z][T][2 N], added in order; 8 columns a thread.
template <Activation kAct>
__global__ __launch_bounds__(kWide) void gated_reduce(const float *__restrict__ part, int parts, int64_t T, int64_t N,
                                                        GatedOut out) {
  const int64_t zs = 2 * T * N;
  const uint32_t row_runs = (uint32_t)(N / 8), runs = (uint32_t)T * row_runs;  // at most 2^26
  for (uint32_t i = blockIdx.x * kWide + threadIdx.x; i < runs; i += gridDim.x * kWide) {
    const uint32_t row = i / row_runs;
    const float *p = part + row * (2 * N) + 8 * (i - row * row_runs);
    f32x4 v[4] = {};
#pragma unroll 4
    for (int z = 0; z < parts; ++z)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f32x4 a = *(const f32x4 *)(p + z * zs + (k >> 1) * N + 4 * (k & 1));
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k][q] += a[q];
      }
    finish8<kAct>(out, 8 * (int64_t)i, v);
  }
}

// ---- many tokens: decoded weights in the workspace, plain tiles ------------------------------------------------
// The fused GEMM decodes a weight tile once for every 256 tokens; from some hundred tokens on (769 of two 11008 x 4096 weights),
// decoding each weight once (2.5 bytes a weight at HBM speed) and multiplying on plain 256 x 256 tiles is faster: 2048 of two
// 11008 x 4096 weights 342 us (the decode 40, 5.6 TB/s; the tiles 303; u 15), fused 407; 4096 tokens of 22016 x 8192 2.25 ms (the
// decode 163 us; the tiles 2.05 ms, 1.45 PFLOP/s), fused 2.98.  Matrix instructions bound the tiles, at the clock that the card's
// power leaves them (a library product of 4096 x 8192 x 44032 runs at 1.5 PFLOP/s).

// What the tiles need beside x, in one launch, whose workgroups take one of two parts:
//   the adapter's operands, whose contraction is the ranks of both members in turn, padded with zeros to `pad`:
//     bp [2 N][pad] (gate's rows hold B_0 at columns 0 .., up's B_1 at r ..), and where 2 r is not whole 64s
//     up [T][pad] from u [T][2 r];
//   the weights, 8 values a thread and pass.
// (u = x A_set^T beside the decode gains nothing: its loads then wait for the decode's stores, 43 + 21 us apart
// and 68 together at 2048 tokens of 2 x 11008 x 4096.)
struct GatedPrep {
  const uint16_t *u, *B[2];
  QWeight w[2];
  int64_t T, N, chunks;  // chunks: of 8 values of a weight
  int r, pad, packs;     // packs: workgroups of the first part
  uint16_t *up, *bp, *wd;
};

__device__ __forceinline__ void prep_pack(const GatedPrep &a) {
  const int per = a.pad / 8;
  const uint32_t i = blockIdx.x * kWide + threadIdx.x;  // (rows and tokens below 2^24, per at most 64)
  const int64_t row = i / (uint32_t)per;
  if (row >= 2 * a.N + (a.up ? a.T : 0)) return;
  const bool token = row >= 2 * a.N;
  const int member = !token && row >= a.N ? 1 : 0;
  const int c = (int)(i - (uint32_t)row * per) * 8, width = token ? 2 * a.r : a.r, first = c - member * a.r;
  const uint16_t *src = token ? a.u + (row - 2 * a.N) * width : a.B[member] + (row - member * a.N) * a.r;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (first >= 0 && first + 8 <= width) {
    v = load8(src + first);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (first + j >= 0 && first + j < width) v[j >> 1] |= (uint32_t)src[first + j] << (16 * (j & 1));
  }
  *(u32x4 *)((token ? a.up + (row - 2 * a.N) * a.pad : a.bp + row * a.pad) + c) = v;
}

template <bool kDQ>
__global__ __launch_bounds__(kWide) void gated_prep(GatedPrep a, Codebook cb) {
  __shared__ float lut[16];
  if ((int)blockIdx.x < a.packs) {
    prep_pack(a);
    return;
  }
  if (threadIdx.x < 16) lut[threadIdx.x] = cb.v[threadIdx.x];
  __syncthreads();
  const int64_t id = (int64_t)blockIdx.x - a.packs, groups = (int64_t)gridDim.x - a.packs;
  constexpr int kDeep = 4;
  const int64_t passes = (a.chunks + kDeep * kWide - 1) / (kDeep * kWide);  // of one weight
  const float mu0 = kDQ ? *a.w[0].mu : 0.f, mu1 = kDQ ? *a.w[1].mu : 0.f;
  for (int64_t pass = id; pass < 2 * passes; pass += groups) {
    const int m = pass >= passes ? 1 : 0;
    const QWeight &w = a.w[m];
    const float mu = m ? mu1 : mu0;
    const int64_t first = (pass - m * passes) * (kDeep * kWide) + threadIdx.x;
    uint32_t code[kDeep];
    float c1[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int64_t c = min(first + j * kWide, a.chunks - 1);
      code[j] = ((const uint32_t *)w.codes)[c];
      c1[j] = kDQ ? decode_constant(w.fp8[c >> 3], w.s2[c >> 11], mu) : w.s2[c >> 3];
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int64_t c = first + j * kWide;
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = pack_bf16x2(decode_product(lut[(code[j] >> (8 * i)) & 15u], c1[j]),
                           decode_product(lut[(code[j] >> (8 * i + 4)) & 15u], c1[j]));
      if (c < a.chunks) *(u32x4 *)(a.wd + ((int64_t)m * a.chunks + c) * 8) = v;
    }
  }
}

constexpr int kGatedPitch = 144;  // bytes of a token's 64 columns in LDS, with 16 of padding
struct GatedTilesArgs {
  const uint16_t *x, *u, *w, *b;  // u [T][pad]; decoded w [2 N][K], b [2 N][pad]: gate's rows, then up's
  int64_t T, N, K;
  int pad, nleft, ntoken, full, tail, steps;  // steps: of a tail tile's range
  float scale;
  float *part;  // [range][tail tile][256 tokens][256]
};

// One 256 x 256 tile: 128 columns of gate and of up, 16 rows of each in turn, by 256 tokens.  Of a lane's
// accumulators acc[2 j] is gate and acc[2 j + 1] up of the same token and 4 columns, and a wave's 64 columns are
// one block of the codes.
__global__ __launch_bounds__(kThreads, 2) void gated_tiles(GatedTilesArgs a, GatedOut out) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int id = blockIdx.x, over = id - a.full;
  const bool split = over >= 0;
  const int tail_tile = split ? over % a.tail : 0, range = split ? over / a.tail : 0;
  const Tile tile = tile_at(split ? a.full + tail_tile : place_of(id, a.full), a.nleft, a.ntoken);
  const int64_t t0 = (int64_t)tile.token * kTileT, d0 = (int64_t)tile.left * (kTileV / 2);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) & 1, wn = (wave & 1) + 2 * (wave >> 2);
  const int last_col = (int)min((int64_t)(kTileV / 2), a.N - d0) - 1, last_token = (int)min((int64_t)kTileT, a.T - t0) - 1;
  f32x4 acc[8][4];
  tile_zero(acc);
  const int all_steps = (int)(a.K / kStep), first = split ? range * a.steps : 0;
  const int steps = split ? min(a.steps, all_steps - first) : all_steps;
  for (int half = range == 0 ? 0 : 1; half < 2; ++half) {  // the adapter's ranks (the first range's), then n_in
    const uint32_t row_bytes = 2u * (uint32_t)(half ? a.K : (int64_t)a.pad);
    Operands o;
    o.left = uniform(half ? a.w + d0 * a.K + first * kStep : a.b + d0 * a.pad);
    o.right = uniform(half ? a.x + t0 * a.K + first * kStep : a.u + t0 * a.pad);
    o.left_step = o.right_step = 2 * kStep;
    o.left_pitch = 0;
    o.left_rows = 0;
    const uint32_t up = (uint32_t)a.N * row_bytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (2 * wave + (i & 1)) * 8 + (lane >> 3), v = 128 * (r >> 6) + 64 * (i >> 1) + (r & 63);
      const int col = min(64 * (v >> 7) + 16 * ((v >> 5) & 3) + (v & 15), last_col);
      o.left_off[i] = (uint32_t)col * row_bytes + ((v >> 4) & 1 ? up : 0u) + (((lane & 7) ^ swizzle_rows(r)) << 4);
      const int rt = (4 * wave + i) * 8 + (lane >> 3);
      o.right_off[i] = (uint32_t)min(rt, last_token) * row_bytes + (((lane & 7) ^ swizzle_rows(rt)) << 4);
    }
    product<false, false>(o, half ? steps : a.pad / kStep, lds, nullptr, false, acc);
    if (half == 0) {
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][n][q] *= a.scale;
    }
  }
  if (split) {
    float *dst = a.part + ((int64_t)range * a.tail + tail_tile) * (kTileT * kTileV);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int m = 0; m < 8; ++m)
        *(f32x4 *)(dst + (64 * wn + 16 * n + (lane & 15)) * kTileV + 128 * wm + 16 * m + 4 * (lane >> 4)) = acc[m][n];
    return;
  }
  if (d0 + 64 * wm >= a.N) return;
  // A wave's 64 tokens by 64 columns go through its own part of the LDS, so that rows are written 128 bytes at a
  // time: first h, then gate and up.
  char *mine = lds + wave * (2 * kStage / 8);
  auto put = [&](auto value) {  // value(m pair, n, q): bf16 pairs of columns 16 j + 4 (lane / 16) + 2 p ..
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(uint2 *)(mine + (16 * n + (lane & 15)) * kGatedPitch + 32 * j + 8 * (lane >> 4)) =
            make_uint2(value(j, n, 0), value(j, n, 2));
  };
  auto each_row = [&](auto f) {  // f(element of the outputs, the run's 8 values), 8 lanes a token
    TILE_WAIT_LDS();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 8 * i + (lane >> 3);
      const u32x4 v = *(const u32x4 *)(mine + t * kGatedPitch + 16 * (lane & 7));
      if (64 * wn + t <= last_token) f((t0 + 64 * wn + t) * a.N + d0 + 64 * wm + 8 * (lane & 7), v);
    }
    TILE_WAIT_LDS();
  };
  with_activation(out.act, [&](auto act) {
    put([&](int j, int n, int q) {
      return pack_bf16x2(gate_act_of_sum<act()>(acc[2 * j][n][q]) * acc[2 * j + 1][n][q],
                         gate_act_of_sum<act()>(acc[2 * j][n][q + 1]) * acc[2 * j + 1][n][q + 1]);
    });
  });
  each_row([&](int64_t to, const u32x4 &v) {
    if (out.h) *(u32x4 *)(out.h + to) = v;
    if (out.codes) {
      float block;
      const act8_u32x2 c = encode_block(v, block);
      *(act8_u32x2 *)(out.codes + to) = c;
      if ((lane & 7) == 0) out.scale[to >> 6] = block;
    }
  });
  if (!out.gate) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    put([&](int j, int n, int q) { return pack_bf16x2(acc[2 * j + k][n][q], acc[2 * j + k][n][q + 1]); });
    uint16_t *dst = k ? out.up : out.gate;
    each_row([&](int64_t to, const u32x4 &v) { *(u32x4 *)(dst + to) = v; });
  }
}

// h (and what else `out` names) of tail tiles from their ranges' fp32 tiles, added in order; 8 columns a thread.  kPlain:
// tiles of gated_tiles (128 columns, 16 of gate and 16 of up in turn), otherwise of the fused GEMM (64 columns of gate,
// then of up).
template <Activation kAct, bool kPlain>
__global__ __launch_bounds__(kWide) void gated_tail(const float *__restrict__ part, GatedRounds rounds, int nleft,
                                                   int ntoken, int64_t T, int64_t N, GatedOut out) {
  constexpr int kCols = kPlain ? 128 : 64, kRow = 2 * kCols, kRunsRow = kCols / 8;
  constexpr int kTile = 256 * kRow;
  const int64_t i = (int64_t)blockIdx.x * kWide + threadIdx.x;
  const int tail_tile = (int)(i / (256 * kRunsRow)), in = (int)(i % (256 * kRunsRow));
  const int t = in / kRunsRow, c = 8 * (in % kRunsRow);
  int64_t token, col;
  if (kPlain) {
    const Tile tile = tile_at(rounds.full + tail_tile, nleft, ntoken);
    token = (int64_t)tile.token * 256 + t;
    col = (int64_t)tile.left * kCols + c;
  } else {
    const int tile = rounds.full + tail_tile, left = tile / ntoken;
    token = (int64_t)(tile - left * ntoken) * 256 + t;
    col = (int64_t)left * kCols + c;
  }
  if (token >= T || col >= N) return;
  const int at = kPlain ? 128 * (c >> 6) + 32 * ((c >> 4) & 3) + (c & 15) : c, up = kPlain ? 16 : kCols;
  const float *p = part + (int64_t)tail_tile * kTile + t * kRow + at;
  f32x4 v[4] = {};
#pragma unroll 2
  for (int z = 0; z < rounds.splits; ++z)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x4 a = *(const f32x4 *)(p + (int64_t)z * rounds.tail * kTile + (k >> 1) * up + 4 * (k & 1));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[k][q] += a[q];
    }
  finish8<kAct>(out, token * N + col, v);
}

template <bool kPlain>
void launch_tail(const float *part, const GatedRounds &rounds, int nleft, int ntoken, int64_t T, int64_t N,
                 const GatedOut &out, hipStream_t st) {
  with_activation(out.act, [&](auto a) {
    gated_tail<a(), kPlain><<<(unsigned)(rounds.tail * (kPlain ? 16 : 8)), kWide, 0, st>>>(part, rounds, nleft, ntoken, T, N,
                                                                                        out);
  });
}

// Tiles of `steps` steps in rounds of 256 workgroups: whole ones and, where that is faster, the last in ranges.
// round_us + step_us steps: a workgroup's time, of which `fixed` stays in a round that leaves CUs idle.
GatedRounds gated_rounds(int64_t tiles, int64_t steps, double round_us, double step_us, double fixed,
                         int64_t tile_bytes, double *us) {
  auto rounds_us = [&](int64_t groups, int64_t n) {
    const double idle = groups % 256 ? 1.0 - (double)(groups % 256) / 256 : 0.0;
    return ((double)cdiv(groups, 256) - idle * (1.0 - fixed)) * (round_us + step_us * n);
  };
  GatedRounds best{(int)tiles, 0, 0, 0};
  *us = rounds_us(tiles, steps);
  const int64_t full = tiles / 256 * 256, tail = tiles - full;
  for (int64_t s = 2; tail && s <= 16 && steps / s >= 4; ++s) {
    const int64_t range = cdiv(steps, s), splits = cdiv(steps, range);
    // the fp32 tiles are written beside the other ranges' products and read at 6 TB/s, by one launch more
    const double t = rounds_us(full, steps) + rounds_us(tail * splits, range) +
                     (double)(tail * splits * tile_bytes) / 6e6 + 4.0;
    if (t < *us) {
      *us = t;
      best = GatedRounds{(int)full, (int)tail, (int)splits, range};
    }
  }
  return best;
}

// The two forms' times in us, fitted to 509 to 4096 tokens of n_ff x n_in = 5504 x 2048, 11008 x 4096 and 22016 x 8192:
// within 10%, and the faster form at these sizes.  The adapter's ranks do not enter (a step for 32 of
// them in either form, and the decoded form's packed operands), so where they outweigh n_in the other form may be faster.
// (The plain tiles run at the card's power limit: a round of fewer is faster.)  Fused and decoded: 5504 x 2048 1024 tokens 76
// and 62, 2048 tokens 123 and 110; 11008 x 4096 509 tokens 124 and 127, 1024 tokens 210 and 199; 22016 x 8192 509 tokens 386 and
// 488, 1024 tokens 740 and 722.
constexpr double kFusedRound = 5.0, kFusedStep = 0.98, kPlainRound = 7.0, kPlainStep = 1.235;
constexpr int64_t kFusedTile = 256 * 128 * 4, kPlainTile = 256 * 256 * 4;
double fused_us(int64_t T, int64_t N, int64_t K, GatedRounds *rounds) {
  double us;
  *rounds = gated_rounds(cdiv(T, 256) * (N / 64), K / 64, kFusedRound, kFusedStep, 1.0, kFusedTile, &us);
  return 14.0 + us;
}
double plain_us(int64_t T, int64_t N, int64_t K, GatedRounds *rounds) {
  double us;
  *rounds = gated_rounds(cdiv(N, kTileV / 2) * cdiv(T, kTileT), K / 64, kPlainRound, kPlainStep, 0.3, kPlainTile, &us);
  return 20.0 + us + 5.0 * (double)N * K / 5.1e6;
}

// The columns of the decoded form's adapter operands: the ranks of both members, in whole steps.
int64_t padded_ranks(int r) { return cdiv(2 * r, kStep) * kStep; }

// Whether the decoded form is taken.
bool decode_pays(int64_t T, int64_t N, int64_t K, int r) {
  // offsets within a tile, from its first row of gate to its last of up, stay below 2^32 in the weights and in the
  // adapter's operands (of 512 columns they would not at the largest n_ff), and the threads of the launches; the
  // decoded weights below 2 GB
  if (N * K > (int64_t)1 << 29 || K > 65536 || T > (int64_t)1 << 22) return false;
  if ((N + kTileV / 2) * padded_ranks(r) * 2 > (int64_t)1 << 32) return false;
  GatedRounds rounds;
  return 1.03 * plain_us(T, N, K, &rounds) < fused_us(T, N, K, &rounds);
}

// One pass of a workgroup each, up to 2^22 of them.
unsigned grid(int64_t runs) {
  return (unsigned)std::min<int64_t>((runs + kWide * kRuns - 1) / (kWide * kRuns), (int64_t)1 << 22);
}

}  // namespace

hipError_t launch_gated_act_fwd(const uint16_t *gate, const uint16_t *up, int64_t T, int64_t N, Activation act,
                                uint16_t *h, int8_t *codes, float *scale, hipStream_t st) {
  const int64_t runs = T * N / 8;
  with_activation(act, [&](auto a) {
    if (T * N * 4 >= kStreamBytes)
      gated_act_fwd<a(), true><<<grid(runs), kWide, 0, st>>>(gate, up, runs, h, codes, scale);
    else
      gated_act_fwd<a(), false><<<grid(runs), kWide, 0, st>>>(gate, up, runs, h, codes, scale);
  });
  return hipGetLastError();
}

hipError_t launch_gated_act_bwd(const uint16_t *dh, const uint16_t *gate, const uint16_t *up, int64_t T, int64_t N,
                                Activation act, uint16_t *dgate, uint16_t *dup, hipStream_t st) {
  const int64_t runs = T * N / 8;
  with_activation(act, [&](auto a) {
    if (T * N * 6 >= kStreamBytes)
      gated_act_bwd<a(), true><<<grid(runs), kWide, 0, st>>>(dh, gate, up, runs, dgate, dup);
    else
      gated_act_bwd<a(), false><<<grid(runs), kWide, 0, st>>>(dh, gate, up, runs, dgate, dup);
  });
  return hipGetLastError();
}

GatedPlan plan_linear_gated(int64_t T, int64_t N, int64_t K, int r) {
  GatedPlan p{};
  p.T = T;
  p.N = N;
  p.K = K;
  p.r = r;
  p.few = T <= kGatedFewTokens;
  p.parts = p.few ? gated_few_parts(T, N, K) : 0;
  p.decode = !p.few && decode_pays(T, N, K, r);
  size_t tail = 0;
  if (!p.few) {
    p.decode ? plain_us(T, N, K, &p.rounds) : fused_us(T, N, K, &p.rounds);
    tail = (size_t)p.rounds.tail * p.rounds.splits * (p.decode ? kPlainTile : kFusedTile);
  }
  size_t off = 256;
  p.off_u = off;
  off += align256((size_t)T * 2 * r * 2);
  p.own_u = gated_own_u(T, K, r);
  p.off_part = off;
  off += p.own_u ? 0 : align256(lora_part_floats(T, 2 * r, K) * 4);
  p.off_xp = off;
  off += p.few ? align256(gated_few_xp_values(T, K) * 2) : 0;
  p.off_h = off;  // h, where the one pass writes it and only its codes are wanted
  off += p.few && !p.parts ? align256((size_t)T * N * 2) : 0;
  p.off_qpart = off;
  off += align256(std::max((size_t)p.parts * T * 2 * N * 4, tail));
  // the decoded form: both weights, the adapter's operands (u as it is where its ranks need no padding)
  const size_t pad = (size_t)padded_ranks(r);
  p.off_w = off;
  off += p.decode ? align256((size_t)2 * N * K * 2) : 0;
  p.off_b = off;
  off += p.decode ? align256((size_t)2 * N * pad * 2) : 0;
  p.off_up = off;
  off += p.decode && pad != (size_t)2 * r ? align256((size_t)T * pad * 2) : 0;
  p.total = off;
  return p;
}

hipError_t launch_linear_gated_fwd(const GatedPlan &p, const uint16_t *x, const QWeight *w, const uint16_t *A_set,
                                   const uint16_t *const *B, float scale, const GatedOut &out, uint16_t *u_out,
                                   char *ws, const Codebook &cb, hipStream_t st) {
  uint16_t *u = u_out ? u_out : (uint16_t *)(ws + p.off_u);
  float *part = (float *)(ws + p.off_part), *qpart = (float *)(ws + p.off_qpart);
  hipError_t e = hipSuccess;
  if (!p.own_u)
    e = launch_lora(LoraKind::kU, x, p.K, A_set, p.K, p.T, 2 * p.r, p.K, 1.0f, u, part, st);
  else if (!p.few)
    e = launch_gated_u(p.T, x, A_set, p.K, p.r, u, st);
  if (e != hipSuccess) return e;
  if (p.few) {
    GatedOut first = out;
    if (!p.parts) {
      first.codes = nullptr;
      if (!out.h) first.h = (uint16_t *)(ws + p.off_h);
    }
    e = launch_gated_few(p.T, x, w, A_set, B, p.r, scale, first, u, (uint16_t *)(ws + p.off_xp), qpart, cb, st);
    if (e != hipSuccess) return e;
    if (p.parts) {
      const int64_t blocks = cdiv(p.T * p.N / 8, kWide);
      with_activation(out.act, [&](auto a) {
        gated_reduce<a()><<<(unsigned)std::min<int64_t>(blocks, 2048), kWide, 0, st>>>(qpart, p.parts, p.T, p.N, out);
      });
      return hipGetLastError();
    }
    return out.codes ? launch_act8_encode(first.h, p.T, p.N, out.codes, out.scale, st) : hipSuccess;
  }
  if (p.decode) {
    const int pad = (int)padded_ranks(p.r);
    GatedPrep g{};
    g.u = u;
    for (int i = 0; i < 2; ++i) {
      g.B[i] = B[i];
      g.w[i] = w[i];
    }
    g.T = p.T;
    g.N = p.N;
    g.chunks = p.N * p.K / 8;
    g.r = p.r;
    g.pad = pad;
    g.up = pad != 2 * p.r ? (uint16_t *)(ws + p.off_up) : nullptr;
    g.bp = (uint16_t *)(ws + p.off_b);
    g.wd = (uint16_t *)(ws + p.off_w);
    g.packs = (int)cdiv((2 * p.N + (g.up ? p.T : 0)) * (pad / 8), kWide);
    const unsigned blocks = (unsigned)(g.packs + std::min<int64_t>(cdiv(2 * g.chunks, 4 * kWide), 4096));
    TimedLaunch tl;  // the decode and the product
    const bool timed = timing_begin(st, tl, kTimedQgemmFwd);
    if (w[0].dq)
      gated_prep<true><<<blocks, kWide, 0, st>>>(g, cb);
    else
      gated_prep<false><<<blocks, kWide, 0, st>>>(g, cb);
    const int nleft = (int)cdiv(p.N, kTileV / 2), ntoken = (int)cdiv(p.T, kTileT);
    const GatedRounds &n = p.rounds;
    const GatedTilesArgs a{x,     g.up ? g.up : u, g.wd,   g.bp,   p.T,          p.N,   p.K,  pad,
                           nleft, ntoken,          n.full, n.tail, (int)n.steps, scale, qpart};
    gated_tiles<<<(unsigned)(n.full + n.tail * n.splits), kThreads, 0, st>>>(a, out);
    if (timed) timing_end(st, tl);
    if (n.tail) launch_tail<true>(qpart, n, nleft, ntoken, p.T, p.N, out, st);
    return hipGetLastError();
  }
  QgemmSet s{};
  for (int i = 0; i < 2; ++i) {
    s.m[i].w = w[i];
    s.m[i].lb = B[i];
  }
  TimedLaunch tl;
  const bool timed = timing_begin(st, tl, kTimedQgemmFwd);
  e = launch_qgemm_gated(s, p.T, x, u, p.r, scale, p.rounds, out, qpart, cb, st);
  if (timed) timing_end(st, tl);
  if (e != hipSuccess) return e;
  if (p.rounds.tail) launch_tail<false>(qpart, p.rounds, (int)(p.N / 64), (int)cdiv(p.T, 256), p.T, p.N, out, st);
  return hipGetLastError();
}

}  // namespace qlora
