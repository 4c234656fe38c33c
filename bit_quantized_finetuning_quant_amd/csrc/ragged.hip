// grad_x of linears whose sizes are not whole tiles of the fused GEMM (n_out not
// a multiple of 64 or n_in not of 128), or whose products are long, gfx950.
//
//   grad_x = sum_i dy_i W_hat_i + s v A
//
// The fused GEMM decodes W tile by tile inside the product; off its full-tile
// grid it carries every tile through registers with masks and runs at 60 to 70
// TFLOP/s (3284 tokens, 4 x 837 x 6144: 1989 us).  Here the operands are laid
// out whole instead, once per call in the workspace: the adapter rows A and then
// every member's decoded rows, each padded with zero rows to a multiple of 64,
// and beside them [v | dy_0 | dy_1 ..] with zero columns in the same places.
// Then the sum is one product over all rows on plain full tiles: the adapter
// steps come first and their sum is scaled in fp32.
// Decoding costs 2.5 bytes a weight at HBM speed, read again by the product; the
// product then runs at 1.36 PFLOP/s where its tiles fill the CUs, against 0.9 to
// 1.0 with the decode inside.  So long products on whole tiles are taken here too
// (long_pays).

#include <algorithm>

#include "launch.hpp"
#include "tile.hpp"

namespace qlora {

namespace {

constexpr int64_t kMaxDecoded = (int64_t)256 << 20;  // values of the decoded rows; above it the fused GEMM stays

int pad64(int64_t n) { return (int)((n + 63) / 64 * 64); }

// The padded layout: rows (of the weights) and columns (of the gradients) alike.
struct RaggedLayout {
  int count, T, K, rank, rank_pad, total;  // rank: of all members; total: rows in all
  int first[kMaxSetMembers], N[kMaxSetMembers];
  const uint16_t *dy[kMaxSetMembers];
};

// Workgroups below T: row t of [v | dy_0 | ..], eight columns a thread.  The rest: one row of the
// weights each that is not a decoded one (adapter rows, and zeros).
__global__ __launch_bounds__(256) void ragged_pack(RaggedLayout l, const uint16_t *__restrict__ v,
                                                   const uint16_t *__restrict__ A, uint16_t *__restrict__ dyp,
                                                   uint16_t *__restrict__ wp) {
  if ((int)blockIdx.x < l.T) {
    const int64_t t = blockIdx.x;
    for (int c0 = 8 * threadIdx.x; c0 < l.total; c0 += 2048) {
      const uint16_t *src = v + t * l.rank;
      int n = l.rank, c = c0;
      for (int i = 0; i < l.count; ++i)
        if (c0 >= l.first[i]) {
          src = l.dy[i] + t * l.N[i];
          n = l.N[i];
          c = c0 - l.first[i];
        }
      u32x4 x = {0u, 0u, 0u, 0u};
      if (c + 8 <= n) {
        x = load8(src + c);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t value = c + j < n ? src[c + j] : 0u;
          x[j >> 1] |= value << (16 * (j & 1));
        }
      }
      *(u32x4 *)(dyp + t * l.total + c0) = x;
    }
    return;
  }
  // the j-th such row: the adapter block, then the pads of the members in order
  int row = (int)blockIdx.x - l.T;
  const uint16_t *src = row < l.rank ? A + (int64_t)row * l.K : nullptr;
  if (row >= l.rank_pad) {
    int j = row - l.rank_pad;
    for (int i = 0; i < l.count; ++i) {
      const int end = i + 1 < l.count ? l.first[i + 1] : l.total, pad = end - l.first[i] - l.N[i];
      if (j < pad) {
        row = l.first[i] + l.N[i] + j;
        break;
      }
      j -= pad;
    }
  }
  for (int c = 8 * threadIdx.x; c < l.K; c += 2048)
    *(u32x4 *)(wp + (int64_t)row * l.K + c) = src ? *(const u32x4 *)(src + c) : u32x4{0u, 0u, 0u, 0u};
}

// One 256 x 256 tile (columns of grad_x, tokens) over one range of the rows: grad_x itself, or with more than one range
// part [range][tile][256 tokens][256 columns] fp32.  Bound by the matrix cores: 3284 tokens, 4 x 837 x 6144, 169 us (0.80
// PFLOP/s of the unpadded sizes, 1.2 rounds of workgroups); 4096 x 8192 x 22016, 1166 us (1.27).
__global__ __launch_bounds__(kThreads, 2) void ragged_tiles(const uint16_t *__restrict__ dyp,
                                                            const uint16_t *__restrict__ wp, int T, int K, int rows,
                                                            int adapter, float scale, int nleft, int ntoken,
                                                            Split split, float *__restrict__ part,
                                                            uint16_t *__restrict__ out) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int tiles = nleft * ntoken;
  const int slot = place_of(blockIdx.x, tiles * split.count), nth = scalar(slot / tiles);
  const Tile tile = tile_at(slot - nth * tiles, nleft, ntoken);
  const int t0 = tile.token * kTileT, d0 = tile.left * kTileV;
  const int first = nth * split.range, last = min(first + split.range, rows);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) & 1, wn = (wave & 1) + 2 * (wave >> 2);
  Operands o;
  o.left_pitch = (uint32_t)K * 2u;
  o.left_step = (int64_t)kStep * K * 2;
  o.right_step = 2 * kStep;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (2 * wave + (i & 1)) * 8 + (lane >> 3);
    const int d = min(d0 + 128 * (r >> 6) + 64 * (i >> 1), K - 64) - d0;
    o.left_off[i] = (uint32_t)(2 * d) + (((lane & 7) ^ swizzle_cols(r & 63)) << 4);
    const int rt = (4 * wave + i) * 8 + (lane >> 3);
    o.right_off[i] = (uint32_t)min(rt, T - 1 - t0) * (uint32_t)(2 * rows) + (((lane & 7) ^ swizzle_rows(rt)) << 4);
  }
  f32x4 acc[8][4];
  tile_zero(acc);
  for (int half = 0; half < 2; ++half) {  // the adapter's rows of the range, then the weights'
    const int a = half ? max(first, adapter) : first, b = half ? last : min(last, adapter);
    if (a < b) {
      o.left = uniform(wp + (int64_t)a * K + d0);
      o.right = uniform(dyp + (int64_t)t0 * rows + a);
      o.left_rows = b - a;
      product<true, false>(o, (b - a) / kStep, lds, nullptr, false, acc);
    }
    if (half == 0 && a < b) {
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][n][q] *= scale;
    }
  }
  float *mine = part + (int64_t)slot * (kTileT * kTileV);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int t = 64 * wn + 16 * n + (lane & 15);
    if (t0 + t >= T) continue;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int d = 128 * wm + 16 * m + 4 * (lane >> 4);
      if (d0 + d >= K) continue;
      if (split.count > 1)
        *(f32x4 *)(mine + t * kTileV + d) = acc[m][n];
      else
        *(uint2 *)(out + (int64_t)(t0 + t) * K + d0 + d) =
            make_uint2(pack_bf16x2(acc[m][n][0], acc[m][n][1]), pack_bf16x2(acc[m][n][2], acc[m][n][3]));
    }
  }
}

// grad_x from the ranges' tiles, four columns a thread.  kWaves = 4: every wave takes a fourth of the ranges, so that the
// partial sums, from the caches of other XCDs, arrive in few round trips (109 tokens by 256 columns, 60 ranges: 19 ->
// 4.5 us; where one wave a quad fills the CUs it loses, 1500 by 1024, ten ranges: 80 -> 82 us in all).
template <int kWaves>
__global__ __launch_bounds__(256) void ragged_reduce(const float *__restrict__ part, int T, int K, int nleft,
                                                     int ntoken, int splits, uint16_t *__restrict__ out) {
  constexpr int kQuads = 256 / kWaves, kDeep = kWaves > 1 ? 8 : 1;
  __shared__ f32x4 sums[kWaves][kQuads];
  const int64_t quads = (int64_t)T * K / 4, stride = (int64_t)nleft * ntoken * kTileT * kTileV;
  const int own = threadIdx.x % kQuads, wave = threadIdx.x / kQuads;
  for (int64_t i0 = (int64_t)blockIdx.x * kQuads; i0 < quads; i0 += (int64_t)gridDim.x * kQuads) {
    const int64_t i = min(i0 + own, quads - 1);
    const int t = (int)(i / (K / 4)), c = (int)(i % (K / 4)) * 4;
    const float *p = part + (int64_t)place_at(Tile{c / kTileV, t / kTileT}, nleft, ntoken) * (kTileT * kTileV) +
                     t % kTileT * kTileV + c % kTileV;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    auto add = [&s](const f32x4 &x) {
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += x[q];
    };
#pragma unroll kDeep
    for (int k = wave; k < splits; k += kWaves) add(*(const f32x4 *)(p + k * stride));
    if constexpr (kWaves > 1) {
      sums[wave][own] = s;
      __syncthreads();
#pragma unroll
      for (int w = 1; w < kWaves; ++w) add(sums[w][own]);  // of use in the first wave
      __syncthreads();
    }
    if (wave == 0 && i0 + own < quads)
      *(uint2 *)(out + (int64_t)t * K + c) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
  }
}

// Up to 64 tokens: 64 columns over one chunk of the rows; part [chunk][T][K] fp32.
template <int NT>
__global__ __launch_bounds__(kFewThreads, 1) void ragged_few(const uint16_t *__restrict__ dyp,
                                                             const uint16_t *__restrict__ wp, int T, int K, int rows,
                                                             int adapter, float scale, int chunk_steps, int chunks,
                                                             float *__restrict__ part, uint16_t *__restrict__ out) {
  constexpr int kBytes = few_stages<true, NT>() * few_stage<NT>();
  __shared__ __attribute__((aligned(1024))) char lds[4 * kBytes];
  const int slices = K / 64;
  const int chunk = scalar((int)blockIdx.x / slices), slice = (int)blockIdx.x - chunk * slices;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = chunk * chunk_steps, last = min(first + chunk_steps, rows / kStep);
  const int edge = min(max(adapter / kStep - first, 0), last - first);  // the chunk's adapter steps
  uint32_t off[2 * NT];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int r = 8 * j + (lane >> 3);
    off[j] = (uint32_t)min(r, T - 1) * (uint32_t)(2 * rows) + (((lane & 7) ^ swizzle_rows(r)) << 4);
  }
  const char *left = uniform(wp + (int64_t)first * kStep * K + 64 * slice), *right = uniform(dyp + first * kStep);
  char *mine = lds + wave * kBytes;
  f32x4 acc[4][NT];
  few_zero<NT>(acc);
  few_product<true, false, NT>(left, (uint32_t)K * 2u, edge * kStep, (int64_t)kStep * K * 2, right, off, wave, edge,
                               mine, nullptr, acc);
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][n][q] *= scale;
  // the wave's first step past the adapter's
  const int next = edge + ((wave - edge) & 3);
  few_product<true, false, NT>(left, (uint32_t)K * 2u, (last - first) * kStep, (int64_t)kStep * K * 2, right, off,
                               next, last - first, mine, nullptr, acc);
  float *red = (float *)lds;
  few_put<NT>(acc, red);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = i * 16 + (threadIdx.x >> 4), d = 4 * (threadIdx.x & 15);
    if (t >= T) continue;
    const f32x4 s = few_sum<NT>(red, t, d);
    if (chunks > 1)
      *(f32x4 *)(part + ((int64_t)chunk * T + t) * K + 64 * slice + d) = s;
    else
      *(uint2 *)(out + (int64_t)t * K + 64 * slice + d) =
          make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
  }
}

__global__ __launch_bounds__(256) void ragged_few_reduce(const float *__restrict__ part, int64_t n, int chunks,
                                                         uint16_t *__restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 s = *(const f32x4 *)(part + i);
#pragma unroll 8
  for (int k = 1; k < chunks; ++k) {
    const f32x4 x = *(const f32x4 *)(part + k * n + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += x[q];
  }
  *(uint2 *)(out + i) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

RaggedLayout layout_of(int64_t T, int count, const int64_t *N, int64_t K, int r) {
  RaggedLayout l{};
  l.count = count;
  l.T = (int)T;
  l.K = (int)K;
  l.rank = count * r;
  l.rank_pad = pad64(l.rank);
  l.total = l.rank_pad;
  for (int i = 0; i < count; ++i) {
    l.first[i] = l.total;
    l.N[i] = (int)N[i];
    l.total += pad64(N[i]);
  }
  return l;
}

// Chunks of the few-token form: about a workgroup a CU, at least a step for each of its waves.
int few_chunk_steps(const RaggedLayout &l) {
  const int steps = l.total / kStep;
  const int chunks = std::max(1, std::min(256 / (l.K / 64), (steps + 3) / 4));
  return (steps + chunks - 1) / chunks;
}

}  // namespace

// Whether a product on whole tiles is faster here than in the fused GEMM, both estimated in us from the rounds of 256
// workgroups that each takes: here 17.6 a round and 12.6 ns a row of a tile's range, the partial tiles, and the decode
// with the packed gradients at 4.1 TB/s; there 5.2 a round and 0.70 a step of 64 rows, and the splits' partial sums
// (fitted to the 81 shapes of 1024 to 8192 tokens by the linears and sets of 4096, 8192, 11008 and 22016).  This
// form holds the decoded weights in the workspace, so it is taken for a gain of 5% only.  Of the 81 none is then
// slower than in the fused GEMM, and the mean is 0.3% above the faster form's.  Measured, the whole backward pass
// of T x n_out x n_in (here / there): 4096 x 8192 x 22016 1354 / 1556 us, 4096 x 8192 x 8192 510 / 558, 4096 x 4096 x 11008
// 397 / 436, 2049 x 11008 x 4096 289 / 318, 2048 x 22016 x 8192 689 / 712; left to the fused GEMM: 2048 x (2 of 11008) x
// 4096 419 / 393, 2049 x (3 of 8192) x 8192 1210 / 1137, 2048 x 4096 x 4096 122 / 98, 1024 x 22016 x 8192 422 / 372.
static bool long_pays(int64_t T, int count, const int64_t *N, int64_t K, int64_t rows) {
  if (T < 1024) return false;
  const int tiles = (int)(cdiv(K, kTileV) * cdiv(T, kTileT));
  const Split s = choose_split(tiles, (int)rows);
  const double here = (double)cdiv((int64_t)tiles * s.count, 256) * (17.6 + 0.0126 * s.range) +
                      (s.count > 1 ? 0.051 * tiles * s.count : 0.0) + (2.5 * rows * K + 4.0 * T * rows) / 4.1e6;
  int64_t steps = 0;
  bool same_n = true;
  for (int i = 0; i < count; ++i) {
    steps += N[i] / kStep;
    same_n = same_n && N[i] == N[0];
  }
  QgemmSplit f{1, 0};  // a split takes the same range of steps of every member
  if (same_n) f = qgemm_split(T, K, N[0]);
  if (f.splits > 1) steps = f.steps * count;
  const double rounds = (double)cdiv(cdiv(T, 256) * (K / 128) * f.splits, 256);
  const double partial = f.splits > 1 ? 1.3 * (f.splits * (double)T * K / 1e6 + 3.0) : 0.0;
  return 1.05 * here < rounds * (5.2 + 0.70 * steps) + partial;
}

bool ragged_dx_applies(int64_t T, int count, const int64_t *N, int64_t K, int r) {
  bool whole = K % 128 == 0;
  int64_t rows = pad64((int64_t)count * r);
  for (int i = 0; i < count; ++i) {
    whole = whole && N[i] % 64 == 0;
    if (N[i] > kMaxDecoded || K > 65536) return false;
    rows += pad64(N[i]);
  }
  // a few tokens and rows: its own launches cost more than the masks (6 tokens, 2 x 100 x 512: 41 against
  // 47 us; 1 token, 4 x 200 x 512: 62 against 57)
  if (T <= kFewTokens && rows <= 512) return false;
  // T: ragged_pack takes a workgroup of 256 threads a token and a few more, and a launch holds fewer than 2^32 threads
  if (rows > kMaxDecoded / K || T > (int64_t)1 << 23 || rows * T > (int64_t)1 << 32) return false;
  return !whole || long_pays(T, count, N, K, rows);
}

// dyp, the weights' rows, and the partial sums, each 256-byte aligned
RaggedPlan plan_ragged_dx(int64_t T, int count, const int64_t *N, int64_t K, int r) {
  const RaggedLayout l = layout_of(T, count, N, K, r);
  RaggedPlan p{};
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  p.off_dy = take((size_t)T * l.total * 2);
  p.off_w = take((size_t)l.total * K * 2);
  if (T <= kFewTokens) {
    const int steps = few_chunk_steps(l), chunks = (l.total / kStep + steps - 1) / steps;
    p.off_part = take(chunks > 1 ? (size_t)chunks * T * K * 4 : 0);
  } else {
    const int tiles = (int)(cdiv(K, kTileV) * cdiv(T, kTileT)), splits = choose_split(tiles, l.total).count;
    p.off_part = take(splits > 1 ? (size_t)splits * tiles * kTileT * kTileV * 4 : 0);
  }
  p.total = off;
  return p;
}

template <int NT>
static void launch_ragged_few(const RaggedLayout &l, const uint16_t *dyp, const uint16_t *wp, int adapter, float scale,
                              float *part, uint16_t *out, hipStream_t st) {
  const int steps = few_chunk_steps(l), chunks = (l.total / kStep + steps - 1) / steps;
  ragged_few<NT><<<(unsigned)(chunks * (l.K / 64)), kFewThreads, 0, st>>>(dyp, wp, l.T, l.K, l.total, adapter, scale,
                                                                        steps, chunks, part, out);
  const int64_t n = (int64_t)l.T * l.K;
  if (chunks > 1) ragged_few_reduce<<<(unsigned)cdiv(n, 1024), 256, 0, st>>>(part, n, chunks, out);
}

hipError_t launch_ragged_dx(const RaggedPlan &p, int64_t T, int count, const int64_t *N, int64_t K, int r,
                            const uint16_t *const *dy, const QWeight *w, const uint16_t *v, const uint16_t *A_set,
                            float scale, uint16_t *out, char *ws, const Codebook &cb, hipStream_t st) {
  RaggedLayout l = layout_of(T, count, N, K, r);
  uint16_t *dyp = (uint16_t *)(ws + p.off_dy), *wp = (uint16_t *)(ws + p.off_w);
  float *part = (float *)(ws + p.off_part);
  DequantSet set{};
  set.count = count;
  int zero_rows = l.total - l.rank_pad;
  for (int i = 0; i < count; ++i) {
    l.dy[i] = dy[i];
    set.w[i] = w[i];
    set.out[i] = wp + (int64_t)l.first[i] * K;
    zero_rows -= l.N[i];
  }
  const hipError_t e = launch_dequantize_set(set, cb, st);
  if (e != hipSuccess) return e;
  ragged_pack<<<(unsigned)(l.T + l.rank_pad + zero_rows), 256, 0, st>>>(l, v, A_set, dyp, wp);
  if (T <= 16)
    launch_ragged_few<1>(l, dyp, wp, l.rank_pad, scale, part, out, st);
  else if (T <= 32)
    launch_ragged_few<2>(l, dyp, wp, l.rank_pad, scale, part, out, st);
  else if (T <= kFewTokens)
    launch_ragged_few<4>(l, dyp, wp, l.rank_pad, scale, part, out, st);
  else {
    const int nleft = (int)cdiv(K, kTileV), ntoken = (int)cdiv(T, kTileT);
    const Split split = choose_split(nleft * ntoken, l.total);
    ragged_tiles<<<(unsigned)(nleft * ntoken * split.count), kThreads, 0, st>>>(
        dyp, wp, l.T, l.K, l.total, l.rank_pad, scale, nleft, ntoken, split, part, out);
    const int64_t quads = T * K / 4;
    if (split.count >= 8 && quads <= 65536)
      ragged_reduce<4><<<(unsigned)std::min<int64_t>(cdiv(quads, 64), 4096), 256, 0, st>>>(part, l.T, l.K, nleft, ntoken,
                                                                                       split.count, out);
    else if (split.count > 1)
      ragged_reduce<1><<<(unsigned)std::min<int64_t>(cdiv(quads, 256), 2048), 256, 0, st>>>(part, l.T, l.K, nleft, ntoken,
                                                                                        split.count, out);
  }
  return hipGetLastError();
}

}  // namespace qlora
