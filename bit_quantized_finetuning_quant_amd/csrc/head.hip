// The loss of the language-model head over a large vocabulary, with the
// gradient of the hidden states, without ever holding the logits (gfx950).
//
//   l_tv  = sum_d h_td W_vd                      (bf16 operands, fp32 sums)
//   lse_t = log sum_v exp(l_tv),   loss_t = lse_t - l_t,y(t)
//   grad_h_t = c_t (sum_v p_tv W_v - W_y(t)),    p_tv = exp(l_tv - lse_t)
//
// The head is frozen, as every weight of this library, so there is no
// gradient for W.  Per piece of the vocabulary:
//
//   head_logits   one 256 x 256 tile of l per workgroup; its epilogue takes,
//                 per token and 128 words, an integer n above log2 e max l
//                 and writes e_tv = 2^(l log2 e - n) in bf16, s = sum e and
//                 r = sum of the written (rounded) e
//   head_fold     running N_t = max n, S_t = sum 2^(n - N) s and R_t likewise of r
//                 over the tiles, and the distance (N - n) / 64 of each tile, 0 to 3
//   head_grad     G_td += sum_v 2^(n - N) e_tv W_vd: the factor of a tile is a
//                 power of two, so it is one saturating subtraction from the
//                 exponent field of the bf16 operand, exact
//
// n is one of 44 + 64 i: bf16 has the exponents of fp32, so e loses nothing by
// lying up to 2^64 below 1, and the tiles of a token nearly always have the
// same n (where the largest logits of all its tiles lie between -13.8 and
// 30.5).  A workgroup of head_grad whose distances are all 0 subtracts nothing.
// What lies 2^-60 and more below a token's largest exponential may fall out of
// the range (its share of the loss is below the rounding of any other term,
// unless every other word is that unlikely).
//
// and head_finish forms grad_h = c (G - R W_y) / (R + e_y).  So the
// gradient needs the two products it cannot do without (4 T V D operations)
// and no second run over the logits.  The target's own term is kept out of e,
// S and R and added apart: 1 - p_y has no cancellation, and
// loss = log1p(S / e_y) keeps its relative precision for a token the
// model is sure of.  e is rounded to bf16 (half a step, 2^-8 of it) because the
// matrix cores take it in that type; S, of which loss and lse are made, sums the
// unrounded fp32 values.  The gradient takes R, so that its words' weights sum
// to what W_y is subtracted with: a token sure of another word than its target
// gets c p (W_word - W_y) within the rounding of that difference, also where the
// two rows are alike and most of it cancels (with S in R's place it was off by up
// to 2^-8 of W_word: 0.013 of the gradient at a cosine of 0.9, now 0.002).
//
// Tokens whose target is negative carry no loss.  A scan lists the others, the
// products gather their rows by that list, and tiles past its end do nothing.

#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "tile.hpp"

namespace qlora {

namespace {

constexpr int kStatV = 128;       // words that share one exponent n per token
constexpr int kMaxPiece = 32768;  // words of a piece: a range's distances fit 16 KB of LDS
constexpr int kFoldV = 8192;      // words up to which the products fold the tiles themselves
constexpr int64_t kFewMaxWords = (int64_t)1 << 20;
constexpr float kLog2e = 1.44269502162933349609375f;  // fl32(log2 e)
constexpr float kLn2 = 0.693147182464599609375f;      // fl32(ln 2), and the rest of it
constexpr float kLn2Lo = -1.90465429995776804525e-9f;
// |n| from which a row counts as overflown (its loss and gradient are NaN): below it integers and
// their differences are exact in fp32, and l log2 e - n is rounded once
constexpr float kMaxExponent = 4194304.0f;
constexpr float kNoExponent = -3.0e38f;  // n of a tile without any word

// ---------------------------------------------------------------------------

// loss and lse of a token that carries none: 0, or NaN for a target past the vocabulary.
__device__ __forceinline__ void no_loss(int64_t y, int64_t t, float *loss, float *lse) {
  const float v = y < 0 ? 0.f : NAN;
  loss[t] = v;
  if (lse) lse[t] = v;
}

// Lists the tokens of a chunk that carry a loss: rows[j] = token, place[token] = j, or -1 (ignored)
// or -2 (target out of range); these get their loss here.  One workgroup; state[0] |= 2 on a bad
// target, state[1] = the count.  5.3 us for 2048 tokens, latency.
__global__ __launch_bounds__(1024) void head_scan(const int64_t *__restrict__ target, int T, int64_t V, bool first,
                                                  int *__restrict__ rows, int *__restrict__ place,
                                                  uint32_t *__restrict__ state, float *__restrict__ loss,
                                                  float *__restrict__ lse) {
  __shared__ int wave_sum[16];
  __shared__ int any;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) any = 0;
  int base = 0;
  bool bad = false;
  for (int t0 = 0; t0 < T; t0 += 1024) {
    const int t = t0 + tid;
    const int64_t y = t < T ? target[t] : -1;
    const bool live = y >= 0 && y < V;
    bad |= y >= V;
    const uint64_t mask = __ballot(live);
    if (lane == 0) wave_sum[wave] = __popcll(mask);
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? wave_sum[w] : 0;
      all += wave_sum[w];
    }
    const int j = before + __popcll(mask & ((1ull << lane) - 1));
    if (t < T) {
      if (live) rows[j] = t;
      else no_loss(y, t, loss, lse);
      place[t] = live ? j : (y >= V ? -2 : -1);
    }
    base += all;
    __syncthreads();
  }
  if (bad) any = 1;
  __syncthreads();
  if (tid == 0) {
    state[0] = (first ? 0u : state[0]) | (any ? 2u : 0u);
    state[1] = (uint32_t)base;
  }
}

// The same for at most 512 tokens by every workgroup of head_logits (512 threads), which spares the
// launch: returns the count; this thread's token becomes entry j of the list, or j = -1.  The first
// workgroup writes what the later kernels read.
__device__ __forceinline__ int list_tokens(const int64_t *target, int T, int64_t V, int *wave_sum, int &j, int *rows,
                                           int *place, uint32_t *state, float *loss, float *lse) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t y = t < T ? target[t] : -1;
  const bool live = y >= 0 && y < V;
  const uint64_t mask = __ballot(live), bad = __ballot(y >= V);
  if (lane == 0) wave_sum[wave] = __popcll(mask) | (bad ? 1 << 16 : 0);
  __syncthreads();
  int before = 0, all = 0, any = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int n = wave_sum[w] & 0xFFFF;
    before += w < wave ? n : 0;
    all += n;
    any |= wave_sum[w] >> 16;
  }
  j = live ? before + __popcll(mask & ((1ull << lane) - 1)) : -1;
  if (blockIdx.x == 0) {
    if (t < T) {
      if (live) rows[j] = t;
      else no_loss(y, t, loss, lse);
      place[t] = live ? j : (y >= V ? -2 : -1);
    }
    if (t == 0) {
      state[0] = any ? 2u : 0u;
      state[1] = (uint32_t)all;
    }
  }
  return all;
}

// n of a tile from its largest logit.  Finite whatever the logits are: NaN and infinite sums show in s.
__device__ __forceinline__ float tile_exponent(float top) {
  return ceilf(fminf(fmaxf(top * kLog2e, -2.0f * kMaxExponent), 2.0f * kMaxExponent));
}
// The one of 44 + 64 i at or above m, and 2^(m - that).
__device__ __forceinline__ float coarse_exponent(float m, float &factor) {
  const float n = 64.0f * ceilf((m - 44.0f) * 0.015625f) + 44.0f;
  factor = __builtin_ldexpf(1.0f, (int)(m - n));
  return n;
}
// 2^(l log2 e - n).  log2 e is its fp32 value, 1.3e-8 of it too small, so all exponentials of a token belong
// to logits smaller by that much: 1.3e-8 of l - l_y in the ratios, of l in lse (fp32 has 6e-8).
__device__ __forceinline__ float relative_exp(float l, float n) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(l, kLog2e, -n));
}

// r + the two bf16 values of a word.
__device__ __forceinline__ float add_pair(uint32_t pair, float r) {
  constexpr uint32_t kOnes = 0x3F803F80u;
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, kOnes), r, false);
}

// 16 tokens (fragment n) by the wave's 128 words of a tile of the logits: e, n, s and r.  A NaN logit shows in
// s.  kTest: words past nvt are left out, and the token's target y (of this tile, or -1) goes to
// target_logit.  out, exponent, sum, target_logit: this lane's token (out: its first word, too).
template <bool kTest>
__device__ __forceinline__ void put_logits(const f32x4 (&acc)[8][4], int n, bool on, int y, int vl, int nvt,
                                           uint16_t *out, float *exponent, float *sum, float *rounded,
                                           float *target_logit) {
  const int lane = threadIdx.x & 63;
  float top = -INFINITY;
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float l = acc[m][n][q];
      top = fmaxf(top, !kTest || vl + 16 * m + q < nvt ? l : -INFINITY);
    }
  top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  // the exponentials are formed next to 1, where they are exact to 2^-24, and moved from there
  const float ex = tile_exponent(top);
  float factor, n_tile = coarse_exponent(ex, factor);
  if (kTest && (vl & ~127) >= nvt) n_tile = kNoExponent;
  float s = 0.f, r = 0.f, ly = 0.f;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    float p[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float l = acc[m][n][q];
      p[q] = relative_exp(l, ex) * factor;
      if (kTest) {
        const int v = vl + 16 * m + q;
        ly = v == y ? l : ly;
        p[q] = v == y || v >= nvt ? 0.f : p[q];
      }
      s += p[q];
    }
    if (out) {
      const uint2 v = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
      if (on) *(uint2 *)(out + 16 * m) = v;
      r = add_pair(v.y, add_pair(v.x, r));
    }
  }
  if (kTest && y >= 0 && (y & ~127) == (vl & ~127) && ((y >> 2) & 3) == (lane >> 4)) *target_logit = ly;
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if (out) {
    r += __shfl_xor(r, 16);
    r += __shfl_xor(r, 32);
  }
  if (lane < 16 && on) {
    *exponent = n_tile;
    *sum = s;
    if (out) *rounded = r;
  }
}

// One tile of the logits, see the top.  Bound by the matrix cores: of 4096 x 8192 x 16128 one launch takes 743 us
// (1.38 PFLOP/s of the tokens with a loss; MFMAs busy 81% of the cycles at the 1.6 GHz the chip runs under them; a
// library product of these operands alone reaches 1.45).  256 x 256 tiles, since a tile's operands then take a quarter
// of the LDS bandwidth that 128 x 128 would; the epilogue works on the accumulators where they are, so that the logits
// never leave the registers.
// e: [tokens][pitch] bf16 (nullptr: the loss alone, and no rounded); exponent, sum and rounded:
// [tile of 128 words][tpad].  kList: at most 512 tokens, listed here; otherwise head_scan has.
template <bool kList>
__global__ __launch_bounds__(kThreads, 2) void head_logits(
    const uint16_t *__restrict__ h, const uint16_t *__restrict__ w, const int64_t *__restrict__ target, int T, int64_t V,
    int64_t v0, int64_t nv, int D, int nleft, int *__restrict__ rows, int *__restrict__ place,
    uint32_t *__restrict__ state, float *__restrict__ loss, float *__restrict__ lse, uint16_t *__restrict__ e,
    int64_t pitch, float *__restrict__ exponent, float *__restrict__ sum, float *__restrict__ rounded, int64_t tpad,
    float *__restrict__ target_logit) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  __shared__ int list[kList ? kTileT : 1];
  int entry = -1;
  int live;
  if (kList)
    live = scalar(list_tokens(target, T, V, (int *)lds, entry, rows, place, state, loss, lse));
  else
    live = (int)state[1];
  const int ntoken = (live + kTileT - 1) / kTileT;
  if ((int)blockIdx.x >= nleft * ntoken) return;
  const Tile tile = tile_at(place_of(blockIdx.x, nleft * ntoken), nleft, ntoken);
  const int t0 = tile.token * kTileT;
  if (kList) {
    if (entry >= t0 && entry < t0 + kTileT) list[entry - t0] = threadIdx.x;
    __syncthreads();
  }
  auto token = [&](int j) { return kList ? list[j - t0] : rows[j]; };  // j in the tile
  const int64_t vt = (int64_t)tile.left * kTileV;  // within the piece
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) & 1, wn = (wave & 1) + 2 * (wave >> 2);
  const uint32_t row_bytes = (uint32_t)D * 2u;

  Operands o;
  o.left = uniform(w + vt * D);
  o.right = uniform(h);
  o.left_step = o.right_step = 2 * kStep;
  o.left_pitch = 0;
  o.left_rows = 0;
  const int last_v = (int)min((int64_t)kTileV, nv - vt) - 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // unit row (2 wave + i%2) 8 + lane/8: word 128 (row / 64) + 64 (i / 2) + row % 64
    const int r = (2 * wave + (i & 1)) * 8 + (lane >> 3);
    const int v = min(128 * (r >> 6) + 64 * (i >> 1) + (r & 63), last_v);
    o.left_off[i] = (uint32_t)v * row_bytes + (((lane & 7) ^ swizzle_rows(r)) << 4);
    const int rt = (4 * wave + i) * 8 + (lane >> 3);
    o.right_off[i] = (uint32_t)token(min(t0 + rt, live - 1)) * row_bytes + (((lane & 7) ^ swizzle_rows(rt)) << 4);
  }
  f32x4 acc[8][4];
  tile_zero(acc);
  product<false, false>(o, D / kStep, lds, nullptr, false, acc);

  // rows (words) of this lane: 128 wm + 16 m + 4 (lane / 16) + q
  const int vl = 128 * wm + 4 * (lane >> 4), nvt = last_v + 1;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int t = t0 + 64 * wn + 16 * n + (lane & 15);
    const bool on = t < live;
    const int64_t at = on ? target[token(t)] - v0 - vt : -1;  // the target's word, if it is one of this tile's
    const int y = at >= 0 && at < kTileV ? (int)at : -1;
    const int64_t stat = (int64_t)(2 * tile.left + wm) * tpad + t;
    uint16_t *out = e ? e + (int64_t)t * pitch + vt + vl : nullptr;
    // most waves hold no word past the vocabulary and no token's target: their values need no test
    if (nvt == kTileV && !__any(y >> 7 == wm))
      put_logits<false>(acc, n, on, -1, vl, nvt, out, exponent + stat, sum + stat, rounded + stat, nullptr);
    else
      put_logits<true>(acc, n, on, y, vl, nvt, out, exponent + stat, sum + stat, rounded + stat,
                       target_logit + t);
  }
}

// loss, lse and what the gradient needs of one token: 1 / (R + e_y) and R / (R + e_y).
struct Outcome {
  float loss, lse, inv, other;
};
__device__ __forceinline__ Outcome outcome(float N, float others, float R, float ly) {
  Outcome r;
  const float m = tile_exponent(ly);
  const float ey = __builtin_ldexpf(relative_exp(ly, m), (int)fmaxf(m - N, -300.f));  // formed next to 1, as every e
  const float all = others + ey;
  if (others <= ey) {
    r.loss = log1pf(others / ey);
    r.lse = ly + r.loss;
  } else {
    // S = f 2^k and N + k are taken apart: their logarithms would cancel where N is far above log2 S
    int k;
    const float f = __builtin_frexpf(all, &k), n = N + (float)k;
    r.lse = __builtin_fmaf(n, kLn2, __builtin_fmaf(n, kLn2Lo, logf(f)));
    // n ln 2 - l_y first: the two are close when the loss is small
    r.loss = (__builtin_fmaf(n, kLn2, -ly) + n * kLn2Lo) + logf(f);
  }
  r.inv = 1.0f / (R + ey);
  r.other = R / (R + ey);
  if (!(all > 0.f && all < INFINITY) || !(fabsf(N) < kMaxExponent)) r.loss = r.lse = r.inv = r.other = NAN;
  return r;
}

// (N - n) / 64, at most 3 (192 leaves nothing of a bf16 value up to 1).
__device__ __forceinline__ int distance(float d) { return (int)fminf(d * 0.015625f, 3.0f); }
// The distances of the tokens of four neighbouring lanes, two bits each, in all of them.
__device__ __forceinline__ int pack_distances(int d) {
  d <<= 2 * (threadIdx.x & 3);
  d |= __shfl_xor(d, 1);
  return d | __shfl_xor(d, 2);
}

// Folds the piece's tiles into the running exponent N and sums S and R of each token: 8 tokens and 32 lanes
// along the tiles a workgroup, eight tiles of a lane in flight at once.  shift [tile][tpad / 4]: the
// distances of four tokens a byte (0 for tokens past the last); factor: 2^(N before - N), for what the
// pieces before have summed.  loss (nullptr: not yet, or not here): the piece is the last, N and S are final.
// 9.5 us for 4096 tokens by 126 tiles: the tiles' statistics are 12 bytes per token and 128 words, so this is latency.
// kGrad: with rounded, R, shift and factor.
template <bool kGrad>
__global__ __launch_bounds__(256) void head_fold(const float *__restrict__ exponent, const float *__restrict__ sum,
                                                 const float *__restrict__ rounded, int64_t tpad, int tiles, bool first,
                                                 const uint32_t *__restrict__ state, float *__restrict__ N,
                                                 float *__restrict__ S, float *__restrict__ R,
                                                 uint8_t *__restrict__ shift,
                                                 float *__restrict__ factor, const int *__restrict__ rows,
                                                 const float *__restrict__ target_logit, float *__restrict__ loss,
                                                 float *__restrict__ lse) {
  constexpr int kLanes = 32, kDeep = 8;
  __shared__ float part[kLanes][9], part_r[kGrad ? kLanes : 1][9];
  const int live = (int)state[1];
  if ((int)blockIdx.x * 8 >= live) return;
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int t = min((int)blockIdx.x * 8 + c, live - 1);
  const float before = first ? kNoExponent : N[t], held = first ? 0.f : S[t], held_r = kGrad && !first ? R[t] : 0.f;
  float top = before;
  float ex[kDeep], sm[kDeep], rm[kDeep];
  for (int i0 = 0; i0 < tiles; i0 += kLanes * kDeep) {
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int i = i0 + j * kLanes + g;
      ex[j] = i < tiles ? exponent[i * tpad + t] : kNoExponent;
      sm[j] = i < tiles ? sum[i * tpad + t] : 0.f;
      if (kGrad) rm[j] = i < tiles ? rounded[i * tpad + t] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) top = fmaxf(top, ex[j]);
  }
  part[g][c] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kLanes; ++i) top = fmaxf(top, part[i][c]);
  __syncthreads();
  float s = 0.f, r = 0.f;
  for (int i0 = 0; i0 < tiles; i0 += kLanes * kDeep) {
    if (tiles > kLanes * kDeep) {  // more than the registers hold: read again
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        const int i = i0 + j * kLanes + g;
        ex[j] = i < tiles ? exponent[i * tpad + t] : kNoExponent;
        sm[j] = i < tiles ? sum[i * tpad + t] : 0.f;
        if (kGrad) rm[j] = i < tiles ? rounded[i * tpad + t] : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int i = i0 + j * kLanes + g;
      const float d = top - ex[j];
      const float f = __builtin_amdgcn_exp2f(-fminf(d, 300.f));
      s += sm[j] * f;
      if (kGrad) {
        r += rm[j] * f;
        const int four = pack_distances((int)blockIdx.x * 8 + c < live ? distance(d) : 0);
        if (i < tiles && (c & 3) == 0) shift[i * (tpad >> 2) + (int)blockIdx.x * 2 + (c >> 2)] = (uint8_t)four;
      }
    }
  }
  part[g][c] = s;
  if (kGrad) part_r[g][c] = r;
  __syncthreads();
  if (g == 0 && (int)blockIdx.x * 8 + c < live) {
    const float f = first ? 0.f : __builtin_amdgcn_exp2f(-fminf(top - before, 300.f));
    float all = held * f;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) all += part[i][c];
    N[t] = top;
    S[t] = all;
    if (kGrad) {
      float all_r = held_r * f;
#pragma unroll
      for (int i = 0; i < kLanes; ++i) all_r += part_r[i][c];
      R[t] = all_r;
      factor[t] = f;
    }
    if (loss) {
      const Outcome o = outcome(top, all, all, target_logit[t]);
      loss[rows[t]] = o.loss;
      if (lse) lse[rows[t]] = o.lse;
    }
  }
}

// One tile (256 columns d, 256 tokens) of G over one range of the piece's words, see the top.  Bound by the matrix cores
// and, behind them, the LDS, which also transposes W's tile: 791 us for 4096 x 8192 x 16128 (1.30 PFLOP/s, MFMAs busy
// 75% of the cycles; the library's product of plain operands this way round reaches 1.27).  The tiles and their
// splits follow from the tokens that carry a loss; `words` is the length of every piece but the last, so that the
// ranges, and the tiles' places in part, are the same in all.  part: [split][tile][256 tokens][256 d] fp32, in units of
// 2^N.  kFold: the piece is the only one and has at most kFoldV words; the exponents are folded here, which spares the
// launch of head_fold (shift is then unused).
template <bool kFold>
__global__ __launch_bounds__(kThreads, 2) void head_grad(const uint16_t *__restrict__ e, int64_t pitch,
                                                         const uint16_t *__restrict__ w, int nv, int words, int D,
                                                         int nleft, const uint32_t *__restrict__ state,
                                                         const uint8_t *__restrict__ shift,
                                                         const float *__restrict__ exponent, int64_t tpad,
                                                         const float *__restrict__ factor, bool first,
                                                         float *__restrict__ part) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t shifts[kMaxPiece / kStatV * kTileT / 4];
  const int live = (int)state[1];
  const int ntoken = (live + kTileT - 1) / kTileT, tiles = nleft * ntoken;
  const Split split = split_of(tiles, words);
  if ((int)blockIdx.x >= tiles * split.count) return;
  const int slot = place_of(blockIdx.x, tiles * split.count), nth = scalar(slot / tiles);
  const Tile tile = tile_at(slot - nth * tiles, nleft, ntoken);
  const int t0 = tile.token * kTileT, d0 = tile.left * kTileV;
  const int first_word = scalar(nth * split.range);
  const int last_word = scalar(min(min(first_word + split.range, words), nv));  // none: the sums before are rescaled
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) & 1, wn = (wave & 1) + 2 * (wave >> 2);

  Operands o;
  o.left_pitch = (uint32_t)D * 2u;
  o.left_step = (int64_t)kStep * D * 2;
  o.right_step = 2 * kStep;
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // unit row r: columns 128 (r / 64) + 64 (i / 2) .. + 63, contraction row r % 64
    const int r = (2 * wave + (i & 1)) * 8 + (lane >> 3);
    const int d = min(d0 + 128 * (r >> 6) + 64 * (i >> 1), D - 64) - d0;
    o.left_off[i] = (uint32_t)(2 * d) + (((lane & 7) ^ swizzle_cols(r & 63)) << 4);
    const int rt = (4 * wave + i) * 8 + (lane >> 3);
    o.right_off[i] = (uint32_t)min(rt, live - 1 - t0) * (uint32_t)(2 * pitch) + (((lane & 7) ^ swizzle_rows(rt)) << 4);
  }
  f32x4 acc[8][4];
  tile_zero(acc);
  if (first_word < last_word) {
    const int groups = (last_word - first_word + kStatV - 1) / kStatV, g0 = first_word / kStatV;
    int moved = 0;  // any distance of the tile's tokens
    if (kFold) {  // two threads a token
      const int token = threadIdx.x & 255, half = threadIdx.x >> 8, all = (nv + kStatV - 1) / kStatV;
      const float *ex = exponent + min(t0 + token, live - 1);
      float top = kNoExponent;
#pragma unroll 8
      for (int i = half; i < all; i += 2) top = fmaxf(top, ex[i * tpad]);
      float *fold = (float *)lds;
      fold[threadIdx.x] = top;
      __syncthreads();
      top = fmaxf(top, fold[threadIdx.x ^ 256]);
      for (int i = half; i < groups; i += 2) {
        const int four = pack_distances(distance(top - ex[(g0 + i) * tpad]));
        if ((token & 3) == 0) shifts[i * (kTileT / 4) + (token >> 2)] = (uint8_t)four;
        moved |= four;
      }
    } else {  // head_fold's; a group's bytes of the tile's tokens are 16 words
      const uint8_t *src = shift + (int64_t)g0 * (tpad >> 2) + (t0 >> 2);
#pragma unroll 8
      for (int i = threadIdx.x; i < groups * 16; i += kThreads) {
        int four = *(const int *)(src + (i >> 4) * (tpad >> 2) + 4 * (i & 15));
        const int bytes = (live - t0 + 3) / 4 - 4 * (i & 15);  // the others are not written
        if (bytes < 4) four = bytes > 0 ? four & (int)(0xFFFFFFFFu >> (32 - 8 * bytes)) : 0;
        ((int *)shifts)[i] = four;
        moved |= four;
      }
    }
    const bool scaled = scalar(__syncthreads_or(moved)) != 0;
    o.left = uniform(w + (int64_t)first_word * D + d0);
    o.right = uniform(e + (int64_t)t0 * pitch + first_word);
    o.left_rows = last_word - first_word;
    product<true, true>(o, (last_word - first_word + kStep - 1) / kStep, lds, shifts, scaled, acc);
  }
  float *out = part + (int64_t)slot * (kTileT * kTileV);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int t = 64 * wn + 16 * n + (lane & 15);
    if (t0 + t >= live) continue;
    const float f = first ? 0.f : factor[t0 + t];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int d = 128 * wm + 16 * m + 4 * (lane >> 4);
      if (d0 + d >= D) continue;
      f32x4 *p = (f32x4 *)(out + t * kTileV + d);
      f32x4 v = acc[m][n];
      if (!first) {
        const f32x4 old = *p;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(old[q], f, v[q]);
      }
      *p = v;
    }
  }
}

// Eight values of row y of W from column c on (c % 8 == 0), as bf16 pairs: a bf16 head's (q.codes nullptr), or a
// packed one's by the decode of every use of the weight.
__device__ __forceinline__ u32x4 row_values(const uint16_t *w, const QWeight &q, const Codebook &cb, int64_t y, int D,
                                            int c) {
  const int64_t e = y * D + c;
  if (w) return *(const u32x4 *)(w + e);
  const int64_t block = e / kBlock;
  const float c1 = q.dq ? decode_constant(q.fp8[block], q.s2[block / kGroup], *q.mu) : q.s2[block];
  const uint32_t codes = *(const uint32_t *)(q.codes + e / 2);
  auto level = [&](uint32_t k) {  // a register each: the levels are in the kernel's arguments
    float v = cb.v[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) v = k == (uint32_t)i ? cb.v[i] : v;
    return decode_product(v, c1);
  };
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = pack_bf16x2(level((codes >> (8 * i)) & 15u), level((codes >> (8 * i + 4)) & 15u));
  return out;
}

// grad_h of one token a workgroup (and its loss and lse), eight columns a thread and turn.  Bound by HBM: 45 us for 4096
// x 8192 (fp32 sums and W's rows read, bf16 written: 5.7 TB/s).  kFold: as in head_grad, N,
// S and R come from the tiles' exponents and sums.
template <bool kFold>
__global__ __launch_bounds__(256) void head_finish(const int *__restrict__ place, const float *__restrict__ N,
                                                   const float *__restrict__ S, const float *__restrict__ R,
                                                   const float *__restrict__ exponent, const float *__restrict__ sum,
                                                   const float *__restrict__ rounded, int64_t tpad, int stat_tiles,
                                                   const float *__restrict__ target_logit,
                                                   const int64_t *__restrict__ target, const uint16_t *__restrict__ w,
                                                   QWeight q, Codebook cb, const float *__restrict__ weight,
                                                   float scale, const float *__restrict__ part, int words, int nleft,
                                                   const uint32_t *__restrict__ state, int D,
                                                   float *__restrict__ loss, float *__restrict__ lse,
                                                   uint16_t *__restrict__ grad) {
  const int t = blockIdx.x;
  const int j = place[t];
  uint16_t *g = grad + (int64_t)t * D;
  if (j < 0) {
    const uint32_t fill = j == -2 ? 0x7FC07FC0u : 0u;
    for (int c = threadIdx.x * 8; c < D; c += 2048) *(u32x4 *)(g + c) = u32x4{fill, fill, fill, fill};
    return;
  }
  float n, s, rs;
  if (kFold) {  // at most 64 tiles, one a lane, every wave for itself
    const int i = threadIdx.x & 63;
    const float ex = i < stat_tiles ? exponent[i * tpad + j] : kNoExponent;
    const float sm = i < stat_tiles ? sum[i * tpad + j] : 0.f, rm = i < stat_tiles ? rounded[i * tpad + j] : 0.f;
    n = ex;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n = fmaxf(n, __shfl_xor(n, d));
    const float f = __builtin_amdgcn_exp2f(-fminf(n - ex, 300.f));
    s = sm * f;
    rs = rm * f;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      s += __shfl_xor(s, d);
      rs += __shfl_xor(rs, d);
    }
  } else {
    n = N[j];
    s = S[j];
    rs = R[j];
  }
  const Outcome r = outcome(n, s, rs, target_logit[j]);
  if (threadIdx.x == 0) {
    loss[t] = r.loss;
    if (lse) lse[t] = r.lse;
  }
  const float c_t = weight ? scale * weight[t] : scale;
  const float a = c_t * r.inv, b = c_t * r.other;
  const int64_t y = target[t];
  // the token's row in every split's tiles
  const int ntoken = ((int)state[1] + kTileT - 1) / kTileT, tiles = nleft * ntoken;
  const int splits = split_of(tiles, words).count;
  for (int c = threadIdx.x * 8; c < D; c += 2048) {
    const int64_t tile = place_at(Tile{c / kTileV, j / kTileT}, nleft, ntoken);
    const float *p = part + tile * (kTileT * kTileV) + j % kTileT * kTileV + c % kTileV;
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
      const f32x4 x = *(const f32x4 *)p, z = *(const f32x4 *)(p + 4);
      p += (int64_t)tiles * (kTileT * kTileV);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] += x[i];
        hi[i] += z[i];
      }
    }
    const u32x4 wv = row_values(w, q, cb, y, D, c);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g0 = i < 2 ? lo[2 * i] : hi[2 * i - 4], g1 = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
      const uint32_t pair = wv[i];
      o[i] = pack_bf16x2(__builtin_fmaf(a, g0, -b * bf16_lo(pair)), __builtin_fmaf(a, g1, -b * bf16_hi(pair)));
    }
    *(u32x4 *)(g + c) = o;
  }
}

// ---------------------------------------------------------------------------
// Few tokens or few words: the products run on the per-wave streams, 64 words
// (or 64 columns d) by up to 64 tokens a workgroup.  Up to 64 tokens both are
// bound by streaming W once; beyond, this form is for problems with too few
// 256 x 256 tiles to occupy the CUs (few_pays).  Exponents n are the integers
// next above, per token and 64 words, and the gradient's sums of a chunk of
// words are relative to the chunk's own largest n, which few_finish brings
// together: no pass over the tiles lies between the two products.
//   16 x 4096 x 32000 (W 262 MB): few_logits 43 us (6.1 TB/s), with the gradient
//   91 us, the call's launches included; a plain copy reaches 5.2 TB/s.
// A packed head is decoded inside both products up to 64 tokens (one group);
// beyond, every group would decode it again, and it is decoded once before.

constexpr int kFewWords = 64;       // words that share an exponent, and a step of the gradient
constexpr int kFewChunk = 128;      // steps of a chunk at most: its shift bytes are held in LDS

// e (nullptr: the loss alone, and no rounded) [T][pitch] of the piece, exponent, sum and rounded [64 words][tpad] of
// all words; v0: the piece's first word.  Workgroups: the token groups of 64 words, then the next words'.
// kPacked: the rows are decoded from q, the piece's, on their way in (w unused).
template <int NT, bool kPacked>
__global__ __launch_bounds__(kFewThreads, NT == 1 ? 2 : 1) void few_logits(
    const uint16_t *__restrict__ h, const uint16_t *__restrict__ w, QWeight q, Codebook cb,
    const int64_t *__restrict__ target, int T, int64_t v0, int64_t nv, int D, uint16_t *__restrict__ e, int64_t pitch,
    float *__restrict__ exponent, float *__restrict__ sum, float *__restrict__ rounded, int tpad,
    float *__restrict__ target_logit) {
  constexpr int kBytes = (kPacked ? 2 : few_stages<false, NT>()) * few_stage<NT>();
  __shared__ __attribute__((aligned(1024))) char lds[4 * kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = tpad / kFewTokens, place = place_of(blockIdx.x, gridDim.x), block = scalar(place / groups);
  const int t0 = (place - block * groups) * kFewTokens;
  const int64_t vt = (int64_t)block * kFewWords;
  const int words = (int)min((int64_t)kFewWords, nv - vt);
  uint32_t off[2 * NT];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int r = 8 * j + (lane >> 3);
    off[j] = (uint32_t)min(t0 + r, T - 1) * (uint32_t)(2 * D) + (((lane & 7) ^ swizzle_rows(r)) << 4);
  }
  f32x4 acc[4][NT];
  few_zero<NT>(acc);
  if constexpr (kPacked)
    few_product_packed<false, false, NT>(q, cb, vt, words, D / kBlock, 0, uniform(h), off, wave, D / kStep,
                                         lds + wave * kBytes, nullptr, acc);
  else
    few_product<false, false, NT>(uniform(w + vt * D), (uint32_t)D * 2u, words, 2 * kStep, uniform(h), off, wave,
                                  D / kStep, lds + wave * kBytes, nullptr, acc);
  float *red = (float *)lds;
  few_put<NT>(acc, red);
  // 4 NT tokens a wave, 16 / NT lanes a token, 4 NT words a lane
  constexpr int kLanes = 16 / NT, kWords = 4 * NT;
  const int tl = wave * 4 * NT + lane / kLanes, t = t0 + tl, first = lane % kLanes * kWords;
  const bool on = t < T;
  const int64_t at = on ? target[t] - v0 - vt : -1;
  const int y = at >= 0 && at < kFewWords ? (int)at : -1;
  float l[kWords], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kWords; i += 4) {
    const f32x4 x = few_sum<NT>(red, tl, first + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = first + i + q < words;
      l[i + q] = x[q];
      top = fmaxf(top, in ? x[q] : -INFINITY);
    }
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float ex = tile_exponent(top);
  float s = 0.f, r = 0.f;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    float p = relative_exp(l[i], ex);
    if (first + i >= words) p = 0.f;
    if (first + i == y) {
      target_logit[t] = l[i];
      p = 0.f;
    }
    s += p;
    l[i] = p;
  }
  if (e) {
    uint2 *row = (uint2 *)(e + (int64_t)t * pitch + vt + first);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint2 v = make_uint2(pack_bf16x2(l[4 * i], l[4 * i + 1]), pack_bf16x2(l[4 * i + 2], l[4 * i + 3]));
      if (on) row[i] = v;
      r = add_pair(v.y, add_pair(v.x, r));
    }
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) {
    s += __shfl_xor(s, d);
    r += __shfl_xor(r, d);
  }
  if (on && lane % kLanes == 0) {
    const int64_t i = (v0 + vt) / kFewWords * tpad + t;
    exponent[i] = ex;
    sum[i] = s;
    if (e) rounded[i] = r;
  }
}

// What a chunk's slot holds beside its sums: N, S and R [chunk][tpad].
struct FewSlots {
  float *N, *S, *R;
};

// One chunk of words, 64 columns; few_logits' statistics of the chunk are folded on the way.  part[chunk][T][D] relative
// to 2^N of the chunk, and (first columns) its N, S and R in `now`.  exponent and the sums start at the piece.  The
// pieces of a vocabulary share the slots: from the second on (first = false) a chunk's sums are added to what part
// and `before` hold of the pieces before, also where the last piece has no words for it.
template <int NT, bool kPacked>
__global__ __launch_bounds__(kFewThreads, 1) void few_grad(const uint16_t *__restrict__ e, int64_t pitch,
                                                           const uint16_t *__restrict__ w, QWeight q, Codebook cb,
                                                           int T, int64_t nv, int D, int chunk_steps, bool first,
                                                           const float *__restrict__ exponent,
                                                           const float *__restrict__ sum,
                                                           const float *__restrict__ rounded, int tpad,
                                                           FewSlots before, FewSlots now, float *__restrict__ part) {
  constexpr int kBytes = (kPacked ? 2 : few_stages<true, NT>()) * few_stage<NT>(), kT = 16 * NT, kRows = kFewThreads / kT;
  __shared__ __attribute__((aligned(1024))) char lds[4 * kBytes];
  __shared__ uint8_t shifts[kFewChunk * kT];
  __shared__ float fold[kFewThreads], factor[kT][2];  // factors: of the sums before and of these
  // places: the slices of a chunk for one token group, then its other token groups, then the next chunk
  const int slices = D / 64, groups = tpad / kFewTokens, place = place_of(blockIdx.x, gridDim.x);
  const int over = scalar(place / slices), slice = scalar(place - over * slices);
  const int chunk = scalar(over / groups), t0 = (over - chunk * groups) * kFewTokens;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t vb = (int64_t)chunk * chunk_steps * kFewWords;
  const int words = (int)min((int64_t)chunk_steps * kFewWords, nv - vb);
  const int steps = (words + kFewWords - 1) / kFewWords;
  {  // the chunk's largest exponent of each token, every step's distance from it, and its sums: S by the workgroup of
     // the first columns, R by that of the second (both in one delay the launch: 64 tokens, packed, 109 against 119 us)
    const int t = threadIdx.x % kT, g = threadIdx.x / kT;
    const int64_t from = vb / kFewWords * tpad + min(t0 + t, T - 1);
    const float *ex = exponent + from;
    float top = kNoExponent;
#pragma unroll 8
    for (int i = g; i < steps; i += kRows) top = fmaxf(top, ex[i * tpad]);
    fold[threadIdx.x] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) top = fmaxf(top, fold[i * kT + t]);
    __syncthreads();
#pragma unroll 8
    for (int i = g; i < steps; i += kRows) shifts[i * kT + t] = (uint8_t)fminf(top - ex[i * tpad], 255.f);
    const int64_t at = (int64_t)chunk * tpad + t0 + t;
    const bool on = g == 0 && t0 + t < T;
    float n = top, f = 1.f, f_old = 0.f;
    if (on && !first) {
      const float old = before.N[at];
      n = fmaxf(top, old);
      factor[t][0] = f_old = __builtin_amdgcn_exp2f(-fminf(n - old, 300.f));
      factor[t][1] = f = __builtin_amdgcn_exp2f(-fminf(n - top, 300.f));
    }
    if (on && slice == 0) now.N[at] = n;
    for (int kind = slice; kind < 2; kind += slices) {
      const float *src = (kind ? rounded : sum) + from;
      float s = 0.f;
#pragma unroll 8
      for (int i = g; i < steps; i += kRows)
        s += src[i * tpad] * __builtin_amdgcn_exp2f(-fminf(top - ex[i * tpad], 300.f));
      fold[threadIdx.x] = s;
      __syncthreads();
      if (on) {
        for (int i = 1; i < kRows; ++i) s += fold[i * kT + t];
        const float held = first ? 0.f : (kind ? before.R : before.S)[at] * f_old;
        (kind ? now.R : now.S)[at] = held + s * f;
      }
      __syncthreads();
    }
    __syncthreads();
  }
  uint32_t off[2 * NT];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int r = 8 * j + (lane >> 3);
    off[j] = (uint32_t)min(r, T - 1 - t0) * (uint32_t)(2 * pitch) + (((lane & 7) ^ swizzle_rows(r)) << 4);
  }
  f32x4 acc[4][NT];
  few_zero<NT>(acc);
  const char *right = uniform(e + (int64_t)t0 * pitch + vb);
  if constexpr (kPacked)
    few_product_packed<true, true, NT>(q, cb, vb, words, D / kBlock, slice, right, off, wave, steps, lds + wave * kBytes,
                                       shifts, acc);
  else
    few_product<true, true, NT>(uniform(w + vb * D + 64 * slice), (uint32_t)D * 2u, words, (int64_t)kStep * D * 2,
                                right, off, wave, steps, lds + wave * kBytes, shifts, acc);
  float *red = (float *)lds;
  few_put<NT>(acc, red);
  // 16 lanes a token, four columns each
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = i * 16 + (threadIdx.x >> 4), d = 4 * (threadIdx.x & 15);
    if (t0 + t >= T) continue;
    f32x4 sums = few_sum<NT>(red, t, d), *p = (f32x4 *)(part + ((int64_t)chunk * T + t0 + t) * D + 64 * slice + d);
    if (!first) {
      const f32x4 old = *p;
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[q] = __builtin_fmaf(old[q], factor[t][0], sums[q] * factor[t][1]);
    }
    *p = sums;
  }
}

// Notes a target past the vocabulary (one workgroup of 256 threads).
__device__ __forceinline__ void few_state(const int64_t *target, int T, int64_t V, uint32_t *state) {
  __shared__ int any;
  if (threadIdx.x == 0) any = 0;
  __syncthreads();
  bool bad = false;
  for (int t = threadIdx.x; t < T; t += 256) bad |= target[t] >= V;
  if (bad) any = 1;
  __syncthreads();
  if (threadIdx.x == 0) state[0] = any ? 2u : 0u;
}

// Loss and lse of one token a workgroup from the exponents and sums of all its words.
__global__ __launch_bounds__(256) void few_losses(const int64_t *__restrict__ target, int T, int64_t V, int groups,
                                                  const float *__restrict__ exponent, const float *__restrict__ sum,
                                                  int tpad, const float *__restrict__ target_logit,
                                                  uint32_t *__restrict__ state,
                                                  float *__restrict__ loss, float *__restrict__ lse) {
  __shared__ float fold[256];
  const int t = blockIdx.x, tid = threadIdx.x;
  if (t == 0) few_state(target, T, V, state);
  const int64_t y = target[t];
  if (y < 0 || y >= V) {
    if (tid == 0) no_loss(y, t, loss, lse);
    return;
  }
  float top = kNoExponent;
  for (int i = tid; i < groups; i += 256) top = fmaxf(top, exponent[(int64_t)i * tpad + t]);
  fold[tid] = top;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if (tid < d) fold[tid] = fmaxf(fold[tid], fold[tid + d]);
    __syncthreads();
  }
  top = fold[0];
  __syncthreads();
  float s = 0.f;
  for (int i = tid; i < groups; i += 256)
    s += sum[(int64_t)i * tpad + t] * __builtin_amdgcn_exp2f(-fminf(top - exponent[(int64_t)i * tpad + t], 300.f));
  fold[tid] = s;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if (tid < d) fold[tid] += fold[tid + d];
    __syncthreads();
  }
  if (tid == 0) {
    const Outcome r = outcome(top, fold[0], fold[0], target_logit[t]);
    loss[t] = r.loss;
    if (lse) lse[t] = r.lse;
  }
}

// grad_h, loss and lse from the chunks: workgroup (token, 512 columns), eight columns and every fourth
// chunk a thread, so that the chunks' sums (from the caches of other XCDs) arrive in few round trips.
__global__ __launch_bounds__(256) void few_finish(const int64_t *__restrict__ target, int T, int64_t V, int D,
                                                  int chunks, const float *__restrict__ N, const float *__restrict__ S,
                                                  const float *__restrict__ R, int tpad, const float *__restrict__ target_logit,
                                                  const uint16_t *__restrict__ w, QWeight q, Codebook cb,
                                                  const float *__restrict__ weight, float scale,
                                                  const float *__restrict__ part, uint32_t *__restrict__ state,
                                                  float *__restrict__ loss, float *__restrict__ lse,
                                                  uint16_t *__restrict__ grad) {
  __shared__ f32x4 half[3][64][2];
  const int t = blockIdx.x, lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int c = (int)blockIdx.y * 512 + 8 * lane;
  if (t == 0 && blockIdx.y == 0) few_state(target, T, V, state);
  const int64_t y = target[t];
  const bool lead = blockIdx.y == 0 && threadIdx.x == 0;
  u32x4 *g = (u32x4 *)(grad + (int64_t)t * D + c);
  if (y < 0 || y >= V) {
    const uint32_t fill = y < 0 ? 0u : 0x7FC07FC0u;
    if (c < D && group == 0) *g = u32x4{fill, fill, fill, fill};
    if (lead) no_loss(y, t, loss, lse);
    return;
  }
  // N, S and R: the chunks one a lane, every wave for itself
  float top = kNoExponent, s = 0.f, rs = 0.f;
  for (int i = lane; i < chunks; i += 64) top = fmaxf(top, N[(int64_t)i * tpad + t]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  for (int i = lane; i < chunks; i += 64) {
    const float f = __builtin_amdgcn_exp2f(-fminf(top - N[(int64_t)i * tpad + t], 300.f));
    s += S[(int64_t)i * tpad + t] * f;
    rs += R[(int64_t)i * tpad + t] * f;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    s += __shfl_xor(s, d);
    rs += __shfl_xor(rs, d);
  }
  f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
  const float *p = part + (int64_t)t * D + min(c, D - 8);
  for (int i0 = group; i0 < chunks; i0 += 16) {
    f32x4 x[4], z[4];
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(i0 + 4 * j, chunks - 1);
      x[j] = *(const f32x4 *)(p + (int64_t)i * T * D);
      z[j] = *(const f32x4 *)(p + (int64_t)i * T * D + 4);
      f[j] = i0 + 4 * j < chunks ? __builtin_amdgcn_exp2f(-fminf(top - N[(int64_t)i * tpad + t], 300.f)) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i0 + 4 * j >= chunks) continue;  // a factor of 0 would not keep a NaN out
        lo[k] = __builtin_fmaf(x[j][k], f[j], lo[k]);
        hi[k] = __builtin_fmaf(z[j][k], f[j], hi[k]);
      }
  }
  if (group > 0) {
    half[group - 1][lane][0] = lo;
    half[group - 1][lane][1] = hi;
  }
  __syncthreads();
  const Outcome r = outcome(top, s, rs, target_logit[t]);
  if (lead) {
    loss[t] = r.loss;
    if (lse) lse[t] = r.lse;
  }
  if (group > 0 || c >= D) return;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const f32x4 x = half[j][lane][0], z = half[j][lane][1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] += x[k];
      hi[k] += z[k];
    }
  }
  const float c_t = weight ? scale * weight[t] : scale;
  const float a = c_t * r.inv, b = c_t * r.other;
  const u32x4 wv = row_values(w, q, cb, y, D, c);
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float g0 = i < 2 ? lo[2 * i] : hi[2 * i - 4], g1 = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
    const uint32_t pair = wv[i];
    o[i] = pack_bf16x2(__builtin_fmaf(a, g0, -b * bf16_lo(pair)), __builtin_fmaf(a, g1, -b * bf16_hi(pair)));
  }
  *g = o;
}

}  // namespace

// What a workspace holds of e, of decoded rows (values of two bytes) and of fp32 sums (bytes) at most, see plan_head.
constexpr int64_t kPieceValues = (int64_t)64 << 20, kPartBytes = (int64_t)128 << 20, kStatBytes = (int64_t)64 << 20;

// The few-token form in pieces of up to `piece` words: e of a piece, the sums of every chunk of words.
static HeadPlan plan_few(HeadPlan p, int64_t piece) {
  p.pieces = cdiv(p.V, piece);
  p.words = cdiv(cdiv(p.V, p.pieces), kTileV) * kTileV;
  p.pieces = cdiv(p.V, p.words);
  p.splits = p.split_words = 0;
  p.tpad = cdiv(p.T, kFewTokens) * kFewTokens;
  const int64_t groups = cdiv(p.V, kFewWords), piece_steps = cdiv(std::min(p.words, p.V), kFewWords);
  if (p.grad) {
    // about one workgroup a CU, at least a step for each of its waves, at most kFewChunk steps
    const int64_t chunks =
        std::max<int64_t>(1, std::min(256 / (p.D / 64 * (p.tpad / kFewTokens)), cdiv(piece_steps, 4)));
    const int64_t steps = std::min<int64_t>(kFewChunk, cdiv(piece_steps, chunks));
    p.split_words = steps * kFewWords;
    p.splits = cdiv(std::min(p.words, p.V), p.split_words);  // of a piece; the next pieces' are added to them
  }
  size_t off = 256;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  p.off_logit = take((size_t)p.tpad * 4);
  p.off_exponent = take((size_t)groups * p.tpad * 4);
  p.off_sum = take((size_t)groups * p.tpad * 4);
  p.off_rounded = p.grad ? take((size_t)groups * p.tpad * 4) : 0;
  const int64_t sides = p.pieces > 1 ? 2 : 1;  // a piece's slots and those of the piece before
  p.off_n = take((size_t)sides * p.splits * p.tpad * 4);
  p.off_s = take((size_t)sides * p.splits * p.tpad * 4);
  p.off_r = take((size_t)sides * p.splits * p.tpad * 4);
  p.off_e = p.grad ? take((size_t)p.T * piece_steps * kFewWords * 2) : 0;
  p.off_part = p.grad ? take((size_t)p.splits * p.T * p.D * 4) : 0;
  p.off_w = p.decode ? take((size_t)p.words * p.D * 2) : 0;
  p.off_rows = p.off_place = p.off_factor = p.off_shift = 0;
  p.total = off;
  return p;
}

// Rows v0 .. v0 + nv of a packed head; v0 is a multiple of 256, so whole groups of constants lie before it.
static QWeight rows_of(const QWeight &q, int64_t v0, int64_t nv) {
  QWeight rows = q;
  const int64_t block = v0 * q.n_in / kBlock;
  rows.n_out = nv;
  rows.codes += v0 * q.n_in / 2;
  if (rows.dq) {
    rows.fp8 += block;
    rows.s2 += block / kGroup;
  } else {
    rows.s2 += block;
  }
  return rows;
}

template <int NT, bool kPacked>
static hipError_t launch_few(const HeadPlan &p, const uint16_t *h, const uint16_t *w, const QWeight *q,
                             const int64_t *target, const float *weight, float scale, float *loss, float *lse,
                             uint16_t *grad, char *ws, const Codebook &cb, hipStream_t st) {
  uint32_t *state = (uint32_t *)ws;
  float *logit = (float *)(ws + p.off_logit), *rounded = (float *)(ws + p.off_rounded);
  float *exponent = (float *)(ws + p.off_exponent), *sum = (float *)(ws + p.off_sum);
  auto slots = [&](bool odd) {
    const int64_t side = odd ? p.splits * p.tpad : 0;
    return FewSlots{(float *)(ws + p.off_n) + side, (float *)(ws + p.off_s) + side, (float *)(ws + p.off_r) + side};
  };
  FewSlots before{}, now{};
  float *part = (float *)(ws + p.off_part);
  uint16_t *e = p.grad ? (uint16_t *)(ws + p.off_e) : nullptr;
  uint16_t *wp = (uint16_t *)(ws + p.off_w);
  const int T = (int)p.T, D = (int)p.D, groups = (int)cdiv(p.V, kFewWords), tpad = (int)p.tpad;
  const int token_groups = tpad / kFewTokens;
  const QWeight qw = q ? *q : QWeight{};
  const int64_t pitch = cdiv(std::min(p.words, p.V), kFewWords) * kFewWords;
  for (int64_t v0 = 0; v0 < p.V; v0 += p.words) {
    const int64_t nv = std::min(p.words, p.V - v0);
    const uint16_t *piece = w ? w + v0 * p.D : wp;
    if (p.decode) {
      const hipError_t err = launch_dequantize(rows_of(*q, v0, nv), wp, cb, st);
      if (err != hipSuccess) return err;
    }
    const QWeight rows = kPacked ? rows_of(*q, v0, nv) : QWeight{};
    few_logits<NT, kPacked><<<(unsigned)(cdiv(nv, kFewWords) * token_groups), kFewThreads, 0, st>>>(
        h, piece, rows, cb, target, T, v0, nv, D, e, pitch, exponent, sum, rounded, tpad, logit);
    if (!p.grad) continue;
    const int64_t g0 = v0 / kFewWords * tpad;
    before = now;
    now = slots((v0 / p.words & 1) != 0);
    few_grad<NT, kPacked><<<(unsigned)(p.splits * token_groups * (D / 64)), kFewThreads, 0, st>>>(
        e, pitch, piece, rows, cb, T, nv, D, (int)(p.split_words / kFewWords), v0 == 0, exponent + g0, sum + g0,
        rounded + g0, tpad, before, now, part);
  }
  if (!p.grad) {
    few_losses<<<(unsigned)T, 256, 0, st>>>(target, T, p.V, groups, exponent, sum, tpad, logit, state, loss, lse);
    return hipGetLastError();
  }
  few_finish<<<dim3((unsigned)T, (unsigned)cdiv(D, 512)), 256, 0, st>>>(target, T, p.V, D, (int)p.splits, now.N, now.S,
                                                                       now.R, tpad,
                                                                       logit, w, qw, cb, weight, scale, part, state,
                                                                       loss, lse, grad);
  return hipGetLastError();
}

// Whether the streamed form is taken: always up to 64 tokens, and where its time, estimated in us from
// runs of both forms at 66 to 2048 tokens, 256 to 4096 columns and 300 to 32000 words, is below that of
// the tiles.  (The host does not know which tokens carry no loss: every token counts, and the streams compute
// them all, where the tiles skip them.)  A stream's unit is 64 tokens, 64 columns, 4096 words; a workgroup of the logits costs about
// 2.6 us besides.  The tiles have launches and first copies, the chain of a tile's steps, the sums of a
// vocabulary spread over splits, and the operations.  Measured, with the gradient (tiles / streams): 256 x
// 1024 x 4000 63 / 25 us, 1024 x 1024 x 4000 70 / 63, 512 x 1024 x 16000 80 / 108, 66 x 4096 x 16000
// 122 / 95, 256 x 4096 x 16000 135 / 173; the loss alone: 512 x 4096 x 4000 73 / 35, 1024 x 4096 x 4000
// 75 / 67, 200 x 1024 x 32000 31 / 55.
static bool few_pays(int64_t T, int64_t V, int64_t D, bool grad) {
  if (V > kFewMaxWords || T > kHeadMaxTokens) return false;
  if (T <= kFewTokens) return true;
  const double groups = (double)cdiv(T, kFewTokens), units = groups * (D / 64) * (V / 4096.0);
  const double blocks = groups * cdiv(V, kFewWords), ops = 2.0 * T * V * D;
  const double few = grad ? 18 + 0.155 * units + 0.010 * blocks : 12 + 0.055 * units + 0.010 * blocks;
  const double tile = grad ? 34 + 0.0155 * D + 0.0008 * V + ops / 1.0e9 : 16 + std::max(0.0145 * D, ops / 1.35e9);
  return few < tile;
}

HeadPlan plan_head(int64_t T, int64_t V, int64_t D, bool grad, bool packed) {
  HeadPlan p;
  p.T = T;
  p.V = V;
  p.D = D;
  p.grad = grad;
  p.decode = packed;
  p.chunk = std::min<int64_t>(T, kHeadMaxTokens);
  // Words of a piece: 128 MB of e (grad) and of decoded weight (packed).  A larger piece leaves less of
  // the products' last rounds of workgroups empty (2048 tokens, 40% of them masked, V = 32000: 5 tiles of
  // tokens by 125 of words are three rounds of 256, two pieces of 63 and 62 four).
  auto fit = [](int64_t per_word, int64_t least) {  // words of a piece, `least` tiles at least
    return std::max(kPieceValues / per_word / kTileV, least) * kTileV;
  };
  const int64_t whole = cdiv(V, kTileV) * kTileV;
  p.few = few_pays(T, V, D, grad);
  if (p.few) {
    p.decode = packed && T > kFewTokens;  // up to 64 tokens the streams decode the rows themselves
    int64_t vc = whole;
    if (grad)  // also: as many chunks' sums as fit
      vc = std::min({vc, fit(T, 4), std::max<int64_t>(kPartBytes / (T * D * 4), 1) * kFewChunk * kFewWords});
    if (p.decode) vc = std::min(vc, fit(D, 4));
    const HeadPlan few = plan_few(p, vc);
    if ((cdiv(V, kFewWords) * (grad ? 12 : 8) + few.splits * 24) * few.tpad <= kStatBytes) return few;
    p.few = false;
    p.decode = packed;
  }
  p.tpad = cdiv(p.chunk, kTileT) * kTileT;
  int64_t vc = std::min(whole, std::max<int64_t>(((int64_t)1 << 30) / p.tpad / kTileV * kTileV, 8 * kTileV));
  if (grad) vc = std::min<int64_t>(std::min<int64_t>(vc, kMaxPiece), fit(p.tpad, 8));
  if (packed) vc = std::min(vc, fit(D, 4));
  p.pieces = cdiv(V, vc);
  p.words = cdiv(cdiv(V, p.pieces), kTileV) * kTileV;
  p.pieces = cdiv(V, p.words);
  p.split_words = 0;
  p.splits = grad ? split_slots((int)cdiv(D, kTileV), (int)cdiv(p.chunk, kTileT), (int)p.words) : 0;
  const int64_t stat = p.words / kStatV * p.tpad;
  size_t off = 256;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  p.off_rows = take((size_t)p.chunk * 4);
  p.off_place = take((size_t)p.chunk * 4);
  p.off_logit = take((size_t)p.chunk * 4);
  p.off_n = take((size_t)p.chunk * 4);
  p.off_s = take((size_t)p.chunk * 4);
  p.off_r = take((size_t)p.chunk * 4);
  p.off_factor = take((size_t)p.chunk * 4);
  p.off_exponent = take((size_t)stat * 4);
  p.off_sum = take((size_t)stat * 4);
  p.off_rounded = grad ? take((size_t)stat * 4) : 0;
  p.off_shift = grad ? take((size_t)stat / 4) : 0;
  p.off_e = grad ? take((size_t)p.chunk * p.words * 2) : 0;
  p.off_part = grad ? take((size_t)p.splits * kTileT * kTileV * 4) : 0;
  p.off_w = packed ? take((size_t)p.words * D * 2) : 0;
  p.total = off;
  return p;
}

hipError_t launch_head_loss(const HeadPlan &p, const uint16_t *h, const uint16_t *w, const QWeight *q,
                            const int64_t *target, const float *weight, float scale, float *loss, float *lse,
                            uint16_t *grad, char *ws, const Codebook &cb, hipStream_t st) {
  if (p.few) {
    const bool packed = q && !p.decode;
    const auto run = p.T <= 16   ? packed ? launch_few<1, true> : launch_few<1, false>
                     : p.T <= 32 ? packed ? launch_few<2, true> : launch_few<2, false>
                     : packed    ? launch_few<4, true>
                                 : launch_few<4, false>;
    return run(p, h, w, q, target, weight, scale, loss, lse, grad, ws, cb, st);
  }
  uint32_t *state = (uint32_t *)ws;
  int *rows = (int *)(ws + p.off_rows), *place = (int *)(ws + p.off_place);
  float *logit = (float *)(ws + p.off_logit), *N = (float *)(ws + p.off_n), *S = (float *)(ws + p.off_s);
  float *factor = (float *)(ws + p.off_factor), *exponent = (float *)(ws + p.off_exponent);
  float *sum = (float *)(ws + p.off_sum), *part = (float *)(ws + p.off_part);
  float *R = (float *)(ws + p.off_r), *rounded = (float *)(ws + p.off_rounded);
  uint8_t *shift = p.grad ? (uint8_t *)(ws + p.off_shift) : nullptr;
  uint16_t *e = p.grad ? (uint16_t *)(ws + p.off_e) : nullptr;
  uint16_t *wp = (uint16_t *)(ws + p.off_w);
  const int D = (int)p.D;
  for (int64_t c0 = 0; c0 < p.T; c0 += p.chunk) {
    const int T = (int)std::min(p.chunk, p.T - c0);
    const int ntoken = (int)cdiv(T, kTileT), nd = (int)cdiv(p.D, kTileV), words = (int)p.words;
    const uint16_t *hc = h + c0 * p.D;
    const int64_t *yc = target + c0;
    float *lc = loss + c0, *ec = lse ? lse + c0 : nullptr;
    const bool list = p.T <= kThreads;  // head_logits lists the tokens itself
    const bool fold = p.grad && p.pieces == 1 && words <= kFoldV;  // head_grad and head_finish fold the tiles themselves
    if (!list) head_scan<<<1, 1024, 0, st>>>(yc, T, p.V, c0 == 0, rows, place, state, lc, ec);
    for (int64_t v0 = 0; v0 < p.V; v0 += p.words) {
      const int nv = (int)std::min(p.words, p.V - v0), nleft = (int)cdiv(nv, kTileV);
      const bool last = v0 + nv == p.V;
      const uint16_t *piece = w ? w + v0 * p.D : wp;
      if (q) {
        const hipError_t err = launch_dequantize(rows_of(*q, v0, nv), wp, cb, st);
        if (err != hipSuccess) return err;
      }
      const auto logits = list ? head_logits<true> : head_logits<false>;
      logits<<<(unsigned)(nleft * ntoken), kThreads, 0, st>>>(hc, piece, yc, T, p.V, v0, nv, D, nleft, rows, place, state,
                                                            lc, ec, e, p.words, exponent, sum, rounded, p.tpad, logit);
      if (!fold) {
        const auto collect = p.grad ? head_fold<true> : head_fold<false>;
        collect<<<(unsigned)cdiv(T, 8), 256, 0, st>>>(exponent, sum, rounded, p.tpad, (int)cdiv(nv, kStatV), v0 == 0,
                                                      state, N, S, R, shift, factor, rows, logit,
                                                      last && !p.grad ? lc : nullptr, ec);
      }
      if (!p.grad) continue;
      const auto product = fold ? head_grad<true> : head_grad<false>;
      product<<<(unsigned)p.splits, kThreads, 0, st>>>(  // enough for any number of live tokens
          e, p.words, piece, nv, words, D, nd, state, shift, exponent, p.tpad, factor, v0 == 0, part);
    }
    if (!p.grad) continue;
    const auto finish = fold ? head_finish<true> : head_finish<false>;
    finish<<<(unsigned)T, 256, 0, st>>>(place, N, S, R, exponent, sum, rounded, p.tpad, (int)cdiv(p.V, kStatV), logit, yc, w,
                                        q ? *q : QWeight{}, cb, weight ? weight + c0 : nullptr, scale, part, words, nd,
                                        state, D, lc, ec, grad + c0 * p.D);
  }
  return hipGetLastError();
}

}  // namespace qlora
