// The adapter-side products of the QLoRA linear layer (gfx950), one kernel
// family for all four of them.
//
// Adapter algebra: W' = W + s.B.A with A [r x n_in], B [n_out x r] (the LoRA
// formula of the nexusinovation tutorial, section "LoRA: O Padrão Ouro de
// Eficiência"); only the adapters receive gradients ("qlora" encyclopedia
// entry, tonho.wtf, section "a ideia").
//
//   u      = x A^T        [T x r]      A op: x (rows)          B op: A (rows)
//   v      = dy B         [T x r]      A op: dy (rows)         B op: B (columns)
//   grad_A = s v^T x      [r x n_in]   A op: v (columns)       B op: x (columns)
//   grad_B = s dy^T u     [n_out x r]  A op: dy (columns)      B op: u (columns)
//
// C[M x Nc] = scale * sum_k Aop(m, k) Bop(k, n), where an operand is either
// "row" (its contraction index is contiguous: Aop(m, k) = P[m ld + k]) or
// "column" (the contraction index strides: Aop(m, k) = P[k ld + m]).  Tiles of
// both operands are staged in LDS in their natural layout; "column" operands
// reach the MFMA through LDS transpose reads (ds_read_b64_tr_b16).  The
// contraction is split over the grid's z dimension; every split writes an
// fp32 partial tile and a second kernel adds the partials in split order (so
// the result is deterministic) and writes the scaled output.

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace qlora {

namespace {

constexpr int LT = 64;   // output tile (M and N) and contraction step
constexpr int LLD = 72;  // LDS row length (bf16), padded

typedef short v4s __attribute__((ext_vector_type(4)));

// Eight values of which the first `past` are dropped.
__device__ __forceinline__ u32x4 drop(u32x4 v, int past) {
  v = past & 1 ? u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16} : v;
  v = past & 2 ? u32x4{v[1], v[2], v[3], 0u} : v;
  v = past & 4 ? u32x4{v[2], v[3], 0u, 0u} : v;
  return past & 8 ? u32x4{0u, 0u, 0u, 0u} : v;
}

// Columns c .. c + 7 of a row, zero from ncols >= 8 on.  The rows need no alignment (n_out or r may be odd), and the
// row's end no branch: its last eight columns are loaded in its place and shifted down.  (With single 16-bit loads
// wherever a row was not aligned, the products of 2299 x 1684 x 2176 at rank 128 took 46 and 56 us; now 15 and 33.)
__device__ __forceinline__ u32x4 ld8(const uint16_t *row, int64_t c, int64_t ncols) {
  const int64_t at = min(c, ncols - 8);
  return drop(load8(row + at), (int)min(c - at, (int64_t)8));
}

// The same of element `at` of a matrix of `all` >= 8 values with fewer than eight columns, `keep` of them from here on:
// the load goes on into the next rows, whose values are cleared, and at the matrix's end starts before.
__device__ __forceinline__ u32x4 ld8_narrow(const uint16_t *src, int64_t at, int64_t all, int64_t keep) {
  const int64_t from = min(at, all - 8);
  const int k = (int)max(keep, (int64_t)0);
  u32x4 v = drop(load8(src + from), (int)min(at - from, (int64_t)8));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = k > 2 * i + 1 ? v[i] : k == 2 * i + 1 ? v[i] & 0xFFFFu : 0u;
  return v;
}

// Columns c .. c + 7 of a row, zero from ncols on: value by value, or (vec: the rows are 16-byte aligned) in one load
// where the row goes on.
__device__ __forceinline__ u32x4 ld8_by_one(const uint16_t *row, int64_t c, int64_t ncols, bool vec) {
  if (vec && c + 8 <= ncols) return *(const u32x4 *)(row + c);
  u32x4 v = {0u, 0u, 0u, 0u};
  for (int i = 0; i < 8; ++i)
    if (c + i < ncols) v[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  return v;
}

// Tile rows [r0, r0 + 64) x columns [c0, c0 + 64) of a row-major [nrows x ld]
// bf16 matrix (columns >= ncols and rows >= nrows read as zero); thread t
// fetches columns 8 (t%8) .. +7 of rows t/8 and t/8 + 32, so that each wave's
// load covers 8 whole 128-byte rows (a load that covers half of each of 16
// lines moves about half as many bytes per cycle from L2).  kWhole: the tile
// is known to be in range; kNarrow: ncols < 8; kTiny: fewer than eight values in all;
// kByLoad: decided load by load (vec: the rows are 16-byte aligned).
enum Edge { kWhole, kMasked, kNarrow, kTiny, kByLoad };
struct TileRegs {
  u32x4 v[2];
};

template <Edge kEdge>
__device__ __forceinline__ void load_tile(const uint16_t *src, int64_t ld, int64_t nrows, int64_t ncols,
                                          int64_t r0, int64_t c0, bool vec, int tid, TileRegs &t) {
  const int64_t row = r0 + (tid >> 3);
  const int64_t col = c0 + 8 * (tid & 7);
  if (kEdge == kWhole) {
    const uint16_t *p = src + row * ld + col;
    t.v[0] = load8(p);
    t.v[1] = load8(p + 32 * ld);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool in = row + 32 * h < nrows;
    const int64_t at = in ? row + 32 * h : nrows - 1;
    if (kEdge == kNarrow) {
      t.v[h] = ld8_narrow(src, at * ld + col, (nrows - 1) * ld + ncols, in ? ncols - col : 0);
    } else if (kEdge == kTiny || kEdge == kByLoad) {
      t.v[h] = in ? ld8_by_one(src + (row + 32 * h) * ld, col, ncols, kEdge == kByLoad && vec) : u32x4{0u, 0u, 0u, 0u};
    } else {
      const u32x4 v = ld8(src + at * ld, col, ncols);
      t.v[h] = in ? v : u32x4{0u, 0u, 0u, 0u};
    }
  }
}

__device__ __forceinline__ void store_tile(const TileRegs &t, uint16_t *lds, int tid) {
#pragma unroll
  for (int h = 0; h < 2; ++h) *(u32x4 *)&lds[((tid >> 3) + 32 * h) * LLD + 8 * (tid & 7)] = t.v[h];
}

// MFMA operand fragment for output rows/cols [base, base + 32), contraction
// sub-step kk (16 wide).  kTrans = false: the LDS tile is [out][contraction];
// kTrans = true: the LDS tile is [contraction][out] and is read transposed
// (in each 16-lane group, source lane s points at contraction row
// 16 kk + 8 (g/2) + s/4 (and +4) and output column 16 (g%2) + 4 (s%4); lane l
// then holds 4 consecutive contraction rows of output column l%32).
template <bool kTrans>
__device__ __forceinline__ u32x4 frag(const uint16_t *lds, int base, int kk, int lane) {
  if (!kTrans) return *(const u32x4 *)&lds[(base + (lane & 31)) * LLD + 16 * kk + 8 * (lane >> 5)];
  const int s = lane & 15, g = lane >> 4;
  const int row = 16 * kk + 8 * (g >> 1) + (s >> 2);
  const int col = base + 16 * (g & 1) + 4 * (s & 3);
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((v4s __attribute__((address_space(3))) *)(lds_void_t *)&lds[row * LLD + col]);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((v4s __attribute__((address_space(3))) *)(lds_void_t *)&lds[(row + 4) * LLD + col]);
  const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
  return u32x4{l2.x, l2.y, h2.x, h2.y};
}

// Contraction steps fetched at once: 4 (a group of 256) or, when a split is
// exactly 512 long and the launch fits one round of workgroups, all 8 of it,
// so that the whole split arrives in one round trip (128 KB per workgroup in
// flight, 147 KB of LDS).

template <bool kAT, bool kBT, bool kFull, bool kSorted, int kGroupSteps>
__device__ __forceinline__ void lora_body(const uint16_t *__restrict__ P, int64_t ldp,
                                          const uint16_t *__restrict__ Q, int64_t ldq, int64_t M, int64_t Nc,
                                          int64_t kb, int64_t ke, int64_t m0, int64_t n0, uint16_t (*sA)[LT * LLD],
                                          uint16_t (*sB)[LT * LLD], f32x16 &acc) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  // Operand tiles in natural layout: a row operand as [out rows][contraction],
  // a column operand as [contraction rows][out columns].  A group of
  // contraction steps is fetched at once; the next group's loads reuse the
  // registers as soon as the current group is in LDS, so they overlap with its
  // MFMAs.
  TileRegs ta[kGroupSteps], tb[kGroupSteps];
  const bool vp = (ldp % 8) == 0 && ((uintptr_t)P & 15u) == 0, vq = (ldq % 8) == 0 && ((uintptr_t)Q & 15u) == 0;
  // kSorted: which form loads an operand's tiles, rows (its output index) or columns, is decided once for all of them;
  // three forms more and the operands one after the other, which costs kernels that are all whole tiles 0.5 to 1 us.
  auto fetch_one = [&](auto trans, const uint16_t *src, int64_t ld, int64_t outs, int64_t o0, int64_t g0, TileRegs *t) {
    auto all = [&](auto edge) {
#pragma unroll
      for (int st = 0; st < kGroupSteps; ++st) {
        const int64_t k0 = g0 + LT * st;
        if constexpr (!trans.value)
          load_tile<edge.value>(src, ld, outs, ke, o0, k0, false, tid, t[st]);
        else
          load_tile<edge.value>(src, ld, ke, outs, k0, o0, false, tid, t[st]);
      }
    };
    if ((trans.value ? outs : ke) >= 8)
      all(std::integral_constant<Edge, kMasked>{});
    else if ((trans.value ? (ke - 1) * ld + outs : (outs - 1) * ld + ke) >= 8)
      all(std::integral_constant<Edge, kNarrow>{});
    else
      all(std::integral_constant<Edge, kTiny>{});
  };
  auto fetch = [&](int64_t g0) {
    if constexpr (kSorted && !kFull) {
      fetch_one(std::bool_constant<kAT>{}, P, ldp, M, m0, g0, ta);
      fetch_one(std::bool_constant<kBT>{}, Q, ldq, Nc, n0, g0, tb);
      return;
    }
    constexpr Edge kEdge = kFull ? kWhole : kByLoad;
#pragma unroll
    for (int st = 0; st < kGroupSteps; ++st) {
      const int64_t k0 = g0 + LT * st;
      if (!kAT)
        load_tile<kEdge>(P, ldp, M, ke, m0, k0, vp, tid, ta[st]);
      else
        load_tile<kEdge>(P, ldp, ke, M, k0, m0, vp, tid, ta[st]);
      if (!kBT)
        load_tile<kEdge>(Q, ldq, Nc, ke, n0, k0, vq, tid, tb[st]);
      else
        load_tile<kEdge>(Q, ldq, ke, Nc, k0, n0, vq, tid, tb[st]);
    }
  };
  fetch(kb);
  for (int64_t g0 = kb; g0 < ke; g0 += LT * kGroupSteps) {
#pragma unroll
    for (int st = 0; st < kGroupSteps; ++st) {
      store_tile(ta[st], sA[st], tid);
      store_tile(tb[st], sB[st], tid);
    }
    __syncthreads();
    // next group while this one multiplies (a uniform branch: the registers
    // are next needed by the LDS store above, which waits for them anyway)
    if (g0 + LT * kGroupSteps < ke) fetch(g0 + LT * kGroupSteps);
#pragma unroll
    for (int st = 0; st < kGroupSteps; ++st)
#pragma unroll
      for (int kk = 0; kk < LT / 16; ++kk) {
        const u32x4 a = frag<kAT>(sA[st], wm * 32, kk, lane);
        const u32x4 b = frag<kBT>(sB[st], wn * 32, kk, lane);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), acc, 0, 0, 0);
      }
    __syncthreads();
  }
}

template <bool kBf16Out>
__device__ __forceinline__ void emit_out(void *out, int64_t idx, float v) {
  if (kBf16Out) {
    __bf16 h = (__bf16)v;
    ((uint16_t *)out)[idx] = __builtin_bit_cast(uint16_t, h);
  } else {
    ((float *)out)[idx] = v;
  }
}

// v in three bf16 values: its rounding and what that leaves, twice (the differences are exact), which sum to v
// within 2^-24, its own precision.  A finite v that would round to infinity takes bf16's largest value first;
// nothing is left of an infinity.
__device__ __forceinline__ void emit_parts(uint16_t *out, uint16_t *mid, uint16_t *low, int64_t idx, float v) {
  const float top = __uint_as_float(0x7F7F0000u);
  const __bf16 h = (__bf16)(fabsf(v) > top && !__builtin_isinf(v) ? copysignf(top, v) : v);
  const float d = __builtin_isinf(v) ? 0.f : v - (float)h;
  const __bf16 m = (__bf16)d;
  const __bf16 l = (__bf16)(d - (float)m);
  out[idx] = __builtin_bit_cast(uint16_t, h);
  mid[idx] = __builtin_bit_cast(uint16_t, m);
  low[idx] = __builtin_bit_cast(uint16_t, l);
}

// One adapter product of a launch: C[M x Nc] = scale * Aop Bop over a
// contraction of Kc, split in chunks of `chunk` (S splits); tiles are numbered
// column-major (tile = n-tile * tiles_m + m-tile).
struct LoraProblem {
  const uint16_t *P;
  int64_t ldp;
  const uint16_t *Q;
  int64_t ldq;
  int64_t M, Nc, Kc, chunk, tiles_m;
  int S;
  float scale;  // applied here when S == 1, else by the reduction
  void *out;
  int64_t ldo;  // row stride of out (Nc unless the product fills columns of a wider matrix)
  float *part;
};

// A product of the backward pass from an 8-bit checkpoint.
struct Act8Problem : LoraProblem {
  uint16_t *out_mid, *out_low;  // v: what its bf16 rounding leaves
  // grad_A: Q holds the checkpoint's codes, P has the remainders P_mid, P_low
  const uint16_t *P_mid, *P_low;
  const float *code_scale;  // [Kc x Nc / 64]
};

// The finished tile: scaled into the output, or as the partial tile of its split.
template <bool kBf16Out, class Problem>
__device__ __forceinline__ void put_tile(const Problem &pr, int64_t tile, int s, const f32x16 &acc) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = (tile % pr.tiles_m) * LT, n0 = (tile / pr.tiles_m) * LT;
  // result element q of this lane: tile row wm*32 + 8(q/4) + 4(lane/32) + q%4, column wn*32 + lane%32
  const int col = wn * 32 + (lane & 31);
  if (pr.S == 1) {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t gm = m0 + wm * 32 + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3), gn = n0 + col;
      if (gm < pr.M && gn < pr.Nc) {
        if constexpr (kBf16Out && std::is_same_v<Problem, Act8Problem>)
          emit_parts((uint16_t *)pr.out, pr.out_mid, pr.out_low, gm * pr.ldo + gn, acc[q] * pr.scale);
        else
          emit_out<kBf16Out>(pr.out, gm * pr.ldo + gn, acc[q] * pr.scale);
      }
    }
    return;
  }
  // partial tile, row-major 64 x 64, at part[((tile * S) + s) * 4096]
  float *mine = pr.part + (tile * pr.S + s) * (LT * LT);
#pragma unroll
  for (int q = 0; q < 16; ++q) mine[(wm * 32 + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)) * LT + col] = acc[q];
}

template <bool kAT, bool kBT, bool kBf16Out, int kGroupSteps, class Problem>
__device__ __forceinline__ void lora_tile(const Problem &pr, int64_t tile, int s, uint16_t (*sA)[LT * LLD],
                                          uint16_t (*sB)[LT * LLD]) {
  const int64_t m0 = (tile % pr.tiles_m) * LT, n0 = (tile / pr.tiles_m) * LT;
  const int64_t kb = (int64_t)s * pr.chunk, ke = min(pr.Kc, kb + pr.chunk);
  constexpr bool kSorted = std::is_same_v<Problem, Act8Problem>;

  f32x16 acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.f;
  // full: both operand tiles in range, and the chunk is whole groups
  const bool full = (m0 + LT <= pr.M) && (n0 + LT <= pr.Nc) && ((ke - kb) % (LT * kGroupSteps) == 0);
  if (full)
    lora_body<kAT, kBT, true, kSorted, kGroupSteps>(pr.P, pr.ldp, pr.Q, pr.ldq, pr.M, pr.Nc, kb, ke, m0, n0, sA, sB,
                                                      acc);
  else
    lora_body<kAT, kBT, false, kSorted, kGroupSteps>(pr.P, pr.ldp, pr.Q, pr.ldq, pr.M, pr.Nc, kb, ke, m0, n0, sA,
                                                       sB, acc);

  put_tile<kBf16Out>(pr, tile, s, acc);
}

// One or two products of the same operand forms in one launch: workgroups
// below `first` take problem a (tile-major, splits innermost), the rest
// problem b.
template <bool kAT, bool kBT, bool kBf16Out, int kGroupSteps>
__global__ __launch_bounds__(256) void lora_gemm(LoraProblem a, LoraProblem b, int64_t first) {
  __shared__ __attribute__((aligned(16))) uint16_t sA[kGroupSteps][LT * LLD];
  __shared__ __attribute__((aligned(16))) uint16_t sB[kGroupSteps][LT * LLD];
  const int64_t id = blockIdx.x;
  const bool in_a = id < first;
  const LoraProblem &pr = in_a ? a : b;
  const int64_t j = in_a ? id : id - first;
  lora_tile<kAT, kBT, kBf16Out, kGroupSteps>(pr, j / pr.S, (int)(j % pr.S), sA, sB);
}

// out = scale * (sum over splits, in split order) of the partial tiles; one
// thread per 4 consecutive columns of a tile row.  Quads below `first` belong
// to problem a, the rest to problem b.
template <bool kBf16Out, class Problem>
__device__ __forceinline__ void reduce_quad(const Problem &pr, int64_t qd) {
  const int64_t tile = qd / (LT * LT / 4);
  const int local = (int)(qd % (LT * LT / 4)) * 4;
  const int64_t gm = (tile % pr.tiles_m) * LT + local / LT;
  const int64_t gn = (tile / pr.tiles_m) * LT + local % LT;
  if (gm >= pr.M || gn >= pr.Nc) return;
  const int S = pr.S;
  const f32x4 *p = (const f32x4 *)(pr.part + tile * S * (LT * LT) + local);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  // eight loads in flight at a time; the additions stay in split order
  for (int k0 = 0; k0 < S; k0 += 8) {
    f32x4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (k0 + k < S) ? p[(int64_t)(k0 + k) * (LT * LT / 4)] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[0] += v[k][0];
      acc[1] += v[k][1];
      acc[2] += v[k][2];
      acc[3] += v[k][3];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (gn + e < pr.Nc) {
      if constexpr (kBf16Out && std::is_same_v<Problem, Act8Problem>)
        emit_parts((uint16_t *)pr.out, pr.out_mid, pr.out_low, gm * pr.ldo + gn + e, acc[e] * pr.scale);
      else
        emit_out<kBf16Out>(pr.out, gm * pr.ldo + gn + e, acc[e] * pr.scale);
    }
}

template <bool kBf16Out>
__global__ __launch_bounds__(256) void lora_reduce(LoraProblem a, LoraProblem b, int64_t first, int64_t quads) {
  for (int64_t qd = (int64_t)blockIdx.x * 256 + threadIdx.x; qd < quads; qd += (int64_t)gridDim.x * 256) {
    if (qd < first)
      reduce_quad<kBf16Out>(a, qd);
    else
      reduce_quad<kBf16Out>(b, qd - first);
  }
}

// ---- grad_A from an 8-bit checkpoint --------------------------------------
// grad_A = s v^T x_hat: the codes of a 64 x 64 tile (one block of 64 columns a token, so one scale a
// row) are decoded on their way into LDS, and v = dy B enters as the bf16 value the fused GEMM takes
// plus the two bf16 values its rounding leaves, three MFMAs per fragment: the fp32 sums of v are then
// not rounded at all (with one remainder, 2^-16, grad_A was 3 times further from 64 bits than an fp32
// product; the products are small and their time is their loads').
constexpr int kActSteps = 2;  // contraction steps fetched at once: four tiles each

struct CodeRegs {
  uint2 c[2];
  float s[2];
};

// Thread t: codes of columns 8 (t%8) .. +7 of rows t/8 and t/8 + 32 of the tile at (r0, c0).
__device__ __forceinline__ void load_codes(const int8_t *codes, const float *scale, int64_t ld, int64_t nrows, int64_t r0,
                                           int64_t c0, int tid, CodeRegs &t) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = r0 + (tid >> 3) + 32 * h;
    const bool in = row < nrows;
    t.c[h] = in ? *(const uint2 *)(codes + row * ld + c0 + 8 * (tid & 7)) : make_uint2(0u, 0u);
    t.s[h] = in ? scale[row * (ld / kBlock) + c0 / kBlock] : 0.f;
  }
}

__device__ __forceinline__ void store_codes(const CodeRegs &t, uint16_t *lds, int tid) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *(u32x4 *)&lds[((tid >> 3) + 32 * h) * LLD + 8 * (tid & 7)] = act8_values(t.c[h].x, t.c[h].y, t.s[h]);
}

template <Edge kEdge>
__device__ __forceinline__ void act8_body(const Act8Problem &pr, int64_t kb, int64_t ke, int64_t m0, int64_t n0,
                                          uint16_t (*s)[LT * LLD], f32x16 &acc) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  uint16_t(*sh)[LT * LLD] = s, (*sm)[LT * LLD] = s + kActSteps, (*sl)[LT * LLD] = s + 2 * kActSteps;
  uint16_t(*sq)[LT * LLD] = s + 3 * kActSteps;
  TileRegs th[kActSteps], tm[kActSteps], tl[kActSteps];
  CodeRegs tq[kActSteps];
  auto fetch = [&](int64_t g0) {
#pragma unroll
    for (int st = 0; st < kActSteps; ++st) {
      const int64_t k0 = g0 + LT * st;
      load_tile<kEdge>(pr.P, pr.ldp, ke, pr.M, k0, m0, false, tid, th[st]);
      load_tile<kEdge>(pr.P_mid, pr.ldp, ke, pr.M, k0, m0, false, tid, tm[st]);
      load_tile<kEdge>(pr.P_low, pr.ldp, ke, pr.M, k0, m0, false, tid, tl[st]);
      load_codes((const int8_t *)pr.Q, pr.code_scale, pr.ldq, ke, k0, n0, tid, tq[st]);
    }
  };
  fetch(kb);
  for (int64_t g0 = kb; g0 < ke; g0 += LT * kActSteps) {
#pragma unroll
    for (int st = 0; st < kActSteps; ++st) {
      store_tile(th[st], sh[st], tid);
      store_tile(tm[st], sm[st], tid);
      store_tile(tl[st], sl[st], tid);
      store_codes(tq[st], sq[st], tid);
    }
    __syncthreads();
    if (g0 + LT * kActSteps < ke) fetch(g0 + LT * kActSteps);
#pragma unroll
    for (int st = 0; st < kActSteps; ++st)
#pragma unroll
      for (int kk = 0; kk < LT / 16; ++kk) {
        const u32x4 h = frag<true>(sh[st], wm * 32, kk, lane), m = frag<true>(sm[st], wm * 32, kk, lane);
        const u32x4 l = frag<true>(sl[st], wm * 32, kk, lane);
        const u32x4 q = frag<true>(sq[st], wn * 32, kk, lane);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(h), as_bf16x8(q), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(m), as_bf16x8(q), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(l), as_bf16x8(q), acc, 0, 0, 0);
      }
    __syncthreads();
  }
}

__device__ __forceinline__ void act8_tile(const Act8Problem &pr, int64_t tile, int s, uint16_t (*lds)[LT * LLD]) {
  const int64_t m0 = (tile % pr.tiles_m) * LT, n0 = (tile / pr.tiles_m) * LT;
  const int64_t kb = (int64_t)s * pr.chunk, ke = min(pr.Kc, kb + pr.chunk);
  f32x16 acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.f;
  if (m0 + LT <= pr.M && (ke - kb) % (LT * kActSteps) == 0)
    act8_body<kWhole>(pr, kb, ke, m0, n0, lds, acc);
  else if (pr.M >= 8)
    act8_body<kMasked>(pr, kb, ke, m0, n0, lds, acc);
  else if ((ke - 1) * pr.ldp + pr.M >= 8)
    act8_body<kNarrow>(pr, kb, ke, m0, n0, lds, acc);
  else
    act8_body<kTiny>(pr, kb, ke, m0, n0, lds, acc);
  put_tile<false>(pr, tile, s, acc);
}

// The products of one step of that backward pass, all in one launch (a launch costs about 4 us of the
// host and of the GPU, as much as one of these products): problem i takes workgroups first[i] ..
// first[i + 1] - 1.
constexpr int kMaxBatch = kMaxSetMembers + 1;
struct LoraBatch {
  Act8Problem pr[kMaxBatch];
  int64_t first[kMaxBatch + 1];
  int count;
};

__device__ __forceinline__ int batch_index(const LoraBatch &b, int64_t id) {
  int i = 0;
  while (i + 1 < b.count && id >= b.first[i + 1]) ++i;
  return i;
}

// v of every member.  9.5 us for 2048 x 4096 x 64: its reads' latency (17 MB).
__global__ __launch_bounds__(256) void lora_batch_v(LoraBatch b) {
  __shared__ __attribute__((aligned(16))) uint16_t s[8][LT * LLD];
  const int i = batch_index(b, blockIdx.x);
  const int64_t j = (int64_t)blockIdx.x - b.first[i];
  lora_tile<false, true, true, 4>(b.pr[i], j / b.pr[i].S, (int)(j % b.pr[i].S), s, s + 4);
}

// grad_A from the checkpoint (problem 0) and the members' grad_B.  13.6 us for 2048 x 4096 x 64, of which the reads of
// codes and dy (25 MB) would take 5: two workgroups a CU, each two to four round trips and its tile written out.
__global__ __launch_bounds__(256) void lora_batch_grads(LoraBatch b) {
  __shared__ __attribute__((aligned(16))) uint16_t s[8][LT * LLD];
  const int i = batch_index(b, blockIdx.x);
  const int64_t j = (int64_t)blockIdx.x - b.first[i];
  if (i == 0)
    act8_tile(b.pr[0], j / b.pr[0].S, (int)(j % b.pr[0].S), s);
  else
    lora_tile<true, true, false, 4>(b.pr[i], j / b.pr[i].S, (int)(j % b.pr[i].S), s, s + 4);
}

// first counts quads here
template <bool kBf16Out>
__global__ __launch_bounds__(256) void lora_batch_reduce(LoraBatch b) {
  const int64_t quads = b.first[b.count];
  for (int64_t qd = (int64_t)blockIdx.x * 256 + threadIdx.x; qd < quads; qd += (int64_t)gridDim.x * 256) {
    int i = 0;
    while (i + 1 < b.count && qd >= b.first[i + 1]) ++i;
    reduce_quad<kBf16Out>(b.pr[i], qd - b.first[i]);
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Contraction splits: about 256 workgroups in all, chunks of whole groups.
static int64_t lora_chunk(int64_t tiles, int64_t kc) {
  const int64_t grp = LT * 4;
  int64_t s = cdiv(256, tiles);
  const int64_t max_s = cdiv(kc, grp);
  if (s > max_s) s = max_s;
  if (s < 1) s = 1;
  return cdiv(cdiv(kc, s), grp) * grp;
}

int lora_splits(int64_t tiles, int64_t kc) { return (int)cdiv(kc, lora_chunk(tiles, kc)); }

int64_t lora_tiles(int64_t m, int64_t n) { return cdiv(m, LT) * cdiv(n, LT); }

size_t lora_part_floats(int64_t m, int64_t n, int64_t kc) {
  const int64_t tiles = lora_tiles(m, n);
  const int S = lora_splits(tiles, kc);
  return S > 1 ? (size_t)tiles * S * LT * LT : 0;
}

namespace {

LoraProblem make_problem(const uint16_t *P, int64_t ldp, const uint16_t *Q, int64_t ldq, int64_t M, int64_t Nc,
                         int64_t Kc, float scale, void *out, float *part) {
  LoraProblem pr;
  pr.P = P;
  pr.ldp = ldp;
  pr.Q = Q;
  pr.ldq = ldq;
  pr.M = M;
  pr.Nc = Nc;
  pr.Kc = Kc;
  pr.tiles_m = cdiv(M, LT);
  const int64_t tiles = lora_tiles(M, Nc);
  pr.chunk = lora_chunk(tiles, Kc);
  pr.S = (int)cdiv(Kc, pr.chunk);
  pr.scale = scale;
  pr.out = out;
  pr.ldo = Nc;
  pr.part = part;
  return pr;
}

int64_t problem_blocks(const LoraProblem &pr) { return lora_tiles(pr.M, pr.Nc) * pr.S; }
int64_t problem_quads(const LoraProblem &pr) { return pr.S > 1 ? lora_tiles(pr.M, pr.Nc) * (LT * LT / 4) : 0; }

// Launches one product (nb == nullptr) or two of the same operand forms; the
// two must agree on the split length.  A split of exactly 512 is fetched in
// one round trip (8 steps, 147 KB of LDS: one workgroup per CU) when the
// launch fits one round of 256 workgroups; a larger launch (the two gradient
// products) fetches groups of 4 steps, two workgroups per CU, so that all of
// it is resident at once.
template <bool kAT, bool kBT, bool kBf16Out>
hipError_t launch_pair(const LoraProblem &a, const LoraProblem *nb, hipStream_t st) {
  const LoraProblem b = nb ? *nb : a;
  const int64_t wa = problem_blocks(a), wb = nb ? problem_blocks(b) : 0;
  const bool whole = a.chunk == LT * 8 && wa + wb <= 256;
  if (whole)
    lora_gemm<kAT, kBT, kBf16Out, 8><<<(unsigned)(wa + wb), 256, 0, st>>>(a, b, wa);
  else
    lora_gemm<kAT, kBT, kBf16Out, 4><<<(unsigned)(wa + wb), 256, 0, st>>>(a, b, wa);
  const int64_t qa = problem_quads(a), qb = nb ? problem_quads(b) : 0;
  if (qa + qb > 0) {
    int64_t blocks = cdiv(qa + qb, 256);
    if (blocks > 2048) blocks = 2048;
    lora_reduce<kBf16Out><<<(unsigned)blocks, 256, 0, st>>>(a, b, qa, qa + qb);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(LoraKind kind, const uint16_t *P, int64_t ldp, const uint16_t *Q, int64_t ldq, int64_t M,
                       int64_t Nc, int64_t Kc, float scale, void *out, float *part, hipStream_t st) {
  const LoraProblem pr = make_problem(P, ldp, Q, ldq, M, Nc, Kc, scale, out, part);
  switch (kind) {
    case LoraKind::kU:  // x A^T
      return launch_pair<false, false, true>(pr, nullptr, st);
    case LoraKind::kV:  // dy B
      return launch_pair<false, true, true>(pr, nullptr, st);
    case LoraKind::kGrad:  // v^T x, dy^T u
      return launch_pair<true, true, false>(pr, nullptr, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_lora_grads(const uint16_t *v, const uint16_t *x, const uint16_t *dy, const uint16_t *u, int64_t T,
                             int64_t N, int64_t K, int r, float scale_a, float scale_b, float *grad_A, float *grad_B,
                             float *part, size_t part_a_floats, hipStream_t st) {
  // grad_A = s_a v^T x [r x K] and grad_B = s_b dy^T u [N x r], contraction over the tokens
  const LoraProblem a = make_problem(v, r, x, K, r, K, T, scale_a, grad_A, part);
  const LoraProblem b = make_problem(dy, N, u, r, N, r, T, scale_b, grad_B, part + part_a_floats);
  if ((a.chunk == LT * 8) == (b.chunk == LT * 8)) return launch_pair<true, true, false>(a, &b, st);
  const hipError_t e = launch_pair<true, true, false>(a, nullptr, st);
  return e != hipSuccess ? e : launch_pair<true, true, false>(b, nullptr, st);
}

// Adapter products of a projection set (members i < count, ranks r each).
size_t lora_set_part_floats(int64_t T, int count, const int64_t *N, int64_t K, int r) {
  size_t v = 0, g = lora_part_floats((int64_t)count * r, K, T);
  for (int i = 0; i < count; ++i) {
    v += lora_part_floats(T, r, N[i]);
    g += lora_part_floats(N[i], r, T);
  }
  return std::max(lora_part_floats(T, (int64_t)count * r, K), std::max(v, g));
}

// Runs a list of products of one operand form, two per launch where their
// group lengths agree.
template <bool kAT, bool kBT, bool kBf16Out>
static hipError_t launch_list(const LoraProblem *pr, int n, hipStream_t st) {
  for (int i = 0; i < n;) {
    hipError_t e;
    if (i + 1 < n && (pr[i].chunk == LT * 8) == (pr[i + 1].chunk == LT * 8)) {
      e = launch_pair<kAT, kBT, kBf16Out>(pr[i], &pr[i + 1], st);
      i += 2;
    } else {
      e = launch_pair<kAT, kBT, kBf16Out>(pr[i], nullptr, st);
      i += 1;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// v_set [T x count r]: columns [i r, i r + r) = dy_i B_i.
hipError_t launch_lora_set_v(const uint16_t *const *dy, const uint16_t *const *B, const int64_t *N, int count,
                             int64_t T, int r, uint16_t *v_set, float *part, hipStream_t st) {
  LoraProblem pr[kMaxSetMembers];
  size_t off = 0;
  for (int i = 0; i < count; ++i) {
    pr[i] = make_problem(dy[i], N[i], B[i], r, T, r, N[i], 1.0f, v_set + (int64_t)i * r, part + off);
    pr[i].ldo = (int64_t)count * r;
    off += lora_part_floats(T, r, N[i]);
  }
  return launch_list<false, true, true>(pr, count, st);
}

// grad_A_set = scale v_set^T x [count r x K] and grad_B_i = scale dy_i^T u_i [N_i x r]
// (u_i = columns [i r, i r + r) of u_set).
hipError_t launch_lora_set_grads(const uint16_t *v_set, const uint16_t *x, const uint16_t *const *dy,
                                 const uint16_t *u_set, const int64_t *N, int count, int64_t T, int64_t K, int r,
                                 float scale, float *grad_A_set, float *const *grad_B, float *part, hipStream_t st) {
  LoraProblem pr[kMaxSetMembers + 1];
  const int64_t rt = (int64_t)count * r;
  pr[0] = make_problem(v_set, rt, x, K, rt, K, T, scale, grad_A_set, part);
  size_t off = lora_part_floats(rt, K, T);
  for (int i = 0; i < count; ++i) {
    pr[i + 1] = make_problem(dy[i], N[i], u_set + (int64_t)i * r, rt, N[i], r, T, scale, grad_B[i], part + off);
    off += lora_part_floats(N[i], r, T);
  }
  return launch_list<true, true, false>(pr, count + 1, st);
}

static LoraBatch make_batch(const Act8Problem *pr, int count, int64_t (*size)(const LoraProblem &)) {
  LoraBatch b{};
  b.count = count;
  for (int i = 0; i < count; ++i) {
    b.pr[i] = pr[i];
    b.first[i + 1] = b.first[i] + size(pr[i]);
  }
  return b;
}

template <bool kBf16Out>
static hipError_t reduce_batch(const Act8Problem *pr, int count, hipStream_t st) {
  const LoraBatch b = make_batch(pr, count, problem_quads);
  if (b.first[count] > 0)
    lora_batch_reduce<kBf16Out><<<(unsigned)std::min<int64_t>(cdiv(b.first[count], 256), 2048), 256, 0, st>>>(b);
  return hipGetLastError();
}

// Rows of a member up to which v is not split over them: the reduction is a launch more, of 3 us on the host (16 tokens,
// 512 x 1024: 37 -> 33 us; 1000 tokens the same; at 1024 rows, or for the gradients' sums over the tokens, the longer
// loop costs more than it spares: 500 tokens, 1000 x 512 52 -> 61 us).
constexpr int64_t kWholeRows = 512;

// v_set with what its rounding leaves: v [3][T x count r].
hipError_t launch_lora_set_v_exact(const uint16_t *const *dy, const uint16_t *const *B, const int64_t *N, int count,
                                   int64_t T, int r, uint16_t *v, float *part, hipStream_t st) {
  const int64_t plane = T * count * r;
  Act8Problem pr[kMaxSetMembers] = {};
  size_t off = 0;
  for (int i = 0; i < count; ++i) {
    (LoraProblem &)pr[i] = make_problem(dy[i], N[i], B[i], r, T, r, N[i], 1.0f, v + (int64_t)i * r, part + off);
    if (N[i] <= kWholeRows) {
      pr[i].chunk = cdiv(N[i], 4 * LT) * (4 * LT);
      pr[i].S = 1;
    }
    pr[i].ldo = (int64_t)count * r;
    pr[i].out_mid = v + plane + (int64_t)i * r;
    pr[i].out_low = v + 2 * plane + (int64_t)i * r;
    off += lora_part_floats(T, r, N[i]);
  }
  LoraBatch b = make_batch(pr, count, problem_blocks);
  lora_batch_v<<<(unsigned)b.first[count], 256, 0, st>>>(b);
  return reduce_batch<true>(pr, count, st);
}

// grad_A_set and every grad_B in one launch.
hipError_t launch_lora_set_grads_act8(const uint16_t *v, const int8_t *codes, const float *code_scale,
                                      const uint16_t *const *dy, const uint16_t *u_set,
                                      const int64_t *N, int count, int64_t T, int64_t K, int r, float scale,
                                      float *grad_A_set, float *const *grad_B, float *part, hipStream_t st) {
  Act8Problem pr[kMaxBatch] = {};
  const int64_t rt = (int64_t)count * r;
  Act8Problem &a = pr[0];
  (LoraProblem &)a = make_problem(v, rt, (const uint16_t *)codes, K, rt, K, T, scale, grad_A_set, part);
  a.P_mid = v + T * rt;
  a.P_low = v + 2 * T * rt;
  a.code_scale = code_scale;
  size_t off = lora_part_floats(rt, K, T);
  for (int i = 0; i < count; ++i) {
    (LoraProblem &)pr[i + 1] = make_problem(dy[i], N[i], u_set + (int64_t)i * r, rt, N[i], r, T, scale, grad_B[i], part + off);
    off += lora_part_floats(N[i], r, T);
  }
  LoraBatch b = make_batch(pr, count + 1, problem_blocks);
  lora_batch_grads<<<(unsigned)b.first[count + 1], 256, 0, st>>>(b);
  return reduce_batch<false>(pr, count + 1, st);
}

}  // namespace qlora
