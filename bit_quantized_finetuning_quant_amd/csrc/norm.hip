// Root-mean-square norm with the residual's addition, and its backward pass
// (gfx950).
//
//   s    = bf16(x + residual)                          the residual stream's next value
//   rstd = 1 / sqrt(mean_d s_td^2 + eps)
//   y    = bf16(w_d (s_td rstd_t))                     and / or y as an 8-bit checkpoint
//
//   xhat = s rstd,   c_t = mean_d(w_d dy_td xhat_td)
//   grad_s = bf16(dres + rstd (w dy - xhat c)),        grad_w_d = sum_t dy_td xhat_td
//
// A row stays in registers between its sums and its results, so every value
// crosses HBM once.  The backward pass forms rstd again from s, which it
// reads anyway, in the same reduction as c: nothing is kept for it.
// Sums and statistics are fp32; s, y and grad_s round once.
//
// What bounds it is HBM, and for few rows the launch.  On this card's 5.35 TB/s of a 512 MB copy: forward 2048 x 4096 with
// the residual (67 MB) 14.0 us with inputs in turn, 4.8 TB/s, and 11.3 where they lie in the last-level cache; 4096 x 8192 in
// 8 bits too (305 MB) 51; backward 4096 x 8192 with the residual's gradient (268 MB) 51 us, 5.2 TB/s, with the weight's 55 and
// the launch that adds it 5.  One row of 4096: 2.9 us.
//
// Squares past fp32 (a row with |s| > 1.8e19) make the sum infinite, or an eps near fp32's end the mean; the row is
// then summed again with s scaled by 2^-96.  Only the sums take scaled values (those below 2^-30 lose bits there, which
// are nothing beside 2^128); xhat is s times 2^-96 rstd, which is at least 2^-128 and off by 2^-22 of itself at most, where it
// is subnormal.

#include <algorithm>

#include "act8.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace qlora {

namespace {

// w[8 i .. 8 i + 7]
__device__ __forceinline__ void weight8(const void *w, bool wide, int i, float (&out)[8]) {
  if (wide) {
    const f32x4 a = ((const f32x4 *)w)[2 * i], b = ((const f32x4 *)w)[2 * i + 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[j] = a[j];
      out[4 + j] = b[j];
    }
  } else {
    const u32x4 a = ((const u32x4 *)w)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t p = a[j];
      out[2 * j] = bf16_lo(p);
      out[2 * j + 1] = bf16_hi(p);
    }
  }
}

__device__ __forceinline__ void unpack8(const u32x4 &v, float (&out)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t p = v[j];
    out[2 * j] = bf16_lo(p);
    out[2 * j + 1] = bf16_hi(p);
  }
}

// The sums of N values over the kRow threads of a row, the same in all of them.  red: a row's slots.
template <int kRow, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = row16_sum(v[k]);
    v[k] = fold<16>(v[k], v[k]);
    v[k] = fold<32>(v[k], v[k]);
  }
  if constexpr (kRow > 64) {
    constexpr int kWaves = kRow / 64;
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // the slots' last values have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) red[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = red[0][k];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v[k] += red[w][k];
    }
  }
}

constexpr float kLift = 0x1p-96f;  // of s, for rows whose squares pass fp32

template <int kRow>
constexpr int block_threads() {
  return kRow < 256 ? 256 : kRow;
}

struct NormFwd {
  const uint16_t *x, *residual;
  int64_t T;
  int D;
  const void *weight;
  bool wide;
  float eps;
  uint16_t *sum, *y;
  int8_t *codes;
  float *scale;
};

// kRow threads a row, V runs of 8 values a thread, a row's threads apart.
template <int kRow, int V, bool kStream>
__global__ __launch_bounds__(block_threads<kRow>()) void rms_norm_fwd(NormFwd p) {
  constexpr int kRows = block_threads<kRow>() / kRow;
  __shared__ float red[block_threads<kRow>() / 64][1];
  const int lane = threadIdx.x % kRow, runs = p.D / 8;
  for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow; t < p.T; t += (int64_t)gridDim.x * kRows) {
    u32x4 s[V];
    const int64_t row = t * p.D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + v * kRow;
      s[v] = i < runs ? load_run<kStream>(p.x + row + 8 * i) : u32x4{0u, 0u, 0u, 0u};
    }
    if (p.residual) {
      u32x4 r[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = lane + v * kRow;
        r[v] = i < runs ? load_run<kStream>(p.residual + row + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = lane + v * kRow;
        float a[8], b[8];
        unpack8(s[v], a);
        unpack8(r[v], b);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[v][j] = pack_bf16x2(a[2 * j] + b[2 * j], a[2 * j + 1] + b[2 * j + 1]);
        if (i < runs) *(u32x4 *)(p.sum + row + 8 * i) = s[v];
      }
    }
    float lift = 1.0f, rstd;  // rstd of s lift
    for (;;) {
      float sq[1] = {0.f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a[8];
        unpack8(s[v], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float l = a[j] * lift;
          sq[0] = __builtin_fmaf(l, l, sq[0]);
        }
      }
      row_sum<kRow>(sq, red);
      const float mean = sq[0] / (float)p.D + p.eps * lift * lift;
      rstd = 1.0f / sqrtf(mean);
      if (lift != 1.0f || mean < __builtin_inff()) break;  // (a NaN's sum is summed again, to the same)
      lift = kLift;
    }
    const float outer = rstd * lift;  // 1 / the root of the mean square
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + v * kRow;
      if (i >= runs) continue;
      float a[8], w[8];
      unpack8(s[v], a);
      weight8(p.weight, p.wide, i, w);
      u32x4 y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack_bf16x2(w[2 * j] * (a[2 * j] * outer), w[2 * j + 1] * (a[2 * j + 1] * outer));
      if (p.y) *(u32x4 *)(p.y + row + 8 * i) = y;
      if (p.codes) {
        float block;
        const act8_u32x2 c = encode_block(y, block);
        *(act8_u32x2 *)(p.codes + row + 8 * i) = c;
        if ((i & 7) == 0) p.scale[(row >> 6) + (i >> 3)] = block;
      }
    }
  }
}

struct NormBwd {
  const uint16_t *dy, *s, *dres;
  int64_t T;
  int D;
  const void *weight;
  bool wide;
  float eps;
  uint16_t *grad;
  float *part;  // with the weight's gradient: [workgroup][D]
};

// One row: rstd (of s lifted) and c from the sums of s^2 and w dy s.  false: mean s^2 + eps passes fp32.  (c may do so where
// its value does not: it is not finite then, and norm_mean forms it.)
template <int kRow, int V, bool kLifted, typename W>
__device__ __forceinline__ bool norm_sums(const NormBwd &p, const u32x4 (&s)[V], const u32x4 (&g)[V], const W &weight,
                                          float (*red)[2], float &rstd, float &c) {
  const float lift = kLifted ? kLift : 1.0f;
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8], b[8], w[8];
    unpack8(s[v], a);
    unpack8(g[v], b);
    weight(v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float l = kLifted ? a[j] * lift : a[j];
      sum[0] = __builtin_fmaf(l, l, sum[0]);
      sum[1] = __builtin_fmaf(w[j] * b[j], l, sum[1]);
    }
  }
  row_sum<kRow>(sum, red);
  const float mean = sum[0] / (float)p.D + p.eps * lift * lift;
  rstd = 1.0f / sqrtf(mean);
  c = sum[1] * rstd / (float)p.D;
  return mean < __builtin_inff();
}

// c as the sum of w dy xhat / D, whose partial sums are at most the largest |w dy| (a second reduction, for rows whose
// products w dy s pass fp32 before rstd brings them back).
template <int kRow, int V, typename W>
__device__ __forceinline__ float norm_mean(const u32x4 (&s)[V], const u32x4 (&g)[V], const W &weight, float (*red)[2],
                                           float outer, int D) {
  const float part = 1.0f / (float)D;
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8], b[8], w[8];
    unpack8(s[v], a);
    unpack8(g[v], b);
    weight(v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0] = __builtin_fmaf(w[j] * b[j], a[j] * outer * part, sum[0]);
  }
  row_sum<kRow>(sum, red);
  return sum[0];
}

// The weight stays in registers over a workgroup's rows where it has room there.
template <int kRow, int V, bool kWeight, bool kStream>
__global__ __launch_bounds__(block_threads<kRow>()) void rms_norm_bwd(NormBwd p) {
  constexpr int kRows = block_threads<kRow>() / kRow;
  constexpr bool kHeld = V <= 2;
  __shared__ float red[block_threads<kRow>() / 64][2];
  const int lane = threadIdx.x % kRow, runs = p.D / 8;
  float held[kHeld ? V : 1][8];
  if constexpr (kHeld)
#pragma unroll
    for (int v = 0; v < V; ++v) weight8(p.weight, p.wide, min(lane + v * kRow, runs - 1), held[v]);
  auto weight = [&](int v, float (&w)[8]) {
    if constexpr (kHeld) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = held[v][j];
    } else {
      weight8(p.weight, p.wide, min(lane + v * kRow, runs - 1), w);
    }
  };
  float gw[kWeight ? V : 1][8];
#pragma unroll
  for (int v = 0; v < (kWeight ? V : 1); ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[v][j] = 0.f;
  const int64_t first = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow, step = (int64_t)gridDim.x * kRows;
  auto load = [&](int64_t t, u32x4 (&s)[V], u32x4 (&g)[V], u32x4 (&d)[V]) {
    const int64_t row = t * p.D;
    const u32x4 none = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + v * kRow;
      s[v] = i < runs ? load_run<kStream>(p.s + row + 8 * i) : none;
      g[v] = i < runs ? load_run<kStream>(p.dy + row + 8 * i) : none;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + v * kRow;
      d[v] = p.dres && i < runs ? load_run<kStream>(p.dres + row + 8 * i) : none;
    }
  };
  for (int64_t t = first; t < p.T; t += step) {
    const int64_t row = t * p.D;
    u32x4 s[V], g[V], d[V];
    load(t, s, g, d);
    float lift = 1.0f, rstd, c;
    if (!norm_sums<kRow, V, false>(p, s, g, weight, red, rstd, c)) {  // (a NaN's row too, to the same end)
      lift = kLift;
      norm_sums<kRow, V, true>(p, s, g, weight, red, rstd, c);
    }
    const float outer = rstd * lift;  // 1 / the root of the mean square
    if (!(__builtin_fabsf(c) < __builtin_inff())) c = norm_mean<kRow, V>(s, g, weight, red, outer, p.D);
    // long rows are unpacked again below: unpacked over the sums they would take twice the registers, and spill
    if constexpr (V > 2)
#pragma unroll
      for (int v = 0; v < V; ++v) asm("" : "+v"(s[v]), "+v"(g[v]));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + v * kRow;
      float a[8], b[8], w[8], o[8], past[8];
      unpack8(s[v], a);
      unpack8(g[v], b);
      unpack8(d[v], past);
      weight(v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = a[j] * outer;
        o[j] = outer * (w[j] * b[j] - xhat * c);
        if (p.dres) o[j] += past[j];
        if constexpr (kWeight) gw[v][j] = __builtin_fmaf(b[j], xhat, gw[v][j]);
      }
      if (i < runs)
        *(u32x4 *)(p.grad + row + 8 * i) = u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                                pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
    }
  }
  if constexpr (kWeight) {
    // the workgroup's rows side by side are added first
    __shared__ __attribute__((aligned(16))) float sums[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? V * kRow * 8 : 1];
    if constexpr (kRows > 1) {
      const int mine = threadIdx.x / kRow;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (mine > 0) sums[mine - 1][j * V * kRow + lane + v * kRow] = gw[v][j];
      __syncthreads();
      if (mine > 0) return;
#pragma unroll
      for (int k = 0; k < kRows - 1; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) gw[v][j] += sums[k][j * V * kRow + lane + v * kRow];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + v * kRow;
      if (i >= runs) continue;
      float *dst = p.part + (int64_t)blockIdx.x * p.D + 8 * i;
      *(f32x4 *)dst = f32x4{gw[v][0], gw[v][1], gw[v][2], gw[v][3]};
      *(f32x4 *)(dst + 4) = f32x4{gw[v][4], gw[v][5], gw[v][6], gw[v][7]};
    }
  }
}

// grad_w from the workgroups' sums: 64 columns a workgroup, its 16 waves every 16th of them each, in a fixed order.
__global__ __launch_bounds__(1024) void rms_norm_weight(const float *__restrict__ part, int groups, int D,
                                                       float *__restrict__ grad) {
  __shared__ float sums[16][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), wave = threadIdx.x >> 6;
  float s = 0.f;
#pragma unroll 8
  for (int g = wave; g < groups; g += 16) s += part[(int64_t)g * D + col];
  sums[wave][threadIdx.x & 63] = s;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) s += sums[w][threadIdx.x];
  grad[col] = s;
}

// A row's threads and runs, every run in registers.  The backward pass holds three rows' worth and takes at most two
// runs a thread up to 16384 columns (4096 x 8192: four runs 73.6 us, two 64.7, one 72.7).
template <bool kBackward, typename F>
void with_shape(int64_t D, const F &f) {
  const int64_t runs = D / 8;
  auto shape = [&](auto row, auto per) { f(row, per); };
#define NORM_SHAPE(ROW, RUNS) shape(std::integral_constant<int, ROW>(), std::integral_constant<int, RUNS>())
  if (runs <= 64)
    NORM_SHAPE(64, 1);
  else if (runs <= 128)
    NORM_SHAPE(64, 2);
  else if (runs <= 256)
    NORM_SHAPE(256, 1);
  else if (runs <= 512)
    NORM_SHAPE(256, 2);
  else if (runs <= 1024)
    kBackward ? NORM_SHAPE(512, 2) : NORM_SHAPE(256, 4);
  else if (runs <= 2048)
    kBackward ? NORM_SHAPE(1024, 2) : NORM_SHAPE(512, 4);
  else if (runs <= 4096)
    NORM_SHAPE(1024, 4);
  else
    NORM_SHAPE(1024, 8);
#undef NORM_SHAPE
}

int rows_of_block(int64_t D) { return D <= 1024 ? 4 : 1; }

// Workgroups of the launch with the weight's gradient: each holds partial sums of a row's length, written and read
// again, so they are few; two a CU of 256 threads, one of 512 or more (4096 x 8192: 51.4 us with two, 49.0 with one, 512 x
// 8192 16.9 and 13.2; 2048 x 4096 16.9 with two, 19.5 with one).
int64_t weight_blocks(int64_t T, int64_t D) {
  const int rows = rows_of_block(D);
  return std::min<int64_t>((T + rows - 1) / rows, D <= 4096 ? 512 : 256);
}

// Workgroups of a launch of one row (or four) each; past 2^20 they take several in turn.
int64_t row_blocks(int64_t T, int64_t D) {
  const int rows = rows_of_block(D);
  return std::min<int64_t>((T + rows - 1) / rows, (int64_t)1 << 20);
}

}  // namespace

hipError_t launch_rms_norm_fwd(const uint16_t *x, const uint16_t *residual, int64_t T, int64_t D, const void *weight,
                               bool w_fp32, float eps, uint16_t *sum, uint16_t *y, int8_t *codes, float *scale,
                               hipStream_t st) {
  const NormFwd p{x, residual, T, (int)D, weight, w_fp32, eps, sum, y, codes, scale};
  with_shape<false>(D, [&](auto row, auto runs) {
    constexpr int kThreads = block_threads<row()>();
    if (T * D * (residual ? 4 : 2) >= kStreamBytes)
      rms_norm_fwd<row(), runs(), true><<<(unsigned)row_blocks(T, D), kThreads, 0, st>>>(p);
    else
      rms_norm_fwd<row(), runs(), false><<<(unsigned)row_blocks(T, D), kThreads, 0, st>>>(p);
  });
  return hipGetLastError();
}

size_t rms_norm_part_floats(int64_t T, int64_t D) { return (size_t)(weight_blocks(T, D) * D); }

hipError_t launch_rms_norm_bwd(const uint16_t *dy, const uint16_t *s, const uint16_t *dres, int64_t T, int64_t D,
                               const void *weight, bool w_fp32, float eps, uint16_t *grad_s, float *grad_weight,
                               float *part, hipStream_t st) {
  const NormBwd p{dy, s, dres, T, (int)D, weight, w_fp32, eps, grad_s, part};
  with_shape<true>(D, [&](auto row, auto runs) {
    constexpr int kThreads = block_threads<row()>();
    const bool stream = T * D * (dres ? 6 : 4) >= kStreamBytes;
    const unsigned blocks = (unsigned)(grad_weight ? weight_blocks(T, D) : row_blocks(T, D));
    if (grad_weight && stream)
      rms_norm_bwd<row(), runs(), true, true><<<blocks, kThreads, 0, st>>>(p);
    else if (grad_weight)
      rms_norm_bwd<row(), runs(), true, false><<<blocks, kThreads, 0, st>>>(p);
    else if (stream)
      rms_norm_bwd<row(), runs(), false, true><<<blocks, kThreads, 0, st>>>(p);
    else
      rms_norm_bwd<row(), runs(), false, false><<<blocks, kThreads, 0, st>>>(p);
  });
  if (grad_weight)
    rms_norm_weight<<<(unsigned)(D / 64), 1024, 0, st>>>(part, (int)weight_blocks(T, D), (int)D, grad_weight);
  return hipGetLastError();
}

}  // namespace qlora
