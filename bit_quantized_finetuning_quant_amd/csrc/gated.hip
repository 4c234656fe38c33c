// The gated product of a feed-forward block (gfx950): h = act(gate) up behind
// the projections of a gate and an up weight, the product alone, and its
// backward pass.
//
//   gate = x Wg^T + s u_g Bg^T,   up = x Wu^T + s u_u Bu^T,   h = bf16(act(gate) up)
//   dgate = bf16(dh up act'(gate)),   dup = bf16(dh act(gate))
//
// Behind the projections the product takes gate and up in fp32; the bf16 copies
// of both are what the backward pass reads, and need not be written.

#include <algorithm>

#include "act8.hpp"
#include "common.hpp"
#include "gated.hpp"
#include "launch.hpp"

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kRuns = 2;  // runs of 8 values a thread takes, a workgroup's stride apart

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
template <Activation kAct>
__global__ __launch_bounds__(kThreads) void gated_act_fwd(const uint16_t *gate, const uint16_t *up, int64_t runs,
                                                         uint16_t *h, int8_t *codes, float *scale) {
  const int64_t step = (int64_t)gridDim.x * (kThreads * kRuns);
  for (int64_t first = (int64_t)blockIdx.x * (kThreads * kRuns) + threadIdx.x; first < runs; first += step) {
    u32x4 g[kRuns], u[kRuns];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kThreads;
      g[j] = i < runs ? *(const u32x4 *)(gate + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      u[j] = i < runs ? *(const u32x4 *)(up + 8 * i) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kThreads;
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

template <Activation kAct>
__global__ __launch_bounds__(kThreads) void gated_act_bwd(const uint16_t *dh, const uint16_t *gate, const uint16_t *up,
                                                         int64_t runs, uint16_t *dgate, uint16_t *dup) {
  const int64_t step = (int64_t)gridDim.x * (kThreads * kRuns);
  for (int64_t first = (int64_t)blockIdx.x * (kThreads * kRuns) + threadIdx.x; first < runs; first += step) {
    u32x4 d[kRuns], g[kRuns], u[kRuns];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kThreads;
      d[j] = i < runs ? *(const u32x4 *)(dh + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      g[j] = i < runs ? *(const u32x4 *)(gate + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      u[j] = i < runs ? *(const u32x4 *)(up + 8 * i) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int64_t i = first + j * kThreads;
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

// h (and what else `out` names) from the fused GEMM's partial tiles part[z][T][2 N], added in order; 8 columns a thread.
template <Activation kAct>
__global__ __launch_bounds__(kThreads) void gated_reduce(const float *__restrict__ part, int parts, int64_t T, int64_t N,
                                                        GatedOut out) {
  const int64_t runs = T * N / 8, zs = 2 * T * N;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < runs; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = 8 * i / N, col = 8 * i - row * N;
    const float *p = part + row * (2 * N) + col;
    f32x4 v[4] = {};
#pragma unroll 4
    for (int z = 0; z < parts; ++z)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f32x4 a = *(const f32x4 *)(p + z * zs + (k >> 1) * N + 4 * (k & 1));
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k][q] += a[q];
      }
    u32x4 h, g, u;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float g0 = v[k][2 * q], g1 = v[k][2 * q + 1], u0 = v[2 + k][2 * q], u1 = v[2 + k][2 * q + 1];
        h[2 * k + q] = pack_bf16x2(gate_act<kAct>(g0) * u0, gate_act<kAct>(g1) * u1);
        g[2 * k + q] = pack_bf16x2(g0, g1);
        u[2 * k + q] = pack_bf16x2(u0, u1);
      }
    store_gated(out, 8 * i, h, g, u);
  }
}

// One pass of a workgroup each, up to 2^22 of them.
unsigned grid(int64_t runs) {
  return (unsigned)std::min<int64_t>((runs + kThreads * kRuns - 1) / (kThreads * kRuns), (int64_t)1 << 22);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

hipError_t launch_gated_act_fwd(const uint16_t *gate, const uint16_t *up, int64_t T, int64_t N, Activation act,
                                uint16_t *h, int8_t *codes, float *scale, hipStream_t st) {
  const int64_t runs = T * N / 8;
  with_activation(act, [&](auto a) {
    gated_act_fwd<a()><<<grid(runs), kThreads, 0, st>>>(gate, up, runs, h, codes, scale);
  });
  return hipGetLastError();
}

hipError_t launch_gated_act_bwd(const uint16_t *dh, const uint16_t *gate, const uint16_t *up, int64_t T, int64_t N,
                                Activation act, uint16_t *dgate, uint16_t *dup, hipStream_t st) {
  const int64_t runs = T * N / 8;
  with_activation(act, [&](auto a) {
    gated_act_bwd<a()><<<grid(runs), kThreads, 0, st>>>(dh, gate, up, runs, dgate, dup);
  });
  return hipGetLastError();
}

GatedPlan plan_linear_gated(int64_t T, int64_t N, int64_t K, int r) {
  GatedPlan p{};
  p.T = T;
  p.N = N;
  p.K = K;
  p.r = r;
  p.few = gemv_fwd_applies(T, 2 * N, K);
  p.parts = p.few ? 0 : qgemm_gated_parts(T, N, K);
  const int64_t both[2] = {N, N};
  size_t off = 256;
  p.off_u = off;
  off += align256((size_t)T * 2 * r * 2);
  p.off_part = off;
  off += align256((p.few ? gemv_set_fwd_part_floats(T, both, 2, K, r) : lora_part_floats(T, 2 * r, K)) * 4);
  p.off_qpart = off;
  off += align256((size_t)p.parts * T * 2 * N * 4);
  p.total = off;
  return p;
}

hipError_t launch_linear_gated_fwd(const GatedPlan &p, const uint16_t *x, const QWeight *w, const uint16_t *A_set,
                                   const uint16_t *const *B, float scale, const GatedOut &out, uint16_t *u_out,
                                   char *ws, const Codebook &cb, hipStream_t st) {
  uint16_t *u = u_out ? u_out : (uint16_t *)(ws + p.off_u);
  float *part = (float *)(ws + p.off_part), *qpart = (float *)(ws + p.off_qpart);
  if (p.few) return launch_gemv_gated(p.T, x, w, A_set, B, p.r, scale, out, u, part, cb, st);
  hipError_t e = launch_lora(LoraKind::kU, x, p.K, A_set, p.K, p.T, 2 * p.r, p.K, 1.0f, u, part, st);
  if (e != hipSuccess) return e;
  QgemmSet s{};
  for (int i = 0; i < 2; ++i) {
    s.m[i].w = w[i];
    s.m[i].lb = B[i];
  }
  e = launch_qgemm_gated(s, p.T, x, u, p.r, scale, out, qpart, cb, st);
  if (e != hipSuccess || p.parts == 0) return e;
  const int64_t blocks = (p.T * p.N / 8 + kThreads - 1) / kThreads;
  with_activation(out.act, [&](auto a) {
    gated_reduce<a()><<<(unsigned)std::min<int64_t>(blocks, 2048), kThreads, 0, st>>>(qpart, p.parts, p.T, p.N, out);
  });
  return hipGetLastError();
}

}  // namespace qlora
