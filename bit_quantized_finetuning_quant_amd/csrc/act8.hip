// 8-bit activation checkpoints (gfx950): the input of a linear layer kept in
// 8.5 instead of 16 bits per value until the backward pass, which needs it for
// grad_A only.
//
//   c1_b  = max |x| over 64 columns of a token,   scale_b = fl32(c1_b / 127)
//   code  = the integer nearest to the exact 127 x / c1_b, ties to the even one
//   x_hat = bf16( fl32(code scale_b) )
//
// A NaN or Inf makes the scale of its block NaN, so the whole block reads back
// as NaN: nothing is lost silently.  A block of zeros has scale 0.
//
// Both kernels are bound by HBM: 3.06 bytes a value are moved, once, in runs of
// 1 KB (x) and 512 bytes (codes) a wave.  4096 x 22016: write 45.5 us (6.1 TB/s,
// non-temporal; 50.1 us with ordinary accesses), read 43.6 us (6.3 TB/s; its
// result is read next, and non-temporal stores made it 46.8 us); a plain copy
// of 1 GB reaches 5.2 TB/s.

#include <algorithm>

#include "act8.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kRuns = 4;  // runs of 8 values a thread takes, a workgroup's stride apart

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

// Values [8 i, 8 i + 8) of x per thread and run; 8 consecutive lanes share a block.
__global__ __launch_bounds__(kThreads) void act8_encode(const uint16_t *__restrict__ x, int64_t runs,
                                                       int8_t *__restrict__ codes, float *__restrict__ scale) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kRuns) + threadIdx.x;
  u32x4 v[kRuns];
#pragma unroll
  for (int j = 0; j < kRuns; ++j) {
    const int64_t i = first + j * kThreads;
    v[j] = i < runs ? __builtin_nontemporal_load((const u32x4 *)(x + 8 * i)) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int j = 0; j < kRuns; ++j) {
    const int64_t i = first + j * kThreads;
    float block;
    const u32x2v c = encode_block(v[j], block);
    if (i >= runs) continue;
    __builtin_nontemporal_store(c, (u32x2v *)(codes + 8 * i));
    if ((i & 7) == 0) scale[i >> 3] = block;
  }
}

// 8 codes (an eighth of a block) per thread and run.
__global__ __launch_bounds__(kThreads) void act8_decode(const int8_t *__restrict__ codes,
                                                       const float *__restrict__ scale, int64_t runs,
                                                       uint16_t *__restrict__ x) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kRuns) + threadIdx.x;
  u32x2v c[kRuns];
  float s[kRuns];
#pragma unroll
  for (int j = 0; j < kRuns; ++j) {
    const int64_t i = first + j * kThreads;
    c[j] = i < runs ? *(const u32x2v *)(codes + 8 * i) : u32x2v{0u, 0u};
    s[j] = i < runs ? scale[i >> 3] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kRuns; ++j) {
    const int64_t i = first + j * kThreads;
    if (i < runs) *(u32x4 *)(x + 8 * i) = act8_values(c[j][0], c[j][1], s[j]);
  }
}

size_t aligned(size_t v) { return (v + 255) & ~(size_t)255; }

unsigned grid(int64_t runs) { return (unsigned)((runs + kThreads * kRuns - 1) / (kThreads * kRuns)); }

}  // namespace

hipError_t launch_act8_encode(const uint16_t *x, int64_t T, int64_t K, int8_t *codes, float *scale, hipStream_t st) {
  const int64_t runs = T * K / 8;
  act8_encode<<<grid(runs), kThreads, 0, st>>>(x, runs, codes, scale);
  return hipGetLastError();
}

hipError_t launch_act8_decode(const int8_t *codes, const float *scale, int64_t T, int64_t K, uint16_t *x,
                              hipStream_t st) {
  const int64_t runs = T * K / 8;
  act8_decode<<<grid(runs), kThreads, 0, st>>>(codes, scale, runs, x);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Backward from an 8-bit checkpoint of the input.  Any token count runs on the
// fused GEMM and the adapter products (a checkpoint of a few tokens saves
// nothing, so there is no few-token form).

// v's three planes, and the partial tiles of the products: those of one step are at most count + 1 products (grad_A and
// every grad_B), of which one splits only with fewer than 256 tiles, in about 256 workgroups (510 at most).
size_t act8_bound(int64_t T, int count, int r) {
  return 256 + aligned((size_t)6 * T * count * r) + (size_t)(count + 1) * 510 * 64 * 64 * 4;
}

Act8BwdPlan plan_linear_set_act8(int64_t T, int count, const int64_t *N, int64_t K, int r, bool lean) {
  Act8BwdPlan p;
  p.T = T;
  p.K = K;
  p.r = r;
  p.count = count;
  bool same_n = true;
  for (int i = 0; i < kMaxSetMembers; ++i) {
    p.N[i] = i < count ? N[i] : 0;
    same_n = same_n && (i >= count || N[i] == N[0]);
  }
  size_t off = 256;
  p.off_v = off;
  off += aligned((size_t)3 * T * count * r * 2);
  p.off_part = off;
  off += aligned(lora_set_part_floats(T, count, N, K, r) * 4);
  p.ragged = !lean && ragged_dx_applies(T, count, N, K, r);
  p.off_qpart = p.off_rg = 0;
  if (lean) {
    p.total = off;
    return p;
  }
  if (p.ragged) {
    p.rg = plan_ragged_dx(T, count, N, K, r);
    p.off_rg = off;
    off += p.rg.total;
  } else {
    size_t qsplit = same_n ? qgemm_split_floats(T, K, N[0]) : 0;
    if (count > 1) qsplit = std::max(qsplit, qgemm_set_dx_member_floats(T, count, N, K));
    p.off_qpart = qsplit ? off : 0;
    off += aligned(qsplit * 4);
  }
  p.total = off;
  return p;
}

hipError_t launch_linear_set_bwd_act8(const Act8BwdPlan &p, const uint16_t *const *dy, const int8_t *codes,
                                      const float *code_scale, const QWeight *w, const uint16_t *A_set,
                                      const uint16_t *const *B, float scale, const uint16_t *u, uint16_t *grad_x,
                                      float *grad_A_set, float *const *grad_B, char *ws, const Codebook &cb,
                                      hipStream_t st) {
  float *part = (float *)(ws + p.off_part);
  uint16_t *v = (uint16_t *)(ws + p.off_v);
  const int64_t rt = (int64_t)p.count * p.r;
  hipError_t e = launch_lora_set_v_exact(dy, B, p.N, p.count, p.T, p.r, v, part, st);
  if (e != hipSuccess) return e;
  if (grad_x && p.ragged) {
    e = launch_ragged_dx(p.rg, p.T, p.count, p.N, p.K, p.r, dy, w, v, A_set, scale, grad_x, ws + p.off_rg, cb, st);
    if (e != hipSuccess) return e;
  } else if (grad_x) {
    QgemmSet s{};
    s.count = p.count;
    s.ld_la = rt;
    for (int i = 0; i < p.count; ++i) {
      s.m[i].w = w[i];
      s.m[i].act = dy[i];
    }
    TimedLaunch tl;
    const bool timed = timing_begin(st, tl, kTimedQgemmDx);
    e = launch_qgemm_set(true, s, p.T, nullptr, v, A_set, (int)rt, scale, grad_x, cb, st, nullptr,
                         p.off_qpart ? (float *)(ws + p.off_qpart) : nullptr);
    if (timed) timing_end(st, tl);
    if (e != hipSuccess) return e;
  }
  return launch_lora_set_grads_act8(v, codes, code_scale, dy, u, p.N, p.count, p.T, p.K, p.r, scale, grad_A_set,
                                    grad_B, part, st);
}

}  // namespace qlora
