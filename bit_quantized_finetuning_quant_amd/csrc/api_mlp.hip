// C ABI of what stands around the linears of a feed-forward block (declared in
// include/qlora.h): the root-mean-square norm and the gated product, with their
// backward passes.  Host code only.

#include <string.h>

#include <initializer_list>

#include "validate.hpp"

using namespace qlora;

namespace {

// An enumeration's code read as an integer: a caller may pass any value.
template <typename E>
int code_of(const E &e) {
  int v;
  memcpy(&v, &e, sizeof v);
  return v;
}

bool norm_shape_ok(int64_t T, int64_t D) { return D <= kNormMaxDim && product_ok(T, D) && D % kBlock == 0; }
bool act_shape_ok(int64_t T, int64_t N) { return product_ok(T, N) && N % kBlock == 0; }

// A checkpoint that a call writes (may be NULL): its sizes and buffers.
qlora_status check_out8(const qlora_act8 *a, int64_t T, int64_t K) {
  if (!a) return QLORA_OK;
  if (a->T != T || a->K != K) return QLORA_ERR_SHAPE;
  if (!a->codes || !a->scale) return QLORA_ERR_NULL;
  return aligned16(a->codes) && aligned16(a->scale) ? QLORA_OK : QLORA_ERR_ALIGN;
}

qlora_status check_norm(int64_t T, int64_t D, int dtype, float eps) {
  if (!norm_shape_ok(T, D)) return QLORA_ERR_SHAPE;
  if (dtype != QLORA_F32 && dtype != QLORA_BF16) return QLORA_ERR_DTYPE;
  return std::isfinite(eps) && eps > 0.f ? QLORA_OK : QLORA_ERR_VALUE;
}

bool activation_ok(int act) { return act == QLORA_SILU || act == QLORA_GELU_TANH; }

// Whether a buffer is named for two results (or for one and the input that every workgroup reads).
bool named_twice(std::initializer_list<const void *> buffers) {
  for (const void *const *a = buffers.begin(); a != buffers.end(); ++a)
    for (const void *const *b = a + 1; b != buffers.end(); ++b)
      if (*a && *a == *b) return true;
  return false;
}

// n_in: byte offsets within a row tile of x stay below 2^32; n_ff, and its tiles with the tokens': a launch's grid.
constexpr int64_t kGatedMaxDim = (int64_t)1 << 22, kGatedMaxTiles = (int64_t)1 << 22;

bool gated_shape_ok(int64_t T, int64_t N, int64_t K, int r) {
  return linear_shape_ok(T, N, K, r) && N % kBlock == 0 && N < kGatedMaxDim && K < kGatedMaxDim &&
         product_ok(T, 2 * (int64_t)r) && (T / 256 + 1) * (N / 64) <= kGatedMaxTiles;
}

}  // namespace

extern "C" {

qlora_status qlora_rms_norm_fwd(const uint16_t *x, const uint16_t *residual, int64_t T, int64_t D, const void *weight,
                                qlora_dtype w_dtype, float eps, uint16_t *sum, uint16_t *y, const qlora_act8 *y8,
                                void *stream) {
  qlora_status s = check_norm(T, D, code_of(w_dtype), eps);
  if (s != QLORA_OK) return s;
  if (!x || !weight || (!y && !y8) || (residual == nullptr) != (sum == nullptr)) return QLORA_ERR_NULL;
  s = check_out8(y8, T, D);
  if (s != QLORA_OK) return s;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(sum) || !aligned16(y))
    return QLORA_ERR_ALIGN;
  if (named_twice({sum, y})) return QLORA_ERR_VALUE;
  const hipError_t e = launch_rms_norm_fwd(x, residual, T, D, weight, code_of(w_dtype) == QLORA_F32, eps, sum, y,
                                           y8 ? y8->codes : nullptr, y8 ? y8->scale : nullptr, (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

size_t qlora_rms_norm_bwd_workspace_bytes(int64_t T, int64_t D) {
  return norm_shape_ok(T, D) ? rms_norm_part_floats(T, D) * 4 : 0;
}

qlora_status qlora_rms_norm_bwd(const uint16_t *dy, const uint16_t *s, const uint16_t *dres, int64_t T, int64_t D,
                                const void *weight, qlora_dtype w_dtype, float eps, uint16_t *grad_s,
                                float *grad_weight, void *ws, size_t ws_bytes, void *stream) {
  const qlora_status st = check_norm(T, D, code_of(w_dtype), eps);
  if (st != QLORA_OK) return st;
  if (!dy || !s || !weight || !grad_s || (grad_weight && !ws)) return QLORA_ERR_NULL;
  if (!aligned16(dy) || !aligned16(s) || !aligned16(dres) || !aligned16(weight) || !aligned16(grad_s) ||
      !aligned16(grad_weight) || (grad_weight && !aligned16(ws)))
    return QLORA_ERR_ALIGN;
  if (grad_weight && ws_bytes < rms_norm_part_floats(T, D) * 4) return QLORA_ERR_WORKSPACE;
  const hipError_t e = launch_rms_norm_bwd(dy, s, dres, T, D, weight, code_of(w_dtype) == QLORA_F32, eps, grad_s,
                                           grad_weight, (float *)ws, (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

qlora_status qlora_gated_act_fwd(const uint16_t *gate, const uint16_t *up, int64_t T, int64_t N, qlora_activation act,
                                 uint16_t *h, const qlora_act8 *h8, void *stream) {
  if (!act_shape_ok(T, N)) return QLORA_ERR_SHAPE;
  if (!activation_ok(code_of(act))) return QLORA_ERR_VALUE;
  if (!gate || !up || (!h && !h8)) return QLORA_ERR_NULL;
  const qlora_status s = check_out8(h8, T, N);
  if (s != QLORA_OK) return s;
  if (!aligned16(gate) || !aligned16(up) || !aligned16(h)) return QLORA_ERR_ALIGN;
  const hipError_t e = launch_gated_act_fwd(gate, up, T, N, (Activation)code_of(act), h, h8 ? h8->codes : nullptr,
                                            h8 ? h8->scale : nullptr, (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

qlora_status qlora_gated_act_bwd(const uint16_t *dh, const uint16_t *gate, const uint16_t *up, int64_t T, int64_t N,
                                 qlora_activation act, uint16_t *dgate, uint16_t *dup, void *stream) {
  if (!act_shape_ok(T, N)) return QLORA_ERR_SHAPE;
  if (!activation_ok(code_of(act))) return QLORA_ERR_VALUE;
  if (!dh || !gate || !up || !dgate || !dup) return QLORA_ERR_NULL;
  if (!aligned16(dh) || !aligned16(gate) || !aligned16(up) || !aligned16(dgate) || !aligned16(dup))
    return QLORA_ERR_ALIGN;
  if (named_twice({dgate, dup})) return QLORA_ERR_VALUE;
  const hipError_t e =
      launch_gated_act_bwd(dh, gate, up, T, N, (Activation)code_of(act), dgate, dup, (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

size_t qlora_linear_gated_workspace_bytes(int64_t T, int64_t n_ff, int64_t n_in, int r) {
  return gated_shape_ok(T, n_ff, n_in, r) ? plan_linear_gated(T, n_ff, n_in, r).total : 0;
}

qlora_status qlora_linear_gated_fwd(const uint16_t *x, int64_t T, const qlora_nf4_weight *q, const uint16_t *A_set,
                                    const uint16_t *const *B, int r, float scale, qlora_activation act, uint16_t *h,
                                    const qlora_act8 *h8, uint16_t *gate, uint16_t *up, uint16_t *u_out, void *ws,
                                    size_t ws_bytes, void *stream) {
  int64_t N[kMaxSetMembers];
  qlora_status s = check_set(T, 2, q, r, scale, N);
  if (s != QLORA_OK) return s;
  if (N[0] != N[1] || !gated_shape_ok(T, N[0], q[0].n_in, r)) return QLORA_ERR_SHAPE;
  if (!activation_ok(code_of(act))) return QLORA_ERR_VALUE;
  if (!x || !A_set || !B || !B[0] || !B[1] || !ws || (!h && !h8) || (gate == nullptr) != (up == nullptr))
    return QLORA_ERR_NULL;
  s = check_out8(h8, T, N[0]);
  if (s != QLORA_OK) return s;
  if (!aligned16(x) || !aligned16(A_set) || !aligned16(B[0]) || !aligned16(B[1]) || !aligned16(h) || !aligned16(gate) ||
      !aligned16(up) || !aligned16(u_out) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  const GatedPlan p = plan_linear_gated(T, N[0], q[0].n_in, r);
  if (ws_bytes < p.total) return QLORA_ERR_WORKSPACE;
  if (named_twice({x, h, gate, up, u_out})) return QLORA_ERR_VALUE;
  const QWeight w[2] = {qweight(&q[0]), qweight(&q[1])};
  const GatedOut out{(Activation)code_of(act), h, h8 ? h8->codes : nullptr, h8 ? h8->scale : nullptr, gate, up};
  const hipError_t e = launch_linear_gated_fwd(p, x, w, A_set, B, scale, out, u_out, (char *)ws, nf4_levels(),
                                               (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

}  // extern "C"
