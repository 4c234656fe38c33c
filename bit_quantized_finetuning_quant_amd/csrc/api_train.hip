// C ABI of the operators around the linear layer in a training step (declared
// in include/qlora.h): 8-bit activation checkpoints with the backward pass that
// reads them, and the loss of the head.  Host code only.

#include "validate.hpp"

using namespace qlora;

namespace {

qlora_status check_act8(const qlora_act8 *a) {
  if (!a) return QLORA_ERR_NULL;
  if (!product_ok(a->T, a->K) || a->K % kBlock != 0) return QLORA_ERR_SHAPE;
  if (!a->codes || !a->scale) return QLORA_ERR_NULL;
  return aligned16(a->codes) && aligned16(a->scale) ? QLORA_OK : QLORA_ERR_ALIGN;
}

// The shapes the head's loss accepts.
bool head_shape_ok(int64_t T, int64_t V, int64_t D) {
  return D >= kBlock && D % kBlock == 0 && D <= kHeadMaxDim && product_ok(T, D) && product_ok(V, D);
}

// The loss of a bf16 head (w) or a packed one (q), the other one nullptr and both already checked.
qlora_status head_loss(const uint16_t *h, int64_t T, const uint16_t *w, const QWeight *q, int64_t V, int64_t D,
                       const int64_t *target, const float *weight, float scale, float *loss, float *lse,
                       uint16_t *grad_h, void *ws, size_t ws_bytes, void *stream) {
  if (!head_shape_ok(T, V, D)) return QLORA_ERR_SHAPE;
  if (!std::isfinite(scale)) return QLORA_ERR_VALUE;
  if (!h || !target || !loss || !ws) return QLORA_ERR_NULL;
  if (!aligned16(h) || !aligned16(target) || !aligned16(loss) || !aligned16(ws) || (weight && !aligned16(weight)) ||
      (lse && !aligned16(lse)) || (grad_h && !aligned16(grad_h)))
    return QLORA_ERR_ALIGN;
  const HeadPlan p = plan_head(T, V, D, grad_h != nullptr, q != nullptr);
  if (ws_bytes < p.total) return QLORA_ERR_WORKSPACE;
  hipError_t e = launch_head_loss(p, h, w, q, target, weight, scale, loss, lse, grad_h, (char *)ws, nf4_levels(),
                                  (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

}  // namespace

extern "C" {

qlora_status qlora_act8_write(const uint16_t *x, const qlora_act8 *a, void *stream) {
  const qlora_status s = check_act8(a);
  if (s != QLORA_OK) return s;
  if (!x) return QLORA_ERR_NULL;
  if (!aligned16(x)) return QLORA_ERR_ALIGN;
  hipError_t e = launch_act8_encode(x, a->T, a->K, a->codes, a->scale, (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

qlora_status qlora_act8_read(const qlora_act8 *a, uint16_t *x, void *stream) {
  const qlora_status s = check_act8(a);
  if (s != QLORA_OK) return s;
  if (!x) return QLORA_ERR_NULL;
  if (!aligned16(x)) return QLORA_ERR_ALIGN;
  hipError_t e = launch_act8_decode(a->codes, a->scale, a->T, a->K, x, (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

size_t qlora_linear_set_act8_workspace_bytes(int64_t T, int count, const int64_t *n_out, int64_t n_in, int r) {
  if (!n_out || count < 1 || count > kMaxSetMembers || r < 1 || r > 256) return 0;
  for (int i = 0; i < count; ++i)
    if (!linear_shape_ok(T, n_out[i], n_in, r)) return 0;
  if (!product_ok(T, (int64_t)count * r)) return 0;
  return plan_linear_set_act8(T, count, n_out, n_in, r, false).total;
}

size_t qlora_linear_set_act8_workspace_bound(int64_t T, int count, int r) {
  if (count < 1 || count > kMaxSetMembers || r < 1 || r > 256 || !product_ok(T, (int64_t)count * r)) return 0;
  return act8_bound(T, count, r);
}

qlora_status qlora_linear_set_bwd_act8(const uint16_t *const *dy, const qlora_act8 *a, int count,
                                       const qlora_nf4_weight *q, const uint16_t *A_set, const uint16_t *const *B,
                                       int r, float scale, const uint16_t *u, uint16_t *grad_x, float *grad_A_set,
                                       float *const *grad_B, void *ws, size_t ws_bytes, void *stream) {
  int64_t N[kMaxSetMembers];
  qlora_status s = check_act8(a);
  if (s != QLORA_OK) return s;
  s = check_set(a->T, count, q, r, scale, N);
  if (s != QLORA_OK) return s;
  if (q[0].n_in != a->K) return QLORA_ERR_SHAPE;
  if (!dy || !A_set || !B || !u || !grad_A_set || !grad_B || !ws) return QLORA_ERR_NULL;
  if (!aligned16(A_set) || !aligned16(u) || !aligned16(grad_A_set) || !aligned16(ws) ||
      (grad_x && !aligned16(grad_x)))
    return QLORA_ERR_ALIGN;
  QWeight w[kMaxSetMembers];
  for (int i = 0; i < count; ++i) {
    if (!dy[i] || !B[i] || !grad_B[i]) return QLORA_ERR_NULL;
    if (!aligned16(dy[i]) || !aligned16(B[i]) || !aligned16(grad_B[i])) return QLORA_ERR_ALIGN;
    w[i] = qweight(&q[i]);
  }
  Act8BwdPlan p = plan_linear_set_act8(a->T, count, N, a->K, r, false);
  if (ws_bytes < p.total) {
    if (ws_bytes < act8_bound(a->T, count, r)) return QLORA_ERR_WORKSPACE;
    p = plan_linear_set_act8(a->T, count, N, a->K, r, true);
  }
  hipError_t e = launch_linear_set_bwd_act8(p, dy, a->codes, a->scale, w, A_set, B, scale, u, grad_x, grad_A_set,
                                            grad_B, (char *)ws, nf4_levels(), (hipStream_t)stream);
  return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP;
}

qlora_status qlora_linear_bwd_act8(const uint16_t *dy, const qlora_act8 *a, const qlora_nf4_weight *q,
                                   const uint16_t *A, const uint16_t *B, int r, float scale, const uint16_t *u,
                                   uint16_t *grad_x, float *grad_A, float *grad_B, void *ws, size_t ws_bytes,
                                   void *stream) {
  return qlora_linear_set_bwd_act8(&dy, a, 1, q, A, &B, r, scale, u, grad_x, grad_A, &grad_B, ws, ws_bytes, stream);
}

size_t qlora_head_loss_workspace_bytes(int64_t T, int64_t V, int64_t D, int grad, int packed) {
  if (!head_shape_ok(T, V, D)) return 0;
  return plan_head(T, V, D, grad != 0, packed != 0).total;
}

qlora_status qlora_head_loss(const uint16_t *h, int64_t T, const uint16_t *w, int64_t V, int64_t D,
                             const int64_t *target, const float *weight, float scale, float *loss, float *lse,
                             uint16_t *grad_h, void *ws, size_t ws_bytes, void *stream) {
  if (!w) return QLORA_ERR_NULL;
  if (!aligned16(w)) return QLORA_ERR_ALIGN;
  return head_loss(h, T, w, nullptr, V, D, target, weight, scale, loss, lse, grad_h, ws, ws_bytes, stream);
}

qlora_status qlora_head_loss_nf4(const uint16_t *h, int64_t T, const qlora_nf4_weight *q, const int64_t *target,
                                 const float *weight, float scale, float *loss, float *lse, uint16_t *grad_h,
                                 void *ws, size_t ws_bytes, void *stream) {
  const qlora_status s = check_weight(q);
  if (s != QLORA_OK) return s;
  const QWeight qw = qweight(q);
  return head_loss(h, T, nullptr, &qw, q->n_out, q->n_in, target, weight, scale, loss, lse, grad_h, ws, ws_bytes,
                   stream);
}

}  // extern "C"
