// Host-side argument checks shared by the files that implement the C ABI.
#pragma once

#include <cmath>

#include "../../include/qlora.h"
#include "common.hpp"
#include "launch.hpp"

namespace qlora {

constexpr int64_t kMaxNumel = (int64_t)1 << 37;

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// a * b <= kMaxNumel for positive a, b, without forming a product that could overflow
inline bool product_ok(int64_t a, int64_t b) { return a > 0 && b > 0 && a <= kMaxNumel / b; }

inline bool shape_ok(int64_t n_out, int64_t n_in) { return product_ok(n_out, n_in); }

inline bool double_quantized(const qlora_nf4_weight *q) { return (q->flags & QLORA_NF4_FP32_CONSTANTS) == 0u; }

inline qlora_status check_weight(const qlora_nf4_weight *q) {
  if (!q) return QLORA_ERR_NULL;
  if (!shape_ok(q->n_out, q->n_in)) return QLORA_ERR_SHAPE;
  if ((q->flags & ~QLORA_NF4_FP32_CONSTANTS) != 0u) return QLORA_ERR_VALUE;
  if (!q->codes || !q->absmax_scale) return QLORA_ERR_NULL;
  if (!aligned16(q->codes) || !aligned16(q->absmax_scale)) return QLORA_ERR_ALIGN;
  if (double_quantized(q)) {
    if (!q->absmax_fp8 || !q->absmax_mean) return QLORA_ERR_NULL;
    if (!aligned16(q->absmax_fp8) || !aligned16(q->absmax_mean)) return QLORA_ERR_ALIGN;
  }
  return QLORA_OK;
}

inline QWeight qweight(const qlora_nf4_weight *q) {
  return QWeight{q->codes, q->absmax_fp8, q->absmax_scale, q->absmax_mean, q->n_out, q->n_in, double_quantized(q)};
}

inline qlora_status check_linear(int64_t T, const qlora_nf4_weight *q, int r, float scale) {
  qlora_status s = check_weight(q);
  if (s != QLORA_OK) return s;
  if (T < 1 || T > kMaxNumel || q->n_in % kBlock != 0 || r < 1 || r > 256) return QLORA_ERR_SHAPE;
  if (!product_ok(T, q->n_in) || !product_ok(T, q->n_out)) return QLORA_ERR_SHAPE;
  if (!std::isfinite(scale)) return QLORA_ERR_VALUE;
  return QLORA_OK;
}

// A projection set: 1..kMaxSetMembers members sharing n_in and the storage
// form, adapter rank r per member.
inline qlora_status check_set(int64_t T, int count, const qlora_nf4_weight *q, int r, float scale, int64_t *N) {
  if (!q) return QLORA_ERR_NULL;
  if (count < 1 || count > kMaxSetMembers) return QLORA_ERR_SHAPE;
  for (int i = 0; i < count; ++i) {
    const qlora_status s = check_linear(T, &q[i], r, scale);
    if (s != QLORA_OK) return s;
    if (q[i].n_in != q[0].n_in) return QLORA_ERR_SHAPE;
    if (q[i].flags != q[0].flags) return QLORA_ERR_VALUE;
    N[i] = q[i].n_out;
  }
  if (!product_ok(T, (int64_t)count * r)) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

// the shapes every linear call accepts (check_linear), for the size helpers
inline bool linear_shape_ok(int64_t T, int64_t n_out, int64_t n_in, int r) {
  return shape_ok(n_out, n_in) && n_in % kBlock == 0 && r >= 1 && r <= 256 && product_ok(T, n_in) &&
         product_ok(T, n_out);
}

}  // namespace qlora
