/* Calls the entry points of the feed-forward block (the root-mean-square norm, the gated product) with arguments that
 * must be refused, and their size helpers with extreme shapes.  Nothing here reaches the GPU: every call fails before
 * anything is enqueued.  Built with the address and undefined-behaviour sanitizers. */
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "qlora.h"

static int failures;
#define EXPECT(call, want)                                                     \
  do {                                                                         \
    const int got = (int)(call);                                               \
    if (got != (int)(want)) {                                                  \
      printf("line %d: %s = %d, want %d\n", __LINE__, #call, got, (int)(want)); \
      ++failures;                                                              \
    }                                                                          \
  } while (0)

int main(void) {
  _Alignas(16) static unsigned char mem[512];
  uint16_t *h = (uint16_t *)mem;
  float *f = (float *)mem;
  const uint16_t *B[2] = {h, h};
  /* an enumeration's object may hold any value */
  qlora_dtype odd_dtype;
  qlora_activation odd_act;
  const int any = 77;
  memcpy(&odd_dtype, &any, sizeof odd_dtype);
  memcpy(&odd_act, &any, sizeof odd_act);
  const int64_t big[] = {INT64_MAX, INT64_MIN, -1, 0, (int64_t)1 << 62, (int64_t)1 << 38};
  for (int i = 0; i < 6; ++i) {
    const int64_t b = big[i];
    EXPECT(qlora_rms_norm_fwd(h, 0, b, 64, f, QLORA_F32, 1e-6f, 0, h, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_rms_norm_fwd(h, 0, 4, b, f, QLORA_F32, 1e-6f, 0, h, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_rms_norm_bwd(h, h, 0, b, 64, f, QLORA_F32, 1e-6f, h, 0, 0, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_rms_norm_bwd(h, h, 0, 4, b, f, QLORA_F32, 1e-6f, h, 0, 0, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_gated_act_fwd(h, h, b, 64, QLORA_SILU, h, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_gated_act_fwd(h, h, 4, b, QLORA_SILU, h, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_gated_act_bwd(h, h, h, b, 64, QLORA_SILU, h, h, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_gated_act_bwd(h, h, h, 4, b, QLORA_SILU, h, h, 0), QLORA_ERR_SHAPE);
    const qlora_nf4_weight rows[2] = {{b, 256, mem, mem, f, f, 0}, {b, 256, mem, mem, f, f, 0}};
    const qlora_nf4_weight cols[2] = {{128, b, mem, mem, f, f, 0}, {128, b, mem, mem, f, f, 0}};
    const qlora_nf4_weight fine[2] = {{128, 256, mem, mem, f, f, 0}, {128, 256, mem, mem, f, f, 0}};
    EXPECT(qlora_linear_gated_fwd(h, 4, rows, h, B, 8, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_linear_gated_fwd(h, 4, cols, h, B, 8, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_linear_gated_fwd(h, b, fine, h, B, 8, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_linear_gated_fwd(h, 4, fine, h, B, (int)b, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_SHAPE);
    if (qlora_rms_norm_bwd_workspace_bytes(b, 64) || qlora_rms_norm_bwd_workspace_bytes(4, b) ||
        qlora_linear_gated_workspace_bytes(b, 128, 256, 8) || qlora_linear_gated_workspace_bytes(4, b, 256, 8) ||
        qlora_linear_gated_workspace_bytes(4, 128, b, 8) || qlora_linear_gated_workspace_bytes(4, 128, 256, (int)b)) {
      printf("a bad shape has a workspace\n");
      ++failures;
    }
  }
  /* the largest shapes that are accepted: the plans must not overflow */
  if (!qlora_rms_norm_bwd_workspace_bytes((int64_t)1 << 31, 64) || !qlora_rms_norm_bwd_workspace_bytes(1 << 21, 65536) ||
      !qlora_linear_gated_workspace_bytes(1 << 29, 64, 64, 128) || !qlora_linear_gated_workspace_bytes(255, (1 << 22) - 64, 64, 256) ||
      !qlora_linear_gated_workspace_bytes(1, 64, (1 << 22) - 64, 1) || !qlora_linear_gated_workspace_bytes(64, 1 << 20, 65536, 1) ||
      !qlora_linear_gated_workspace_bytes(1 << 20, 1 << 13, 1 << 13, 250) ||
      !qlora_linear_gated_workspace_bytes(1 << 14, 22016, 8192, 64)) {
    printf("a large shape has no workspace\n");
    ++failures;
  }
  if (qlora_linear_gated_workspace_bytes(1 << 30, 64, 64, 8)) {
    printf("more tiles than a launch holds have a workspace\n");
    ++failures;
  }
  const qlora_nf4_weight q[2] = {{128, 256, mem, mem, f, f, 0}, {128, 256, mem, mem, f, f, 0}};
  const qlora_act8 a = {4, 128, (int8_t *)mem, f}, none = {4, 128, 0, f};
  EXPECT(qlora_rms_norm_fwd(h, 0, 4, 128, f, odd_dtype, 1e-6f, 0, h, 0, 0), QLORA_ERR_DTYPE);
  EXPECT(qlora_rms_norm_fwd(h, 0, 4, 128, f, QLORA_F32, NAN, 0, h, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_rms_norm_fwd(h, h, 4, 128, f, QLORA_F32, 1e-6f, 0, h, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_rms_norm_fwd(h, 0, 4, 128, f, QLORA_F32, 1e-6f, 0, 0, &none, 0), QLORA_ERR_NULL);
  EXPECT(qlora_rms_norm_bwd(h, h, 0, 4, 128, f, QLORA_BF16, 0.f, h, 0, 0, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_rms_norm_bwd(h, h, 0, 4, 128, f, QLORA_BF16, 1e-6f, h, f, mem, 0, 0), QLORA_ERR_WORKSPACE);
  EXPECT(qlora_gated_act_fwd(h, h, 4, 128, odd_act, h, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_gated_act_fwd(h, h, 5, 128, QLORA_SILU, h, &a, 0), QLORA_ERR_SHAPE);
  EXPECT(qlora_gated_act_bwd(h, h, h, 4, 128, odd_act, h, h, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_gated_act_bwd(h, h, h, 4, 128, QLORA_GELU_TANH, h, h + 1, 0), QLORA_ERR_ALIGN);
  EXPECT(qlora_linear_gated_fwd(h, 4, 0, h, B, 8, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, 0, 8, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, INFINITY, QLORA_SILU, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, 1.f, odd_act, h, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, 1.f, QLORA_SILU, 0, 0, 0, 0, 0, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, 1.f, QLORA_SILU, h + 8, &a, h + 16, h + 24, h + 32, mem, 0, 0), QLORA_ERR_WORKSPACE);
  /* a buffer named for two results */
  EXPECT(qlora_rms_norm_fwd(h, h, 4, 8 * 16, f, QLORA_F32, 1e-6f, h + 8, h + 8, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_gated_act_bwd(h, h, h, 4, 128, QLORA_SILU, h, h, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, 1.f, QLORA_SILU, h + 8, 0, h + 8, h + 16, 0, mem, 1 << 24, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, 1.f, QLORA_SILU, h + 8, 0, h + 16, h + 16, 0, mem, 1 << 24, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_linear_gated_fwd(h, 4, q, h, B, 8, 1.f, QLORA_SILU, h, 0, 0, 0, 0, mem, 1 << 24, 0), QLORA_ERR_VALUE);
  if (failures) {
    printf("%d failures\n", failures);
    return 1;
  }
  printf("all refusals as documented\n");
  return 0;
}
