/* Calls the entry points of the training operators (8-bit checkpoints, the backward pass that reads
 * them, the loss of the head) with arguments that must be refused, and their size helpers with extreme
 * shapes.  Nothing here reaches the GPU: every call fails before anything is enqueued.  Built with the
 * address and undefined-behaviour sanitizers. */
#include <math.h>
#include <stdio.h>

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
  _Alignas(16) static unsigned char mem[256];
  uint16_t *h = (uint16_t *)mem;
  float *f = (float *)mem;
  int64_t *y = (int64_t *)mem;
  const int64_t big[] = {INT64_MAX, INT64_MIN, -1, 0, (int64_t)1 << 62, (int64_t)1 << 38};
  for (int i = 0; i < 6; ++i) {
    const int64_t b = big[i];
    const qlora_act8 a = {b, 64, (int8_t *)mem, f}, c = {64, b, (int8_t *)mem, f};
    EXPECT(qlora_act8_write(h, &a, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_act8_read(&c, h, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss(h, b, h, 100, 64, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss(h, 4, h, b, 64, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss(h, 4, h, 100, b, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_SHAPE);
    if (qlora_head_loss_workspace_bytes(b, 100, 64, 1, 1) || qlora_head_loss_workspace_bytes(4, b, 64, 0, 1) ||
        qlora_head_loss_workspace_bytes(4, 100, b, 1, 0) ||
        qlora_linear_set_act8_workspace_bytes(b, 1, big + 2, 64, 8) ||
        qlora_linear_set_act8_workspace_bytes(4, 1, big + i, 64, 8) ||
        qlora_linear_set_act8_workspace_bytes(4, (int)b, big, 64, 8)) {
      printf("a bad shape has a workspace\n");
      ++failures;
    }
  }
  /* the largest shapes that are accepted: the plans must not overflow */
  const int64_t n37 = (int64_t)1 << 31;
  if (!qlora_head_loss_workspace_bytes(n37, 100, 64, 1, 1) || !qlora_head_loss_workspace_bytes(64, n37, 64, 1, 1) ||
      !qlora_head_loss_workspace_bytes(1000, n37, 64, 0, 0) || !qlora_head_loss_workspace_bytes(100000, n37, 64, 1, 1) ||
      !qlora_head_loss_workspace_bytes(1 << 21, 1 << 21, 65536, 1, 1) ||
      !qlora_linear_set_act8_workspace_bytes(1 << 20, 1, (const int64_t[]){1 << 17}, 1 << 17, 256) ||
      !qlora_linear_set_act8_workspace_bytes(1 << 26, 4, (const int64_t[]){7, 9, 11, 2047}, 64, 256)) {
    printf("a large shape has no workspace\n");
    ++failures;
  }
  const qlora_act8 a = {16, 256, (int8_t *)mem, f}, null = {16, 256, 0, f}, off = {16, 256, (int8_t *)mem + 8, f};
  EXPECT(qlora_act8_write(0, &a, 0), QLORA_ERR_NULL);
  EXPECT(qlora_act8_write(h, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_act8_write(h, &null, 0), QLORA_ERR_NULL);
  EXPECT(qlora_act8_read(&off, h, 0), QLORA_ERR_ALIGN);
  qlora_nf4_weight w = {512, 256, mem, mem, f, f, 0};
  EXPECT(qlora_linear_bwd_act8(h, &a, 0, h, h, 8, 1.f, h, h, f, f, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_bwd_act8(h, &a, &w, h, h, 8, 1.f, h, h, f, f, mem, 0, 0), QLORA_ERR_WORKSPACE);
  EXPECT(qlora_linear_bwd_act8(h, &a, &w, h, h, 8, NAN, h, h, f, f, mem, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_linear_bwd_act8(0, &a, &w, h, h, 8, 1.f, h, h, f, f, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_bwd_act8(h, &a, &w, h, h, 8, 1.f, 0, h, f, f, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_bwd_act8(h, &a, &w, h, h, 257, 1.f, h, h, f, f, mem, 0, 0), QLORA_ERR_SHAPE);
  w.flags = 4;
  EXPECT(qlora_linear_bwd_act8(h, &a, &w, h, h, 8, 1.f, h, h, f, f, mem, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_head_loss_nf4(h, 4, &w, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_VALUE);
  w.flags = 0;
  EXPECT(qlora_linear_set_bwd_act8(0, &a, 1, &w, h, 0, 8, 1.f, h, h, f, 0, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_linear_set_bwd_act8(0, &a, 5, &w, h, 0, 8, 1.f, h, h, f, 0, mem, 0, 0), QLORA_ERR_SHAPE);
  EXPECT(qlora_linear_set_bwd_act8(0, &a, -1, &w, h, 0, 8, 1.f, h, h, f, 0, mem, 0, 0), QLORA_ERR_SHAPE);
  EXPECT(qlora_head_loss_nf4(h, 4, &w, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_WORKSPACE);
  EXPECT(qlora_head_loss_nf4(h, 4, 0, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_NULL);
  EXPECT(qlora_head_loss(h, 4, h, 100, 64, y, 0, INFINITY, f, f, h, mem, 0, 0), QLORA_ERR_VALUE);
  EXPECT(qlora_head_loss(h, 4, h, 100, 64, y, f + 1, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_ALIGN);
  EXPECT(qlora_head_loss(h, 4, 0, 100, 64, y, 0, 1.f, f, f, h, mem, 0, 0), QLORA_ERR_NULL);
  if (failures) return 1;
  printf("all refusals as documented\n");
  return 0;
}
