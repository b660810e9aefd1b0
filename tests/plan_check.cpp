/* plan_check.cpp -- the host-side choices of csrc/plan.h, called on the CPU for
 * GPUs of any size.  Exit status 0 and "ok" when all of them hold. */
#include <stdio.h>

#include "plan.h"

static long failures;

#define HOLD(what)                                          \
  do {                                                      \
    if (!(what) && ++failures < 10) printf("%s\n", #what);  \
  } while (0)

/* Every tile of a split product is the only one of its cluster, whatever the
 * GPU has (the grid is sms / split clusters). */
static void splits() {
  for (uint32_t sms = 1; sms <= 160; ++sms)
    for (uint64_t tiles = 1; tiles <= 200; ++tiles)
      for (uint32_t ksteps = 1; ksteps <= 20; ++ksteps) {
        const uint32_t s = matmul_split(tiles, ksteps, sms, 4);
        HOLD(s == 1 || s == 2 || s == 4);
        HOLD(s == 1 || tiles <= sms / s);
        HOLD(s == 1 || s <= ksteps);  /* no CTA without a stage */
      }
  HOLD(matmul_split(32, 16, 148, 4) == 4);  /* 1 x 4096 x 4096 on a whole B200 */
  HOLD(matmul_split(32, 16, 127, 4) == 2);
  HOLD(matmul_split(32, 16, 70, 4) == 2);
  HOLD(matmul_split(32, 16, 63, 4) == 1);
  HOLD(matmul_split(1, 3, 148, 4) == 2);
  HOLD(matmul_split(1ull << 40, 16, 148, 4) == 1);
}

int main() {
  splits();
  if (failures == 0) printf("ok\n");
  return failures != 0;
}
