/* plan_check.cpp -- the host-side parts in csrc/plan.h, called on the CPU: choices
 * for GPUs of any size, and what is told of products that gave up.  Exit status 0
 * and "ok" when all of it holds. */
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

/* A failure is told once to every (thread, device, stream) that asks, whoever
 * asked before. */
static void tellings() {
  const char streams[64] = {};
  Told a, b; /* two threads */
  HOLD(!a.news(0, 0, 0) && !b.news(0, 0, 0) && !a.news(0, streams, 0));
  /* the counter goes to 3: both threads and both streams hear of it, once */
  HOLD(a.news(0, 0, 3) && !a.news(0, 0, 3));
  HOLD(a.news(0, streams, 3) && !a.news(0, streams, 3));
  HOLD(b.news(0, 0, 3) && !b.news(0, 0, 3));
  /* a stream first asked about after it; another device's own counter */
  HOLD(a.news(0, streams + 1, 3) && !a.news(1, 0, 0) && a.news(1, 0, 1) && !a.news(0, 0, 3));
  /* once more */
  HOLD(a.news(0, 0, 4) && a.news(0, streams, 4) && b.news(0, 0, 4) && !a.news(0, 0, 4));
  /* more streams than are remembered: told again at worst, never not told */
  Told c;
  for (int i = 0; i < 64; ++i) HOLD(c.news(0, streams + i, 5));
  for (int i = 32; i < 64; ++i) HOLD(!c.news(0, streams + i, 5));
  for (int i = 0; i < 64; ++i) HOLD(c.news(0, streams + i, 6 + i));
  HOLD(c.news(0, streams, 70));
  /* the one asked about longest ago is forgotten */
  Told d;
  for (int i = 0; i < 32; ++i) d.news(0, streams + i, 5);
  HOLD(!d.news(0, streams, 5) && d.news(0, streams + 40, 5));
  HOLD(!d.news(0, streams, 5) && d.news(0, streams + 1, 5));
}

int main() {
  splits();
  tellings();
  if (failures == 0) printf("ok\n");
  return failures != 0;
}
