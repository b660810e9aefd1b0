// plan.h -- choices of the host side that depend on the GPU only through numbers
// given to them (plain C++, no CUDA: tests/plan_check.cpp calls them on the CPU).
#pragma once

#include <stdint.h>

// CTAs of a cluster that share one tile's k: 1, 2 or 4 (`most`).  A CTA of a
// split leaves its part of the sums in the stage ring and adds up once, behind
// its walk, so no cluster may meet a second tile: tiles x split CTAs are at most
// the SMs, of which a grid has one CTA each (and at most 128, up to which splits
// were measured).
inline uint32_t matmul_split(uint64_t tiles, uint32_t ksteps, uint32_t sms, uint32_t most) {
  const uint32_t ctas = sms < 128u ? sms : 128u;
  uint32_t split = 1;
  while (split < most && tiles * (split * 2u) <= ctas && ksteps >= split * 2u) split *= 2u;
  return split;
}
