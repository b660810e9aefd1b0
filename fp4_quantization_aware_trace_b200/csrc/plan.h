// plan.h -- parts of the host side that see the GPU only through numbers given to
// them (plain C++, no CUDA: tests/plan_check.cpp calls them on the CPU).
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

// What one host thread has been told of a counter per device that only grows
// (products that gave up), apart for each stream it asks about: no other thread's
// question and none about another stream hides what one has not heard yet.  Of
// more than kAsked (device, stream) pairs the one asked about longest ago is
// forgotten and would be told everything again.
struct Told {
  static constexpr int kAsked = 32;
  struct {
    int dev;
    const void* stream;
    uint32_t count;
    uint64_t when;  // 0: free
  } asked[kAsked] = {};
  uint64_t now = 0;

  // Whether `count` has grown since this was last asked (at first: since 0).
  bool news(int dev, const void* stream, uint32_t count) {
    int at = 0;
    for (int i = 0; i < kAsked; ++i) {
      if (asked[i].when && asked[i].dev == dev && asked[i].stream == stream) {
        at = i;
        break;
      }
      if (asked[i].when < asked[at].when) at = i;
    }
    auto& a = asked[at];
    if (!(a.when && a.dev == dev && a.stream == stream)) a = {dev, stream, 0u, 0u};
    a.when = ++now;
    const bool grown = a.count != count;
    a.count = count;
    return grown;
  }
};
