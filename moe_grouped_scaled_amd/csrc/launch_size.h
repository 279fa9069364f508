// Host arithmetic on how many workgroups a launch has.  No HIP types: it is tested on the CPU by itself.
#pragma once

#include <stdint.h>

namespace mgs {

// Workgroups of `threads` threads that one launch takes: its threads are counted in 32 bits.
inline int64_t most_workgroups(int threads) { return (int64_t)UINT32_MAX / threads; }

// Workgroups that share the passes over a group's rows, where the group with the most rows has `want` passes and one pass
// over all groups has `base` workgroups (at most most_workgroups()): up to 16, and no more than a launch takes.  With fewer than
// `want` each takes several passes in turn.
inline int64_t shared_passes(int64_t want, int64_t base, int threads) {
  const int64_t most = most_workgroups(threads) / base, p = want < 16 ? want : 16;
  return most < p ? most : p;
}

}  // namespace mgs
