// Host checks that several sources share: memory ranges of a call's tensors, and alignment.
#pragma once

#include <initializer_list>

#include "mgs_internal.h"

namespace mgs {

// A named range of memory; NULL and empty tensors take none.
struct Range {
  const char* name;
  const void* p;
  int64_t bytes;
};

inline bool ranges_meet(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes;
}

// No output may be or overlap another tensor of the call: workgroups read and write in any order.
inline int check_ranges(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range* q = o + 1; q != outs.end(); ++q)
      if (ranges_meet(*o, *q)) return fail(MGS_ERR_INVALID_ARG, "%s must not be or overlap %s", o->name, q->name);
    for (const Range& i : ins)
      if (ranges_meet(*o, i)) return fail(MGS_ERR_INVALID_ARG, "%s must not be or overlap %s", o->name, i.name);
  }
  return MGS_OK;
}

inline int check_aligned(std::initializer_list<Range> ts, int bytes) {
  for (const Range& t : ts)
    if (reinterpret_cast<uintptr_t>(t.p) % bytes)
      return fail(MGS_ERR_INVALID_ARG, "%s must be %d-byte aligned", t.name, bytes);
  return MGS_OK;
}

}  // namespace mgs
