// What the C-ABI files share: the per-thread error message and the checks of
// raw buffers.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

extern thread_local char g_last_error[512];

// Formats the calling thread's message and returns `st`.
gdn_status fail(gdn_status st, const char *fmt, ...);

struct Span {
  const void *p;
  unsigned long long bytes;
  const char *name;
};

inline bool overlap(const Span &a, const Span &b) {
  const auto a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace gdn
