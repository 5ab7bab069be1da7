// mrr_checks.h -- what the host checks of the operators share (no HIP header).
// Pointers are compared and tested for alignment, never dereferenced.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_rerouting_v2.h"

namespace mrr {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int wide_bytes(int32_t dt) { return dt == MRR_F32 ? 4 : dt == MRR_F16 || dt == MRR_BF16 ? 2 : 0; }

// Buffers of one call: no output may overlap any other.
struct Buffers {
  struct {
    uintptr_t lo, hi;
    bool out;
  } b[16];
  int n = 0;
  void add(const void* p, int64_t bytes, bool out) {
    if (p == nullptr || bytes <= 0) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    b[n++] = {lo, lo + static_cast<uintptr_t>(bytes), out};
  }
  bool clash() const {
    for (int x = 0; x < n; ++x)
      for (int y = x + 1; y < n; ++y)
        if ((b[x].out || b[y].out) && b[x].lo < b[y].hi && b[y].lo < b[x].hi) return true;
    return false;
  }
};

// All sizes below are bounded so that no byte count passes 2^62.
inline bool fits(int64_t a, int64_t b, int64_t c) {
  const int64_t most = int64_t(1) << 62;
  if (a == 0 || b == 0 || c == 0) return true;
  if (a > most / b) return false;
  return a * b <= most / c;
}

}  // namespace mrr
