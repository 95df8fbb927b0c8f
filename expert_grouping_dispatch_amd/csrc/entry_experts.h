// Checks that the entry points of the experts' products share: sizes, and
// buffers that lie on one another.
#pragma once

#include <initializer_list>

#include "entry.h"

namespace moe {

constexpr int64_t kMaxRows = 0xFFFFFFFEll;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int32_t kMaxFewWidth = 1 << 17;  // 4 bytes each of MOE_FEW_MAX_SLOTS rows stay below 2^31

inline bool width_ok(int32_t n) { return n > 0 && n <= kMaxWidth && n % 16 == 0; }

struct Span {
  const void* at;
  uint64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
  return a.at != nullptr && b.at != nullptr && a.bytes > 0 && b.bytes > 0 && p < q + b.bytes && q < p + a.bytes;
}

// Whether something written lies on something read or on something else written.
inline bool clash(std::initializer_list<Span> reads, std::initializer_list<Span> writes) {
  for (const Span* w = writes.begin(); w != writes.end(); ++w) {
    for (const Span& r : reads)
      if (overlap(r, *w)) return true;
    for (const Span* v = writes.begin(); v != w; ++v)
      if (overlap(*v, *w)) return true;
  }
  return false;
}

}  // namespace moe
