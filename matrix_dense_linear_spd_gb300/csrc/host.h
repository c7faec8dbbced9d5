// Host-side helpers shared by the C entry points.
#pragma once

#include <cstdint>

#include "../../include/bl.h"

namespace bl {

// Record a printf-style message for bl_last_error and return `st`.
bl_status fail(bl_status st, const char *fmt, ...);
// Forget the previous call's message (every entry point starts with it).
void clear_error();
// SMs of the current device (cached per device); 0 if it cannot be queried.
int sm_count();

// Bytes [lo, hi) of memory that a call reads or writes.
struct Range {
    uintptr_t lo, hi;
};
inline Range range_of(const void *p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + static_cast<uintptr_t>(bytes)};
}
inline bool meet(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace bl
