// Argument checks shared by the files that implement the C ABI: byte ranges of buffers,
// element types and alignment.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/retention.h"

namespace {

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

Range span(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}

bool overlaps(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

size_t elem_bytes(retn_dtype dt) { return dt == RETN_BF16 ? 2 : 4; }

bool valid_dtype(retn_dtype dt) { return dt == RETN_F32 || dt == RETN_BF16; }

// The matrix-core kernels move 16-byte units of q, k, v and store 8-byte units of o.
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
