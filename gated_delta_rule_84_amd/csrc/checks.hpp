// checks.hpp -- host checks of pointers, strides and overlaps that the entry points of mixer_api.hip and
// delta_api.hip share.  Not installed.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdr {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Byte ranges [a, a + na) and [b, b + nb) intersect (both non-empty).
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Extent in bytes of `rows` rows of `width` elements, `ld` elements apart.
size_t extent(long long rows, long long width, int64_t ld, size_t es) {
    return rows > 0 ? (size_t)((rows - 1) * ld + width) * es : 0;
}

// `ld` elements between tokens (0: dense) fits rows of `width` elements, and the last row's end is addressable.
bool stride_ok(int64_t &ld, long long rows, long long width) {
    if (ld == 0) ld = width;
    if (ld < width) return false;
    return rows <= 1 || ld <= (int64_t)(1ll << 56) / rows;
}

struct Span {
    const void *p;
    size_t n;
};

// No output overlaps an input or another output.
bool apart(const Span *outs, int no, const Span *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return false;
        for (int j = i + 1; j < no; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return false;
    }
    return true;
}

}  // namespace
}  // namespace gdr
