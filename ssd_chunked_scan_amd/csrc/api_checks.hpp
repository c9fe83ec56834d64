// api_checks.hpp -- argument checks that the newer operators' host sides share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "ssd.h"

namespace ssd {

struct Range {
    const void *p;
    size_t n;
};
inline bool overlaps(Range a, Range b)
{
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}
// Whether no output overlaps an input or another output.
template <size_t NI, size_t NO> bool apart(const Range (&ins)[NI], const Range (&outs)[NO])
{
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (overlaps(outs[i], ins[j])) return false;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlaps(outs[i], outs[j])) return false;
    }
    return true;
}
inline bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline size_t elem_size(int dtype) { return dtype == SSD_DTYPE_BF16 ? 2 : 4; }
inline bool known_dtype(int dtype) { return dtype == SSD_DTYPE_F32 || dtype == SSD_DTYPE_BF16; }
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// A launch has fewer than 2^32 threads: workgroups of 256.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;

}  // namespace ssd
