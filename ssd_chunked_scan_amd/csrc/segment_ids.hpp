// segment_ids.hpp -- where a packed stream's segments are, in range for any 32-bit ids
// (plain C++: the host's tests compile it too).
#pragma once

#include <cstdint>

#ifdef __HIPCC__
#define SSD_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SSD_HOST_DEVICE inline
#endif

namespace ssd {

// Segments from .. to - 1, in [0, nseq].
struct Segments {
    int32_t from, to;
};
// Ids outside [0, nseq) become -1 and nseq before anything is added to them.
SSD_HOST_DEVICE int32_t clamp_id(int32_t id, int32_t nseq) { return id < 0 ? -1 : id < nseq ? id : nseq; }
// Those after `prev` and up to `id`: their first token, or the first of a later one, is the token with `id` that
// follows one with `prev` (-1 in front of the stream).
SSD_HOST_DEVICE Segments segments_through(int32_t prev, int32_t id, int32_t nseq)
{
    const int32_t p = clamp_id(prev, nseq), i = clamp_id(id, nseq);
    return Segments{p < nseq ? p + 1 : nseq, i < nseq ? i + 1 : nseq};
}
// The first of T tokens whose id is not below `q`, T if there is none.
SSD_HOST_DEVICE int32_t first_from(const int32_t *ids, int32_t T, int32_t q)
{
    int32_t lo = 0, hi = T;
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (ids[mid] < q) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

}  // namespace ssd
