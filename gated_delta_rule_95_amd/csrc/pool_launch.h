// Internal launch interface of the state pools (pool_*) between the C-ABI
// layer (pool_api.cpp) and the kernels.  Arguments arrive here already
// validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pool.h"

namespace pool {

// The pairs of slots that a launch copies: pair i is (src[i], dst[i]) for i <
// n, or for i < *count (at most n) where count is not NULL.
struct Pairs {
    const int32_t *src, *dst, *count;
    int32_t n, from_slots, to_slots;
};

// rows to rows (from nullptr: zeros to rows; pairs.src is not read then)
hipError_t launch_copy(const pool_rows *from, const pool_rows *to, int32_t n_pools, const Pairs &pairs,
                       hipStream_t s);
// dst[i]: the free slot row i gets, or -1, with the rows of slot src[i]; src
// nullptr: every row wants one, of zeros
hipError_t launch_take(const pool_rows *pools, int32_t n_pools, uint8_t *used, int32_t n_slots,
                       const int32_t *src, int32_t n, int32_t *dst, hipStream_t s);
hipError_t launch_free(uint8_t *used, int32_t n_slots, const int32_t *slots, int32_t n, hipStream_t s);

// the workspace of a compaction: how many slots move, from where, to where
struct Moves {
    int32_t *count, *src, *dst;
    static size_t list(int32_t n_slots) { return (((size_t)n_slots / 2 * 4) + 255) & ~(size_t)255; }
    static size_t bytes(int32_t n_slots) { return 256 + 2 * list(n_slots); }
    Moves(void *ws, int32_t n_slots)
    {
        char *w = static_cast<char *>(ws);
        count = reinterpret_cast<int32_t *>(w);
        src = reinterpret_cast<int32_t *>(w + 256);
        dst = reinterpret_cast<int32_t *>(w + 256 + list(n_slots));
    }
};
hipError_t launch_plan(uint8_t *used, int32_t n_slots, int32_t *table, int64_t n_table, int32_t *remap,
                       const Moves &m, hipStream_t s);

}  // namespace pool
