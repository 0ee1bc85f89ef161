// Index arithmetic of the tiles' kernels that asks nothing of a device: the
// tests run the same code on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace glr {

// Where a wave's `rows` rows of `row` bytes each lie behind the first of them.
// A row past the last counts as the last (as the first where there is none):
// these offsets are formed as scalar offsets of buffer loads, which the bounds
// check of a resource need not see, so none may lead out of the rows by itself.
struct RowSpan {
    unsigned row, last;
    __host__ __device__ RowSpan(int rows, unsigned row) : row(row), last(rows > 0 ? (unsigned)(rows - 1) * row : 0u) {}
    __host__ __device__ unsigned at(int k) const
    {
        const unsigned x = (unsigned)k * row;
        return x < last ? x : last;
    }
};

// a lane's offset where it has no channel: past every resource, and so is its
// sum with any of the offsets above
constexpr unsigned kNowhere = 0x80000000u;

}  // namespace glr
