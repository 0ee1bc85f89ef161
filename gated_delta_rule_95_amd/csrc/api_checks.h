// Argument checks that the C-ABI layers of the gated delta rule, the gated
// linear recurrence and the pools share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_launch.h"

namespace api {

using kda::set_error;

inline kda_status ok() { return set_error(KDA_OK, "%s", ""); }

inline kda_status hip_status(hipError_t e, const char *what)
{
    if (e == hipSuccess) return ok();
    return set_error(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline kda_status check_dtype(kda_dtype t)
{
    if (t != KDA_F32 && t != KDA_BF16)
        return set_error(KDA_ERR_INVALID_ARG, "in_dtype %d is not a kda_dtype", (int)t);
    return KDA_OK;
}

struct Buf {
    const void *p;
    const char *name;
    bool required;
    size_t align, bytes;
    bool written;
};

inline kda_status check_bufs(const Buf *b, int n)
{
    for (int i = 0; i < n; ++i) {
        if (!b[i].p) {
            if (b[i].required) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", b[i].name);
        } else if (reinterpret_cast<uintptr_t>(b[i].p) % b[i].align)
            return set_error(KDA_ERR_INVALID_ARG, "%s is not %zu-byte aligned", b[i].name, b[i].align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; b[i].written && j < n; ++j) {
            if (j == i || !b[i].p || !b[j].p || !b[i].bytes || !b[j].bytes) continue;
            const char *x = static_cast<const char *>(b[i].p), *y = static_cast<const char *>(b[j].p);
            if (x < y + b[j].bytes && y < x + b[i].bytes)
                return set_error(KDA_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
        }
    return KDA_OK;
}

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace api
