// C-ABI layer of the state pools: argument validation and errors.
// Declarations and the contract of every entry point are in include/pool.h.
#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "pool.h"
#include "pool_launch.h"

#define POOL_API extern "C" __attribute__((visibility("default")))

namespace {

using api::Buf;
using api::check_bufs;
using api::hip_status;
using api::ok;
using api::set_error;

constexpr int32_t kMost = 1 << 24;

kda_status check_count(int64_t n, const char *name)
{
    if (n < 0) return set_error(KDA_ERR_INVALID_ARG, "%s must be >= 0 (got %lld)", name, (long long)n);
    if (n > kMost) return set_error(KDA_ERR_INVALID_ARG, "%s must be at most 2^24", name);
    return KDA_OK;
}

bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return a && b && an && bn && x < y + bn && y < x + an;
}

size_t bytes_of(const pool_rows &p, int32_t n_slots) { return p.row_bytes * (size_t)n_slots; }

kda_status check_pools(const pool_rows *p, int32_t n_pools, int32_t n_slots, const char *name)
{
    if (n_pools < 0) return set_error(KDA_ERR_INVALID_ARG, "n_pools must be >= 0 (got %d)", n_pools);
    if (n_pools && !p) return set_error(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    for (int i = 0; i < n_pools; ++i) {
        if (p[i].row_bytes < 1 || p[i].row_bytes > (size_t)1 << 40)
            return set_error(KDA_ERR_INVALID_ARG, "row_bytes of %s[%d] must be 1 .. 2^40", name, i);
        // (by division: 2^40 times 2^24 is 0 in 64 bits)
        if (n_slots && p[i].row_bytes > (((size_t)1 << 46) - 1) / (size_t)n_slots)
            return set_error(KDA_ERR_INVALID_ARG, "%s[%d] must be below 2^46 bytes", name, i);
        if (n_slots && !p[i].base) return set_error(KDA_ERR_INVALID_ARG, "%s[%d] is NULL", name, i);
    }
    return KDA_OK;
}

// no written pool may share memory with another pool or one of the arrays
kda_status check_apart(const pool_rows *p, int32_t n_pools, int32_t n_slots, const char *name, const Buf *b,
                       int n)
{
    for (int i = 0; i < n_pools; ++i) {
        const size_t pb = bytes_of(p[i], n_slots);
        for (int j = 0; j < n; ++j)
            if (overlap(p[i].base, pb, b[j].p, b[j].bytes))
                return set_error(KDA_ERR_INVALID_ARG, "%s[%d] overlaps %s", name, i, b[j].name);
        for (int j = 0; j < i; ++j)
            if (overlap(p[i].base, pb, p[j].base, bytes_of(p[j], n_slots)))
                return set_error(KDA_ERR_INVALID_ARG, "%s[%d] overlaps %s[%d]", name, i, name, j);
    }
    return KDA_OK;
}

}  // namespace

POOL_API kda_status pool_copy(const pool_rows *from, const pool_rows *to, int32_t n_pools,
                              int32_t from_slots, int32_t to_slots, const int32_t *src,
                              const int32_t *dst, int32_t n, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_count(from_slots, "from_slots")) != KDA_OK) return s;
    if ((s = check_count(to_slots, "to_slots")) != KDA_OK) return s;
    if ((s = check_count(n, "n")) != KDA_OK) return s;
    if ((s = check_pools(from, n_pools, from_slots, "from")) != KDA_OK) return s;
    if ((s = check_pools(to, n_pools, to_slots, "to")) != KDA_OK) return s;
    const Buf bufs[] = {{src, "src", n > 0, 4, (size_t)n * 4, false}, {dst, "dst", n > 0, 4, (size_t)n * 4, false}};
    if ((s = check_bufs(bufs, 2)) != KDA_OK) return s;
    if ((s = check_apart(to, n_pools, to_slots, "to", bufs, 2)) != KDA_OK) return s;
    for (int i = 0; i < n_pools; ++i) {
        if (from[i].row_bytes != to[i].row_bytes)
            return set_error(KDA_ERR_INVALID_ARG, "from[%d] and to[%d] have rows of different sizes", i, i);
        for (int j = 0; j < n_pools; ++j) {
            const bool same = i == j && from[j].base == to[i].base;
            if (!same && overlap(to[i].base, bytes_of(to[i], to_slots), from[j].base, bytes_of(from[j], from_slots)))
                return set_error(KDA_ERR_INVALID_ARG, "to[%d] overlaps from[%d] without being the same pool", i, j);
        }
    }
    if (!n || !n_pools || !from_slots || !to_slots) return ok();
    return hip_status(pool::launch_copy(from, to, n_pools, pool::Pairs{src, dst, nullptr, n, from_slots, to_slots},
                                        static_cast<hipStream_t>(stream)), "pool_copy launch");
}

POOL_API kda_status pool_alloc(const pool_rows *pools, int32_t n_pools, uint8_t *used,
                               int32_t n_slots, int32_t n, int32_t *slots, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_count(n_slots, "n_slots")) != KDA_OK) return s;
    if ((s = check_count(n, "n")) != KDA_OK) return s;
    if ((s = check_pools(pools, n_pools, n_slots, "pools")) != KDA_OK) return s;
    const Buf bufs[] = {{used, "used", n_slots > 0, 1, (size_t)n_slots, true},
                        {slots, "slots", n > 0, 4, (size_t)n * 4, true}};
    if ((s = check_bufs(bufs, 2)) != KDA_OK) return s;
    if ((s = check_apart(pools, n_pools, n_slots, "pools", bufs, 2)) != KDA_OK) return s;
    if (!n) return ok();
    return hip_status(pool::launch_take(pools, n_pools, used, n_slots, nullptr, n, slots, static_cast<hipStream_t>(stream)),
                      "pool_alloc launch");
}

POOL_API kda_status pool_fork(const pool_rows *pools, int32_t n_pools, uint8_t *used, int32_t n_slots,
                              const int32_t *src, int32_t n, int32_t *dst, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_count(n_slots, "n_slots")) != KDA_OK) return s;
    if ((s = check_count(n, "n")) != KDA_OK) return s;
    if ((s = check_pools(pools, n_pools, n_slots, "pools")) != KDA_OK) return s;
    const Buf bufs[] = {{used, "used", n_slots > 0, 1, (size_t)n_slots, true},
                        {src, "src", n > 0, 4, (size_t)n * 4, false},
                        {dst, "dst", n > 0, 4, (size_t)n * 4, true}};
    if ((s = check_bufs(bufs, 3)) != KDA_OK) return s;
    if ((s = check_apart(pools, n_pools, n_slots, "pools", bufs, 3)) != KDA_OK) return s;
    if (!n) return ok();
    return hip_status(pool::launch_take(pools, n_pools, used, n_slots, src, n, dst, static_cast<hipStream_t>(stream)),
                      "pool_fork launch");
}

POOL_API kda_status pool_free(uint8_t *used, int32_t n_slots, const int32_t *slots, int32_t n,
                              kda_stream_t stream)
{
    kda_status s;
    if ((s = check_count(n_slots, "n_slots")) != KDA_OK) return s;
    if ((s = check_count(n, "n")) != KDA_OK) return s;
    const Buf bufs[] = {{used, "used", n_slots > 0, 1, (size_t)n_slots, true},
                        {slots, "slots", n > 0, 4, (size_t)n * 4, false}};
    if ((s = check_bufs(bufs, 2)) != KDA_OK) return s;
    if (!n || !n_slots) return ok();
    return hip_status(pool::launch_free(used, n_slots, slots, n, static_cast<hipStream_t>(stream)),
                      "pool_free launch");
}

POOL_API size_t pool_compact_workspace_bytes(int32_t n_slots)
{
    return check_count(n_slots, "n_slots") == KDA_OK ? pool::Moves::bytes(n_slots) : 0;
}

POOL_API kda_status pool_compact(const pool_rows *pools, int32_t n_pools, uint8_t *used,
                                 int32_t n_slots, int32_t *table, int64_t n_table, int32_t *remap,
                                 void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    kda_status s;
    if ((s = check_count(n_slots, "n_slots")) != KDA_OK) return s;
    if ((s = check_count(n_table, "n_table")) != KDA_OK) return s;
    if ((s = check_pools(pools, n_pools, n_slots, "pools")) != KDA_OK) return s;
    const size_t need = pool::Moves::bytes(n_slots);
    if (workspace && workspace_bytes < need)
        return set_error(KDA_ERR_INVALID_ARG,
                         "workspace_bytes %zu is below the %zu bytes pool_compact_workspace_bytes gives",
                         workspace_bytes, need);
    const Buf bufs[] = {{used, "used", n_slots > 0, 1, (size_t)n_slots, true},
                        {table, "table", n_table > 0, 4, (size_t)n_table * 4, true},
                        {remap, "remap", n_slots > 0, 4, (size_t)n_slots * 4, true},
                        {workspace, "workspace", true, 256, need, true}};
    if ((s = check_bufs(bufs, 4)) != KDA_OK) return s;
    if ((s = check_apart(pools, n_pools, n_slots, "pools", bufs, 4)) != KDA_OK) return s;
    if (!n_slots) return ok();
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const pool::Moves m(workspace, n_slots);
    hipError_t e = pool::launch_plan(used, n_slots, table, n_table, remap, m, st);
    if (e == hipSuccess && n_pools && n_slots > 1)
        e = pool::launch_copy(pools, pools, n_pools,
                              pool::Pairs{m.src, m.dst, m.count, n_slots / 2, n_slots, n_slots}, st);
    return hip_status(e, "pool_compact launch");
}
