// The plans of the state pools (which slots are taken, moved and renamed)
// without a device's builtins: the tests run the same code on the host.  A
// `Block` is Block::threads threads that do each step together: each(f) runs
// f(t) for thread t, sync() orders what they wrote, a Block::Each<T> is a T for
// each thread, and rank(f, g) asks f(t) of all of them, then runs g(t, f(t), how
// many threads below t said yes, how many in all) and returns how many in all.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pool_launch.h"

namespace pool {

__host__ __device__ __forceinline__ bool valid(const uint8_t *used, int n_slots, const int32_t *src, int i)
{
    if (!src) return true;
    const int j = src[i];
    return j >= 0 && j < n_slots && used[j];
}

// dst first holds the free slots in order (entry k the k-th lowest, k < n);
// rows, from the last to the first, then replace them by their own: row i
// has rank <= i, so what rows before it still want is not yet replaced.
// (What comes back from memory here, in the plan and at the copies is held
// against the bounds again: a list or workspace that another call writes
// meanwhile, against the contract, must not move an address out of its array.)
template <typename Block>
__host__ __device__ __forceinline__ void take(const Block &block, uint8_t *used, int n_slots, const int32_t *src, int n,
                                              int32_t *dst)
{
    constexpr int PT = Block::threads;
    int nfree = 0;
    for (int base = 0; base < n_slots && nfree < n; base += PT)
        nfree += block.rank(
            [&](int t) {
                const int j = base + t;
                return j < n_slots && !used[j];
            },
            [&](int t, bool f, int k, int) {
                k += nfree;
                if (f && k < n) dst[k] = base + t;
            });
    const auto row = [&](int i) { return i < n && valid(used, n_slots, src, i); };
    int before = 0;
    for (int base = 0; base < n; base += PT)
        before += block.rank([&](int t) { return row(base + t); }, [](int, bool, int, int) {});
    block.sync();
    for (int base = (n - 1) / PT * PT; base >= 0; base -= PT) {
        typename Block::template Each<int> to;
        before -= block.rank([&](int t) { return row(base + t); },
                             [&](int t, bool v, int k, int total) {
                                 k += before - total;
                                 to[t] = v && k >= 0 && k < nfree ? dst[k] : -1;
                             });
        block.sync();
        block.each([&](int t) {
            if (base + t < n) dst[base + t] = to[t];
        });
    }
    block.sync();
    block.each([&](int t) {
        for (int i = t; i < n; i += PT) {
            const int j = dst[i];
            if (j >= 0 && j < n_slots) used[j] = 1;
        }
    });
}

// A compaction: the k-th used slot at or behind the count of used ones moves
// into the k-th free one before it.
template <typename Block>
__host__ __device__ __forceinline__ void plan(const Block &block, uint8_t *used, int n_slots, int32_t *table, int64_t n_table,
                                              int32_t *remap, const Moves &m)
{
    constexpr int PT = Block::threads;
    int live = 0;
    for (int base = 0; base < n_slots; base += PT)
        live += block.rank([&](int t) { return base + t < n_slots && used[base + t]; }, [](int, bool, int, int) {});
    int holes = 0, movers = 0;
    for (int base = 0; base < n_slots; base += PT) {
        typename Block::template Each<bool> is;
        holes += block.rank(
            [&](int t) {
                const int j = base + t;
                is[t] = j < n_slots && used[j];
                return !is[t] && j < live;
            },
            [&](int t, bool hole, int k, int) {
                k += holes;
                if (hole && k < n_slots / 2) m.dst[k] = base + t;
            });
        movers += block.rank([&](int t) { return is[t] && base + t >= live; },
                             [&](int t, bool mover, int k, int) {
                                 const int j = base + t;
                                 k += movers;
                                 if (mover && k < n_slots / 2) m.src[k] = j;
                                 if (j < n_slots) remap[j] = is[t] ? j : -1;
                             });
    }
    // as many holes as movers, of n_slots in all
    movers = movers < n_slots / 2 ? movers : n_slots / 2;
    block.sync();
    block.each([&](int t) {
        for (int k = t; k < movers; k += PT) {
            const int j = m.src[k];
            if (j >= 0 && j < n_slots) remap[j] = m.dst[k];
        }
        for (int j = t; j < n_slots; j += PT) used[j] = j < live;
        if (t == 0) *m.count = movers;
    });
    block.sync();
    block.each([&](int t) {
        for (int64_t i = t; i < n_table; i += PT) {
            const int j = table[i];
            if (j >= 0 && j < n_slots) table[i] = remap[j];
        }
    });
}

}  // namespace pool
