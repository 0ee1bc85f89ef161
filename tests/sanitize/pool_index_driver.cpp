// Host-only sanitizer driver (AddressSanitizer + UndefinedBehaviorSanitizer) of
// the plans of the state pools (pool_index.h): the kernels' own code, the
// threads of each step one after another in a random order.  Arrays have their
// exact sizes, so that an index outside them ends the run.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <numeric>
#include <random>
#include <vector>

#include "pool_index.h"

static int failures = 0;
#define EXPECT(cond)                                                              \
    do {                                                                          \
        if (!(cond)) {                                                            \
            if (++failures < 20) std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
        }                                                                         \
    } while (0)

static std::mt19937 gen(1);
static int below(int n) { return (int)(gen() % (unsigned)n); }

template <int PT> struct Block {
    static constexpr int threads = PT;
    template <typename T> struct Each {
        T x[PT];
        T &operator[](int t) { return x[t]; }
    };
    static std::vector<int> order()
    {
        std::vector<int> o(PT);
        std::iota(o.begin(), o.end(), 0);
        std::shuffle(o.begin(), o.end(), gen);
        return o;
    }
    template <typename F> void each(const F &f) const
    {
        for (int t : order()) f(t);
    }
    void sync() const {}
    template <typename F, typename G> int rank(const F &f, const G &g) const
    {
        bool x[PT];
        int k[PT], all = 0;
        for (int t : order()) x[t] = f(t);
        for (int t = 0; t < PT; ++t) {
            k[t] = all;
            all += x[t];
        }
        for (int t : order()) g(t, x[t], k[t], all);
        return all;
    }
};

template <int PT> static void takes(int trials, int most)
{
    for (int trial = 0; trial < trials; ++trial) {
        const int n_slots = below(most), n = 1 + below(most), share = below(5);
        std::vector<uint8_t> used(n_slots);
        for (uint8_t &u : used) u = below(4) < share ? 1 + below(255) : 0;
        std::vector<int32_t> src(n), dst(n, -77), want(n, -1);
        for (int32_t &s : src) {
            const int any[] = {n_slots ? below(n_slots) : 0, below(n_slots + 4) - 2, INT32_MIN, INT32_MAX};
            s = any[below(10) < 7 ? 0 : below(4)];
        }
        const bool alloc = below(3) == 0;
        std::vector<uint8_t> after = used;
        int next = 0;
        for (int i = 0; i < n; ++i) {
            if (!alloc && (src[i] < 0 || src[i] >= n_slots || !used[src[i]])) continue;
            while (next < n_slots && used[next]) ++next;
            if (next == n_slots) break;
            after[next] = 1;
            want[i] = next++;
        }
        pool::take(Block<PT>(), used.data(), n_slots, alloc ? nullptr : src.data(), n, dst.data());
        EXPECT(dst == want && used == after);
    }
}

template <int PT> static void plans(int trials, int most)
{
    for (int trial = 0; trial < trials; ++trial) {
        const int n_slots = 1 + below(most), n_table = below(most), share = below(5);
        std::vector<uint8_t> used(n_slots);
        for (uint8_t &u : used) u = below(4) < share ? 1 + below(255) : 0;
        std::vector<int32_t> table(n_table), remap(n_slots, -77), src(n_slots / 2, -77), dst(n_slots / 2, -77);
        for (int32_t &x : table) {
            const int any[] = {below(n_slots), below(n_slots + 4) - 2, INT32_MIN, INT32_MAX};
            x = any[below(4)];
        }
        int live = 0, count = -1;
        for (uint8_t u : used) live += u != 0;
        std::vector<int32_t> want_map(n_slots, -1), from, to;
        for (int j = 0; j < n_slots; ++j) {
            if (used[j] && j < live) want_map[j] = j;
            if (used[j] && j >= live) from.push_back(j);
            if (!used[j] && j < live) to.push_back(j);
        }
        EXPECT(from.size() == to.size());
        for (size_t k = 0; k < from.size(); ++k) want_map[from[k]] = to[k];
        std::vector<int32_t> want_table = table;
        for (int32_t &x : want_table)
            if (x >= 0 && x < n_slots) x = want_map[x];
        pool::Moves m(nullptr, n_slots);
        m.count = &count;
        m.src = src.data();
        m.dst = dst.data();
        pool::plan(Block<PT>(), used.data(), n_slots, table.data(), n_table, remap.data(), m);
        EXPECT(count == (int)from.size() && std::equal(from.begin(), from.end(), src.begin()) && std::equal(to.begin(), to.end(), dst.begin()));
        EXPECT(remap == want_map && table == want_table);
        for (int j = 0; j < n_slots; ++j) EXPECT(used[j] == (j < live));
    }
}

int main()
{
    takes<1>(500, 12);
    takes<4>(3000, 40);
    takes<64>(1000, 300);
    takes<1024>(20, 5000);
    plans<1>(500, 12);
    plans<4>(3000, 40);
    plans<64>(1000, 300);
    plans<1024>(20, 5000);
    if (failures) return 1;
    std::printf("sanitized plans of the pools passed\n");
    return 0;
}
