// Host-only sanitizer driver (AddressSanitizer + UndefinedBehaviorSanitizer) of
// what the gated linear recurrence's kernels do with indices, tables of
// sequences and the words of the chain (glr_index.h): the kernels' own code,
// its 64 lanes one after another.  Tables and words lie in arrays of their exact
// sizes, so that an index outside them ends the run.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <functional>
#include <random>
#include <vector>

#include "glr_index.h"
#include "glr_plan.h"

static int failures = 0;
#define EXPECT(cond)                                                              \
    do {                                                                          \
        if (!(cond)) {                                                            \
            if (++failures < 20) std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
        }                                                                         \
    } while (0)

// Every address of a wave's loads lies in its rows, whether or not the scalar
// offset counts for a resource's bounds check; what the check drops, it drops
// either way.
static void rows()
{
    for (int64_t D : {1, 2, 63, 64, 77, 1001, 4096, 8191, (1 << 24) - 2, (1 << 24) - 1})
        for (int size : {2, 4})
            for (int n = 0; n <= glr::kScanTokens; ++n) {
                const uint64_t row = D * size, bytes = n * row;
                const glr::RowSpan s(n, (unsigned)row);
                EXPECT(bytes < glr::kNowhere);
                for (int k = 0; k < glr::kScanTokens; ++k) {
                    const uint64_t at = s.at(k);
                    EXPECT(k >= n || at == k * row);
                    // a row's last channel
                    EXPECT(n ? at + row <= bytes : at == 0);
                    // a lane without a channel: past the resource with and without `at`, and no wrap
                    EXPECT(glr::kNowhere >= bytes && glr::kNowhere + at <= UINT32_MAX && glr::kNowhere >= bytes - at);
                }
            }
}

static std::mt19937 gen(1);
static int below(int n) { return (int)(gen() % (unsigned)n); }

struct Wave {
    mutable int *rounds = nullptr;                       // loads that follow each other
    std::function<void()> wait;
    template <typename T> struct Each {
        T x[64];
        T &operator[](int lane) { return x[lane]; }
    };
    template <typename F> void each(const F &f) const
    {
        if (rounds) ++*rounds;
        for (int l = 0; l < 64; ++l) f(l);
    }
    template <typename F> int count(const F &f) const
    {
        if (rounds) ++*rounds;
        int n = 0;
        for (int l = 0; l < 64; ++l) n += f(l) ? 1 : 0;
        return n;
    }
    template <typename F> bool any(const F &f) const
    {
        for (int l = 0; l < 64; ++l)
            if (f(l)) return true;
        return false;
    }
    template <typename F> bool all(const F &f) const
    {
        for (int l = 0; l < 64; ++l)
            if (!f(l)) return false;
        return true;
    }
    template <typename F> int last(const F &f) const { return f(63); }
    void sleep() const { wait(); }
};

// the borders in a tile, as the kernels find them
static int borders(const gdr::SeqArgs &s, int t0, int C, std::vector<int> &first, std::vector<int> &last)
{
    first.assign(C, -1);
    last.assign(C, -1);
    int rounds = 0;
    Wave w;
    w.rounds = &rounds;
    glr::Edges few[64];
    for (int l = 0; l < 64; ++l) few[l] = glr::few_edges(s, l);
    glr::mark_borders(w, s, [&](int l) { return few[l]; }, t0, C, first.data(), last.data());
    return rounds;
}

// ... and of a table that keeps its contract, sequence after sequence
static void check_borders(const std::vector<int32_t> &cu, int tokens, int t0, int C, bool count_rounds)
{
    const gdr::SeqArgs s{cu.data(), (int32_t)cu.size() - 1, tokens, 0};
    std::vector<int> first, last, f(C, -1), e(C, -1);
    const int rounds = borders(s, t0, C, first, last);
    int ends = 0;
    for (size_t n = 0; n + 1 < cu.size(); ++n) {
        if (cu[n + 1] <= cu[n]) continue;
        if (cu[n] >= t0 && cu[n] < t0 + C) f[cu[n] - t0] = (int)n;
        if (cu[n + 1] > t0 && cu[n + 1] <= t0 + C) e[cu[n + 1] - 1 - t0] = (int)n, ++ends;
    }
    EXPECT(f == first && e == last);
    // a search (3 rounds for 2^18 sequences) and one look for each token at which sequences end, and the first
    if (count_rounds) EXPECT(rounds <= 4 * (ends + 2));
}

static void tables()
{
    for (int n : {1, 2, 5, 63, 64, 65, 127, 300, 5000})
        for (int trial = 0; trial < 25; ++trial) {
            std::vector<int32_t> cu{0};
            const int some[] = {0, 0, 0, 1, 31, 32, 33, 127, 128, 129, below(300)};
            for (int k = 0; k < n; ++k) cu.push_back(cu.back() + (n < 400 ? some[below(11)] : below(4) / 2));
            const int tokens = cu.back() + (trial % 3 ? 0 : 200);
            for (int C : {32, 64, 128})
                for (int k = 0, tiles = (cu.back() + C - 1) / C; k < tiles && k < 30; ++k)
                    check_borders(cu, tokens, (tiles < 30 ? k : below(tiles)) * C, C, false);
            // any numbers at all: sequences that there are, at places of the tile
            std::vector<int32_t> bad(n + 1);
            for (int32_t &x : bad) {
                const int any[] = {below(650) - 50, below(500), INT32_MIN, INT32_MAX};
                x = any[below(4)];
            }
            const gdr::SeqArgs s{bad.data(), n, 1 + below(500), 0};
            for (int C : {32, 64, 128})
                for (int t0 = 0; t0 < s.n_tokens; t0 += C) {
                    std::vector<int> first, last;
                    borders(s, t0, C, first, last);
                    for (int k = 0; k < C; ++k)
                        EXPECT(first[k] >= -1 && first[k] < n && last[k] >= -1 && last[k] < n);
                }
        }
    // the last tokens that there can be
    const std::vector<int32_t> far{0, 5, INT32_MAX - 255};
    check_borders(far, INT32_MAX - 255, (INT32_MAX - 255) / 128 * 128 - 128, 128, false);
    // runs of empty sequences
    for (int C : {32, 128}) {
        const int run = 70000;
        std::vector<int32_t> a(run, 0);
        a.push_back(5);
        a.insert(a.end(), run, 40);
        a.insert(a.end(), run, 200);
        std::vector<int32_t> b{0, 7}, c{0, 10, 10, 11};
        b.insert(b.end(), run, 7 + C);
        c.insert(c.end(), run, 64);
        for (const std::vector<int32_t> &cu : {a, b, c})
            for (int t0 = 0; t0 < cu.back(); t0 += C) check_borders(cu, cu.back(), t0, C, true);
    }
    // equal lengths
    for (int len : {1, 2, 31, 64, 100, 1000})
        for (int n : {1, 3, 70}) {
            const gdr::SeqArgs s{nullptr, n, n * len, len};
            std::vector<int32_t> cu;
            for (int k = 0; k <= n; ++k) cu.push_back(k * len);
            const gdr::SeqArgs t{cu.data(), n, n * len, 0};
            for (int t0 = 0; t0 < n * len; t0 += 128) {
                std::vector<int> f, l, g, m;
                borders(s, t0, 128, f, l);
                borders(t, t0, 128, g, m);
                EXPECT(f == g && l == m);
            }
        }
}

// Words of tiles in any state of progress (a map, or what the tile stores in
// the end) give the same state, bit for bit, and a wait ends once the tiles
// before have stored theirs.
template <int W, int V> static void chains()
{
    std::uniform_real_distribution<float> u(0, 1);
    for (int trial = 0; trial < 300; ++trial) {
        const int n = 1 + below(40), active = 1 + below(64);
        std::vector<glr::Map> maps(n * 64 * V), done(n * 64 * V);
        const auto at = [&](int tile, int lane, int j) { return (tile * 64 + lane) * V + j; };
        for (int k = 0; k < n; ++k) {
            const bool forgets = k == 0 || below(10) == 0;
            for (int l = 0; l < 64; ++l)
                for (int j = 0; j < V; ++j) {
                    glr::Map m{forgets ? glr::kForget : u(gen), 2 * u(gen) - 1};
                    if (!forgets && below(50) == 0) m.A = 0;                 // a product that is too small
                    if (!forgets && below(300) == 0) m.A = -std::nanf("0xfffff");
                    if (below(300) == 0) m.B = below(2) ? INFINITY : std::nanf("");
                    maps[at(k, l, j)] = m;
                    done[at(k, l, j)] = glr::Map{glr::kForget, k ? m(done[at(k - 1, l, j)].B) : m.B};
                }
        }
        int finished = below(n), stored = finished + below(n - finished + 1), waits = 0;
        Wave wave;
        wave.wait = [&] {
            stored = stored < n ? stored + 1 : n;
            finished = finished < n ? finished + 1 : n;
            ++waits;
        };
        const auto peek = [&](int lane, int i, int j) {
            EXPECT(i >= 0 && i < n && j >= 0 && j < V);
            const int tile = n - 1 - i, x = at(tile, lane, j);
            if (lane >= active || tile >= stored) return glr::kEmpty;
            return glr::word_of(tile < finished ? done[x] : maps[x]);
        };
        typename Wave::template Each<glr::Values<V>> in{};
        glr::look<W, V>(wave, peek, n, [&](int lane) { return lane < active; }, in);
        EXPECT(waits <= n + 1);
        for (int l = 0; l < active; ++l)
            for (int j = 0; j < V; ++j) {
                const float want = done[at(n - 1, l, j)].B, got = in[l].x[j];
                EXPECT(glr::bits_of(want) == glr::bits_of(got) || (want != want && got != got));
            }
    }
    // words that never come: the wait ends, and says so
    int looks = 0;
    Wave wave;
    wave.wait = [&] { ++looks; };
    typename Wave::template Each<glr::Values<V>> in{};
    glr::look<W, V>(wave, [](int, int, int) { return glr::kEmpty; }, 3, [](int) { return true; }, in, 50);
    EXPECT(looks == 50 && in[0].x[0] != in[0].x[0] && in[63].x[V - 1] != in[63].x[V - 1]);
}

// a word holds any map, and none is empty
static void words()
{
    const float some[] = {0.f, -0.f, 1.f, 1e-45f, 3.4e38f, INFINITY, -INFINITY, std::nanf(""), -std::nanf("0x3fffff")};
    for (float a : some)
        for (float b : some) {
            const uint64_t w = glr::word_of(glr::Map{a, b});
            const glr::Map m = glr::map_of(w);
            EXPECT(w != glr::kEmpty && glr::bits_of(m.B) == glr::bits_of(b) && (a != a ? m.A != m.A : glr::bits_of(m.A) == glr::bits_of(a)));
            EXPECT(m.forgets() == (a == 0 && std::signbit(a)));
        }
    // what comes in meets no map that forgets, and passes one that is too small
    EXPECT((glr::Map{glr::kForget, 2.f}(std::nanf("")) == 2.f) && std::isnan(glr::Map{0.f, 2.f}(INFINITY)));
    EXPECT(glr::after(glr::Map{0.5f, 1.f}, glr::Map{glr::kForget, 2.f}).forgets() && glr::after(glr::Map{glr::kForget, 1.f}, glr::Map{0.5f, NAN}).B == 1.f);
}

int main()
{
    rows();
    tables();
    words();
    chains<8, 1>();
    chains<4, 2>();
    if (failures) return 1;
    std::printf("sanitized index checks of the linear recurrence passed\n");
    return 0;
}
