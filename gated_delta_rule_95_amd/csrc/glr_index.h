// What the tiles' kernels do with indices, tables of sequences and the words of
// the chain, without a device's builtins: the tests run the same code on the
// host.  A `Wave` is 64 lanes: each(f) runs f(lane) for every lane, count, any
// and all ask f(lane) of all of them, last(f) is f of the last lane, sleep()
// lets time pass; a Wave::Each<T> is a T for each lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_launch.h"
#include "glr_plan.h"

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


// An affine map h -> A h + B of a channel's state.  A = -0 forgets: whatever
// comes in, infinities and NaN of another sequence included, goes nowhere.  (A
// product of factors that is too small for fp32 is +0 and forgets no NaN.)
constexpr float kForget = -0.f;
__host__ __device__ __forceinline__ uint32_t bits_of(float x)
{
    uint32_t u;
    __builtin_memcpy(&u, &x, 4);
    return u;
}
__host__ __device__ __forceinline__ float float_of(uint32_t u)
{
    float x;
    __builtin_memcpy(&x, &u, 4);
    return x;
}
struct Map {
    float A, B;
    __host__ __device__ __forceinline__ bool forgets() const { return bits_of(A) == 0x80000000u; }
    __host__ __device__ __forceinline__ float operator()(float h) const
    {
        return forgets() ? B : __builtin_fmaf(A, h, B);
    }
};
// `late` after `early`
__host__ __device__ __forceinline__ Map after(const Map &late, const Map &early)
{
    return Map{late.forgets() || early.forgets() ? kForget : late.A * early.A, late(early.B)};
}

// Maps travel between workgroups as one 64-bit word that is stored and loaded
// whole, so a word is either empty or a map, and no order between words is
// asked for.  kEmpty is a NaN that no A is stored as.
constexpr uint64_t kEmpty = ~(uint64_t)0;
__host__ __device__ __forceinline__ uint64_t word_of(const Map &m)
{
    const uint32_t a = m.A != m.A ? 0x7fc00000u : bits_of(m.A);
    return (uint64_t)a << 32 | bits_of(m.B);
}
__host__ __device__ __forceinline__ Map map_of(uint64_t w)
{
    return Map{float_of((uint32_t)(w >> 32)), float_of((uint32_t)w)};
}

// The state (or cotangent) that comes into a tile, from the words of the `n`
// tiles before it, the first of which forgets: peek(lane, i, j) is the word of
// the i-th nearest, i < n, and the lane's j-th channel.  Of the nearest W,
// those from the first one on that forgets are not wanted; the others' maps are
// applied to its B, the farthest first.  That is what each of these tiles does,
// or did, to get at the map that forgets which it stores in the end, so the
// result does not depend on how far they have come, to the last bit.  (Eight words a lane; with 16 the scan of 65536
// tokens of 4096 channels takes 369 us and not 357, scan and gradients of 20011
// plain ones 331 and not 316: every look goes past the caches.)
// The wait is bounded all the same, for a workspace that something else writes
// while the call runs: after kPatience looks (a second or more; the longest
// wait of a sound call is some 100 us) the state becomes NaN.
constexpr int kPatience = 1 << 20;
template <int W, int V> struct Words {
    uint64_t w[W][V];
};
template <int V> struct Values {
    float x[V];
};
template <int W, int V, typename Wave, typename Peek, typename Active>
__host__ __device__ __forceinline__ void look(const Wave &wave, const Peek &peek, int n, const Active &active,
                                              typename Wave::template Each<Values<V>> &in, int patience = kPatience)
{
    typename Wave::template Each<Words<W, V>> near;
    int from = W;
    for (int looks = 0; looks < patience; ++looks) {
        wave.each([&](int lane) {
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) near[lane].w[i][j] = peek(lane, i < n ? i : n - 1, j);
        });
        from = W;
        bool there = true;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            there = there && wave.all([&](int lane) {
                bool full = true;
#pragma unroll
                for (int j = 0; j < V; ++j) full = full && near[lane].w[i][j] != kEmpty;
                return full || !active(lane);
            });
            if (there && from == W && wave.all([&](int lane) {
                    bool forgets = true;
#pragma unroll
                    for (int j = 0; j < V; ++j) forgets = forgets && map_of(near[lane].w[i][j]).forgets();
                    return forgets || !active(lane);
                }))
                from = i;
        }
        if (from < W) break;
        wave.sleep();
    }
    wave.each([&](int lane) {
#pragma unroll
        for (int i = W - 1; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const Map m = map_of(near[lane].w[i][j]);
                float &h = in[lane].x[j];
                h = i > from ? 0.f : i == from ? m.B : m(h);
            }
        if (from == W)
#pragma unroll
            for (int j = 0; j < V; ++j) in[lane].x[j] = __builtin_nanf("");
    });
}

// The first sequence from `lo` on that ends behind token t (n_seqs where none
// does), 64 table entries at a time.
template <typename Wave>
__host__ __device__ __forceinline__ int ends_behind(const Wave &wave, const gdr::SeqArgs &s, int lo, int t)
{
    int hi = s.n_seqs;
    while (lo < hi) {
        const int step = (hi - lo + kLanes - 1) / kLanes;
        const int ended = wave.count([&](int lane) {
            const int64_t n = lo + (int64_t)lane * step;
            return n < hi && gdr::seq_edge(s, (int)(n < hi ? n : lo) + 1) <= t;
        });
        const int64_t next = lo + (int64_t)ended * step;
        if (ended) lo += (ended - 1) * step + 1;
        hi = next < hi ? (int)next : hi;
    }
    return lo;
}

// Each lane's sequence, where there are no more of them than lanes: asked for
// before the tile is known (20011 tokens, gated: scan 153 -> 147 us, gradients
// 275 -> 272; 1517 in fp32: gradients 12.1 -> 11.5).
struct Edges {
    int b, e;
};
__host__ __device__ __forceinline__ Edges few_edges(const gdr::SeqArgs &s, int lane)
{
    Edges x{0, 0};
    if (s.cu_seqlens && s.n_seqs <= kLanes) {
        const int n = lane < s.n_seqs ? lane : 0;
        x.b = gdr::seq_edge(s, n);
        x.e = lane < s.n_seqs ? gdr::seq_edge(s, n + 1) : x.b;
    }
    return x;
}

// Borders of sequences inside tokens [t0, t0 + C): first[k] = the sequence
// whose first token is t0 + k, last[k] = the one whose last it is (entries
// that are neither keep the -1 that the caller put there).  few(lane): that
// lane's few_edges.  A table that breaks its contract gives any sequences, but
// only such as there are.  Empty sequences in a row are looked over 64 at once,
// and from the first 64 that end in one on by a search, so that a table padded
// with any number of them costs a tile no more than its tokens' worth of
// searches.
template <typename Wave, typename Few>
__host__ __device__ __forceinline__ void mark_borders(const Wave &wave, const gdr::SeqArgs &s, const Few &few, int t0, int C,
                                                      int *first, int *last)
{
    const auto mark = [&](int n, const Edges &x) {
        if (x.e <= x.b) return;
        if (x.b >= t0 && x.b - t0 < C) first[x.b - t0] = n;
        if (x.e - 1 >= t0 && x.e - 1 - t0 < C) last[x.e - 1 - t0] = n;
    };
    if (!s.cu_seqlens) {
        wave.each([&](int lane) {
            for (int k = lane; k < C; k += kLanes) {
                const unsigned t = (unsigned)(t0 + k), n = t / (unsigned)s.seqlen, at = t - n * (unsigned)s.seqlen;
                if (t >= (unsigned)s.n_tokens) break;
                if (at == 0) first[k] = (int)n;
                if (at + 1 == (unsigned)s.seqlen) last[k] = (int)n;
            }
        });
        return;
    }
    if (s.n_seqs <= kLanes) {
        wave.each([&](int lane) { mark(lane, few(lane)); });
        return;
    }
    for (int64_t base = ends_behind(wave, s, 0, t0); base < s.n_seqs;) {
        typename Wave::template Each<Edges> x;
        wave.each([&](int lane) {
            const int64_t n = base + lane;
            x[lane] = Edges{t0 + C, t0 + C};
            if (n < s.n_seqs) {
                x[lane] = Edges{gdr::seq_edge(s, (int)n), gdr::seq_edge(s, (int)n + 1)};
                mark((int)n, x[lane]);
            }
        });
        if (wave.any([&](int lane) { return x[lane].b - t0 >= C; })) break;
        base += kLanes;
        const int at = wave.last([&](int lane) { return x[lane].e; });
        if (at == wave.last([&](int lane) { return x[lane].b; })) base = ends_behind(wave, s, (int)base, at);
    }
}

}  // namespace glr
