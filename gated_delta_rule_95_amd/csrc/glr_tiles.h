// What the scan and its gradients share: tiles of tokens and channels handed
// out in order, sequence borders inside a tile, and the chain of states from
// tile to tile (gfx950 only).
#pragma once

#include <type_traits>

#include "glr_device.h"
#include "glr_index.h"
#include "glr_plan.h"

namespace glr {

// V neighbouring channels of a row, as stored and in fp32
template <typename T, int V> struct Row {
    typedef T raw __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ float get(raw x, int j) { return (float)x[j]; }
    static __device__ __forceinline__ raw pack(const float *x)
    {
        raw v;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = (T)x[j];
        return v;
    }
};
template <typename T> struct Row<T, 1> {
    typedef T raw;
    static __device__ __forceinline__ float get(raw x, int) { return (float)x; }
    static __device__ __forceinline__ raw pack(const float *x) { return (T)x[0]; }
};
template <int V, typename T>
__device__ __forceinline__ typename Row<T, V>::raw ld(const T *p)
{
    return *reinterpret_cast<const typename Row<T, V>::raw *>(p);
}
template <int V, typename T>
__device__ __forceinline__ void st(T *p, const float *x)
{
    *reinterpret_cast<typename Row<T, V>::raw *>(p) = Row<T, V>::pack(x);
}

// A wave's rows of a tensor [.., D] as a buffer resource: `rows` of them from
// `first` on (D < 2^24 keeps their bytes below 2^31).  A row is a scalar
// offset and a lane's channel a vector one, so addresses cost no vector
// arithmetic.  The resource's size drops channels at kNowhere, and all where
// there is no row; it is not relied on for rows, as the scalar offset may be no
// part of its check: a row past the last is read as the last, and not stored.
// Pairs (the large calls) stream past the caches, "nt" both ways: 65536 tokens
// of 4096 channels 408 -> 391 us, the gradients of 20011 gated ones 281 -> 272;
// single channels (the small calls, whose rows the caches may hold) do not:
// 1517 tokens of 1001 in fp32 took 25.6 us, with it 26.5.
template <typename T, int V> struct Rows {
    static constexpr int kCache = V == 2 ? 2 : 0;
    typedef typename Row<T, V>::raw raw;
    gdr::rsrc_t r;
    RowSpan span;
    __device__ __forceinline__ Rows(const void *p, int64_t first, int rows, int D)
        : r(gdr::make_rsrc(static_cast<const T *>(p) + first * D, rows * D * (int)sizeof(T))),
          span(rows, (unsigned)D * (unsigned)sizeof(T))
    {
    }
    // c: the lane's channel times the size of an element, or kNowhere; st: k below `rows`
    __device__ __forceinline__ raw ld(int k, unsigned c) const
    {
        const unsigned at = span.at(k);
        if constexpr (sizeof(raw) == 2)
            return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b16(r, c, at, kCache));
        else if constexpr (sizeof(raw) == 4)
            return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b32(r, c, at, kCache));
        else
            return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(r, c, at, kCache));
    }
    __device__ __forceinline__ void st(int k, unsigned c, const float *x) const
    {
        const raw v = Row<T, V>::pack(x);
        const unsigned at = span.at(k);
        typedef unsigned u2 __attribute__((ext_vector_type(2)));
        if constexpr (sizeof(raw) == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), r, c, at, kCache);
        else if constexpr (sizeof(raw) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, c, at, kCache);
        else
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, v), r, c, at, kCache);
    }
};

// An affine map h -> A h + B of a channel's state.  A = -0 forgets: whatever
// comes in, infinities and NaN of another sequence included, goes nowhere.  (A
// product of factors that is too small for fp32 is +0 and forgets no NaN.)
constexpr float kForget = -0.f;
struct Map {
    float A, B;
    __device__ __forceinline__ bool forgets() const { return __float_as_uint(A) == 0x80000000u; }
    __device__ __forceinline__ float operator()(float h) const
    {
        return forgets() ? B : __builtin_fmaf(A, h, B);
    }
};
// `late` after `early`
__device__ __forceinline__ Map after(const Map &late, const Map &early)
{
    return Map{late.forgets() || early.forgets() ? kForget : late.A * early.A, late(early.B)};
}

// Maps travel between workgroups as one 64-bit word that is stored and loaded
// whole, so a word is either empty or a map, and no order between words is
// asked for.  kEmpty is a NaN that no A is stored as.
constexpr uint64_t kEmpty = ~(uint64_t)0;
__device__ __forceinline__ void put(uint64_t *p, const Map &m)
{
    const uint32_t a = m.A != m.A ? 0x7fc00000u : __float_as_uint(m.A);
    __hip_atomic_store(p, (uint64_t)a << 32 | __float_as_uint(m.B), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Map map_of(uint64_t w)
{
    return Map{__uint_as_float((uint32_t)(w >> 32)), __uint_as_float((uint32_t)w)};
}

// The block of channels of a tile's workgroup.  Workgroups go to the XCDs in
// turn, so that without the shift by a block a row of tiles each XCD would have
// the same columns of the tensors all along (20011 tokens of 4096 channels:
// scan 161 -> 152 us, gradients 318 -> 277; plain 142 -> 126 and 236 -> 200).
__device__ __forceinline__ int block_of(const Chain &c, int idx) { return (idx + idx / c.blocks) % c.blocks; }

// The next tile of a block of channels (Chain, in glr_plan.h).  Cleared tickets
// are ~0, as words are; what only something else's writes can give counts as
// the last tile.
__device__ __forceinline__ int take(const Chain &c, int block)
{
    if (!c.tickets) return 0;
    const unsigned n = atomicAdd(c.tickets + block * (kTicket / 4), 1u) + 1u, last = (unsigned)c.tiles - 1;
    return (int)(n < last ? n : last);
}
hipError_t clear_chain(const Chain &c, hipStream_t s);

// The state (or cotangent) that comes into a tile.  Words of the `n` tiles
// before it (the first of which forgets) lie `step` apart, from `p` on, the
// nearest first.  Of the nearest W, those from the first one on that forgets
// are not wanted; the others' maps are applied to its B, the farthest first.
// That is what each of these tiles does, or did, to get at the map that
// forgets which it stores in the end, so the result does not depend on how far
// they have come, to the last bit.  (Eight words a lane; with 16 the scan of 65536
// tokens of 4096 channels takes 392 us and not 382, the gradients of 20011 plain
// ones 214 and not 199: every look goes past the caches.)
// The wait is bounded all the same, for a workspace that something else writes
// while the call runs: after kPatience looks (a second or more; the longest
// wait of a sound call is some 100 us) the state becomes NaN.
constexpr int kPatience = 1 << 20;
template <int W, int V>
__device__ __forceinline__ void look_back(const uint64_t *p, int64_t step, int n, bool active, float *in)
{
    uint64_t w[W][V];
    int from = W;
    for (int looks = 0; looks < kPatience; ++looks) {
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) w[i][j] = peek(p + step * (i < n ? i : n - 1) + j * kLanes);
        from = W;
        bool there = true;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            bool full = true, forgets = true;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                full = full && w[i][j] != kEmpty;
                forgets = forgets && map_of(w[i][j]).forgets();
            }
            there = there && __all(full || !active);
            if (there && from == W && __all(forgets || !active)) from = i;
        }
        if (from < W) break;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int i = W - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Map m = map_of(w[i][j]);
            in[j] = i > from ? 0.f : i == from ? m.B : m(in[j]);
        }
    if (from == W)
#pragma unroll
        for (int j = 0; j < V; ++j) in[j] = __builtin_nanf("");
}

// The first sequence from `lo` on that ends behind token t (n_seqs where none
// does), 64 table entries at a time.  One wave; uniform.
__device__ __forceinline__ int ends_behind(const gdr::SeqArgs &s, int lo, int t, int lane)
{
    int hi = s.n_seqs;
    while (lo < hi) {
        const int step = (hi - lo + WAVE - 1) / WAVE;
        const int64_t n = lo + (int64_t)lane * step;
        const int ended = __popcll(__ballot(n < hi && gdr::seq_edge(s, (int)(n < hi ? n : lo) + 1) <= t));
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
__device__ __forceinline__ Edges few_edges(const gdr::SeqArgs &s, int lane)
{
    Edges x{0, 0};
    if (s.cu_seqlens && s.n_seqs <= WAVE) {
        const int n = lane < s.n_seqs ? lane : 0;
        x.b = gdr::seq_edge(s, n);
        x.e = lane < s.n_seqs ? gdr::seq_edge(s, n + 1) : x.b;
    }
    return x;
}

// Borders of sequences inside tokens [t0, t0 + C): first[k] = the sequence
// whose first token is t0 + k, last[k] = the one whose last it is (entries
// that are neither keep the -1 that the caller put there).  One wave; a table
// that breaks its contract gives any sequences, but only such as there are.
// Empty sequences in a row are looked over 64 at once, and from the first 64
// that end in one on by a search, so that a table padded with any number of
// them costs a tile no more than its tokens' worth of searches.
__device__ __forceinline__ void mark_borders(const gdr::SeqArgs &s, const Edges &few, int t0, int C, int lane, int *first,
                                             int *last)
{
    const auto mark = [&](int n, int b, int e) {
        if (e <= b) return;
        if (b >= t0 && b - t0 < C) first[b - t0] = n;
        if (e - 1 >= t0 && e - 1 - t0 < C) last[e - 1 - t0] = n;
    };
    if (!s.cu_seqlens) {
        for (int k = lane; k < C; k += WAVE) {
            const unsigned t = (unsigned)(t0 + k), n = t / (unsigned)s.seqlen, at = t - n * (unsigned)s.seqlen;
            if (t >= (unsigned)s.n_tokens) break;
            if (at == 0) first[k] = (int)n;
            if (at + 1 == (unsigned)s.seqlen) last[k] = (int)n;
        }
        return;
    }
    if (s.n_seqs <= WAVE) {
        mark(lane, few.b, few.e);
        return;
    }
    for (int64_t base = ends_behind(s, 0, t0, lane); base < s.n_seqs;) {
        const int64_t n = base + lane;
        int b = t0 + C, e = b;
        if (n < s.n_seqs) {
            b = gdr::seq_edge(s, (int)n);
            e = gdr::seq_edge(s, (int)n + 1);
            mark((int)n, b, e);
        }
        if (__any(b - t0 >= C)) break;
        base += WAVE;
        const int at = __builtin_amdgcn_readlane(e, WAVE - 1);
        if (at == __builtin_amdgcn_readlane(b, WAVE - 1)) base = ends_behind(s, (int)base, at, lane);
    }
}

// States of empty sequences: to[n] = from[n] (zeros where from is nullptr) for
// those of 64 sequences that have no token.
__device__ __forceinline__ void empty_states(const gdr::SeqArgs &s, int64_t group, int D, const float *from, float *to,
                                             int threads)
{
    const int64_t n = group * WAVE + threadIdx.x % WAVE;
    const bool empty = n < s.n_seqs && gdr::seq_edge(s, (int)n + 1) <= gdr::seq_edge(s, (int)n);
    for (uint64_t left = __ballot(empty); left; left &= left - 1) {
        const int64_t row = (group * WAVE + __builtin_ctzll(left)) * D;
        for (int c = threadIdx.x; c < D; c += threads) to[row + c] = from ? from[row + c] : 0.f;
    }
}

// the forms with pairs of channels that are reached (pairs_fit)
template <typename T, bool GATED> constexpr bool kPairs = sizeof(T) == 2 || !GATED;

// the near polynomial does for every channel of the wave
template <int V> __device__ __forceinline__ bool all_near(const float *neg_rate)
{
    bool near = true;
#pragma unroll
    for (int j = 0; j < V; ++j) near = near && neg_rate[j] >= -kNear;
    return __all(near);
}

// What a tile behind the last sequence stores for the tiles that come to it:
// every tile but the chain's last stores a map whatever the table of sequences
// says, so no wait hangs on what the table says to whom.
template <int V> __device__ __forceinline__ void put_nothing(uint64_t *p, bool active)
{
    if (threadIdx.x >= WAVE || !active) return;
#pragma unroll
    for (int j = 0; j < V; ++j) put(p + j * kLanes, Map{kForget, 0.f});
}

// tokens that sequences have: [0, total)
__device__ __forceinline__ int total_tokens(const gdr::SeqArgs &s)
{
    return s.cu_seqlens ? gdr::seq_edge(s, s.n_seqs) : s.n_tokens;
}

}  // namespace glr
