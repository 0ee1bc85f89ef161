// What the scan and its gradients share on the device: rows of a tensor, tiles
// of tokens and channels handed out in order, and the lanes and words by which
// glr_index.h finds the borders in a tile and what comes into it (gfx950 only).
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

__device__ __forceinline__ void put(uint64_t *p, const Map &m)
{
    __hip_atomic_store(p, word_of(m), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The wave of glr_index.h as the device runs it, a lane each.
struct Lane {
    int lane;
    template <typename T> struct Each {
        T x;
        __device__ __forceinline__ T &operator[](int) { return x; }
    };
    template <typename F> __device__ __forceinline__ void each(const F &f) const { f(lane); }
    template <typename F> __device__ __forceinline__ int count(const F &f) const { return __popcll(__ballot(f(lane))); }
    template <typename F> __device__ __forceinline__ bool any(const F &f) const { return __any(f(lane)); }
    template <typename F> __device__ __forceinline__ bool all(const F &f) const { return __all(f(lane)); }
    template <typename F> __device__ __forceinline__ int last(const F &f) const
    {
        return __builtin_amdgcn_readlane(f(lane), WAVE - 1);
    }
    __device__ __forceinline__ void sleep() const { __builtin_amdgcn_s_sleep(1); }
};

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

// What comes into a tile (look, in glr_index.h): words of the `n` tiles before
// it lie `step` apart, from `p` on, the nearest first.
template <int W, int V>
__device__ __forceinline__ void look_back(const uint64_t *p, int64_t step, int n, bool active, float *in)
{
    Lane::Each<Values<V>> got{};
    look<W, V>(Lane{0}, [&](int, int i, int j) { return peek(p + step * i + j * kLanes); }, n, [&](int) { return active; }, got);
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = got.x.x[j];
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
