// Pools of states: slots taken, freed and moved on the device.
//
// One workgroup plans (the free slots' ranks and the rows' ranks are running
// counts over at most 2^24 bytes), and a second launch moves the bytes (of a
// few rows, the same).  A plan
// of 1000 slots takes 3.3 us, the latency of its loads and counts, which steps of
// 1024 slots add up (a fork in 2^20 slots 356 us, a compaction 2.8 ms, of which
// a table of 2^20 entries is 0.54); copies are bound by HBM (32 copies of 8 slots
// of 4 MB: 168 MB in 26.6 us, 6.3 TB/s), but for rows that 16 does not divide,
// whose words are requested one at a time (16 slots of 299 999 fp32 take 9.3 us,
// of 599 999 bf16, byte by byte, 22.8, of 300 000 fp32 6.1).
#include "kda_device.h"
#include "pool_index.h"
#include "pool_launch.h"

namespace pool {
namespace {

constexpr int PT = 1024;                 // threads of a plan
constexpr int CT = 256;                  // threads that copy
constexpr int kPools = 32;               // pools a launch
constexpr int kPiece = 64 * CT;      // bytes of a row that one workgroup moves at a time

// The block of pool_index.h: the workgroup, a thread each.  `s` holds PT / 64
// counts.
struct Group {
    static constexpr int threads = PT;
    int *s;
    template <typename T> struct Each {
        T x;
        __device__ __forceinline__ T &operator[](int) { return x; }
    };
    template <typename F> __device__ __forceinline__ void each(const F &f) const { f((int)threadIdx.x); }
    __device__ __forceinline__ void sync() const { __syncthreads(); }
    template <typename F, typename G> __device__ __forceinline__ int rank(const F &f, const G &g) const
    {
        const bool x = f((int)threadIdx.x);
        const uint64_t b = __ballot(x);
        const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
        __syncthreads();
        if (lane == 0) s[w] = __popcll(b);
        __syncthreads();
        int before = 0, all = 0;
        for (int i = 0; i < PT / 64; ++i) {
            if (i == w) before = all;
            all += s[i];
        }
        g((int)threadIdx.x, x, before + __popcll(b & (((uint64_t)1 << lane) - 1)), all);
        return all;
    }
};

__global__ __launch_bounds__(PT) void pool_take_kernel(uint8_t *used, int n_slots, const int32_t *src, int n,
                                                       int32_t *dst)
{
    __shared__ int s[PT / 64];
    take(Group{s}, used, n_slots, src, n, dst);
}

__global__ __launch_bounds__(CT) void pool_free_kernel(uint8_t *used, int n_slots, const int32_t *slots, int n)
{
    for (int i = blockIdx.x * CT + threadIdx.x; i < n; i += gridDim.x * CT) {
        const int j = slots[i];
        if (j >= 0 && j < n_slots) used[j] = 0;
    }
}

__global__ __launch_bounds__(PT) void pool_plan_kernel(uint8_t *used, int n_slots, int32_t *table, int64_t n_table,
                                                       int32_t *remap, Moves m)
{
    __shared__ int s[PT / 64];
    plan(Group{s}, used, n_slots, table, n_table, remap, m);
}

struct CopyArgs {
    Pairs pairs;
    struct {
        const char *from;
        char *to;
        size_t row;
    } pool[kPools];
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// bytes (at most 64 NT, a multiple of V's) from one row to another, or zeros, by
// NT threads.  Whole pieces of 16-byte words are requested at once.  What is read may be
// read again (a fork's source by each of its copies: 32 copies of 8 slots of 4
// MB take 28.6 us, 42.2 with loads that bypass the caches), what is written is
// not.
template <typename V, int NT>
__device__ __forceinline__ void move_words(const char *from, char *to, int bytes)
{
    const int tid = threadIdx.x % NT;
    const V *f = reinterpret_cast<const V *>(from);
    V *t = reinterpret_cast<V *>(to);
    constexpr int U = sizeof(V) == 16 ? 4 : 1;
    if (U > 1 && bytes == 64 * NT) {
        V x[U] = {};
        if (from) {
#pragma unroll
            for (int k = 0; k < U; ++k) x[k] = f[tid + k * NT];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) __builtin_nontemporal_store(x[k], t + tid + k * NT);
        return;
    }
    for (int i = tid; i < bytes / (int)sizeof(V); i += NT) t[i] = from ? f[i] : V{};
}
// piece `at` / (64 NT) of row f (of from; nullptr: zeros) to row d
template <int NT>
__device__ __forceinline__ void move_piece(const char *from, char *to, size_t row, int f, int d, size_t at)
{
    const size_t odd = reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to) | row;
    const char *p = from ? from + (size_t)f * row + at : nullptr;
    char *q = to + (size_t)d * row + at;
    const int bytes = row - at < (size_t)(64 * NT) ? (int)(row - at) : 64 * NT;
    if (odd % 16 == 0) move_words<u32x4, NT>(p, q, bytes);
    else if (odd % 4 == 0) move_words<uint32_t, NT>(p, q, bytes);
    else move_words<uint8_t, NT>(p, q, bytes);
}

__global__ __launch_bounds__(CT) void pool_copy_kernel(CopyArgs a)
{
    const char *from = a.pool[blockIdx.y].from;
    char *to = a.pool[blockIdx.y].to;
    const size_t row = a.pool[blockIdx.y].row;
    const int64_t pieces = (row + kPiece - 1) / kPiece;
    int n = a.pairs.n;
    if (a.pairs.count) n = *a.pairs.count < n ? *a.pairs.count : n;
    for (int64_t unit = blockIdx.x; unit < n * pieces; unit += gridDim.x) {
        const int64_t i = unit / pieces, at = (unit - i * pieces) * kPiece;
        const int d = a.pairs.dst[i], f = from ? a.pairs.src[i] : 0;
        if (d < 0 || d >= a.pairs.to_slots || f < 0 || (from && f >= a.pairs.from_slots)) continue;
        move_piece<CT>(from, to, row, f, d, at);
    }
}

// A fork or allocation of a few rows: the workgroup that plans it moves them
// too, a piece of 4 KB a wave, and a launch is saved.  A fork and a free, host
// included: 60 to 64 pieces 12 to 13.3 us, with a launch for the copies 15 to
// 16; 128 pieces of wide rows 14.6 and 14.8; 256 pieces 23.9 and 15.2.
constexpr size_t kHere = 64;             // pieces
constexpr int kWavePiece = 64 * 64;
__global__ __launch_bounds__(PT) void pool_take_copy_kernel(uint8_t *used, int n_slots, const int32_t *src, int n,
                                                            int32_t *dst, CopyArgs a, int pools)
{
    __shared__ int s[PT / 64];
    take(Group{s}, used, n_slots, src, n, dst);
    __syncthreads();
    constexpr int waves = PT / 64;
    int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    for (int k = 0; k < pools; ++k) {
        const size_t row = a.pool[k].row;
        const int pieces = (int)((row + kWavePiece - 1) / kWavePiece), units = n * pieces;
        for (; w < units; w += waves) {
            const int i = w / pieces, d = dst[i], f = src ? src[i] : 0;
            if (d < 0 || d >= n_slots || f < 0 || f >= n_slots) continue;
            move_piece<64>(a.pool[k].from, a.pool[k].to, row, f, d, (size_t)(w - i * pieces) * kWavePiece);
        }
        w -= units;
    }
}

}  // namespace

// pools [first ..] of a launch; how many
int copy_args(CopyArgs &a, const pool_rows *from, const pool_rows *to, int32_t n_pools, int first)
{
    int k = 0;
    for (; k < kPools && first + k < n_pools; ++k) {
        a.pool[k].from = from ? static_cast<const char *>(from[first + k].base) : nullptr;
        a.pool[k].to = static_cast<char *>(to[first + k].base);
        a.pool[k].row = to[first + k].row_bytes;
    }
    return k;
}

hipError_t launch_copy(const pool_rows *from, const pool_rows *to, int32_t n_pools, const Pairs &pairs,
                       hipStream_t s)
{
    for (int first = 0; first < n_pools; first += kPools) {
        CopyArgs a{};
        a.pairs = pairs;
        const int k = copy_args(a, from, to, n_pools, first);
        int64_t units = 1;
        for (int i = 0; i < k; ++i) {
            const int64_t u = (int64_t)((a.pool[i].row + kPiece - 1) / kPiece) * pairs.n;
            if (u > units) units = u;
        }
        // one piece a workgroup while that is a grid of ordinary size (with 2048 of
        // them that go round: 28.6 -> 37.5 us)
        const int64_t most = 65536 / k + 1;
        hipLaunchKernelGGL(pool_copy_kernel, dim3((unsigned)(units < most ? units : most), k), dim3(CT), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_take(const pool_rows *pools, int32_t n_pools, uint8_t *used, int32_t n_slots, const int32_t *src,
                       int32_t n, int32_t *dst, hipStream_t s)
{
    size_t pieces = 0;
    for (int i = 0; i < n_pools && pieces <= kHere; ++i)
        pieces += (pools[i].row_bytes + kWavePiece - 1) / kWavePiece * (size_t)n;        // (below 2^53 each)
    const bool move = n_pools && n_slots, here = move && n_pools <= kPools && pieces <= kHere;
    const pool_rows *from = src ? pools : nullptr;
    if (here) {
        CopyArgs a{};
        copy_args(a, from, pools, n_pools, 0);
        hipLaunchKernelGGL(pool_take_copy_kernel, dim3(1), dim3(PT), 0, s, used, n_slots, src, n, dst, a, n_pools);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(pool_take_kernel, dim3(1), dim3(PT), 0, s, used, n_slots, src, n, dst);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && move ? launch_copy(from, pools, n_pools, Pairs{src, dst, nullptr, n, n_slots, n_slots}, s) : e;
}

hipError_t launch_free(uint8_t *used, int32_t n_slots, const int32_t *slots, int32_t n, hipStream_t s)
{
    const int blocks = (n + CT - 1) / CT;
    hipLaunchKernelGGL(pool_free_kernel, dim3(blocks < 256 ? blocks : 256), dim3(CT), 0, s, used, n_slots, slots, n);
    return hipGetLastError();
}

hipError_t launch_plan(uint8_t *used, int32_t n_slots, int32_t *table, int64_t n_table, int32_t *remap,
                       const Moves &m, hipStream_t s)
{
    hipLaunchKernelGGL(pool_plan_kernel, dim3(1), dim3(PT), 0, s, used, n_slots, table, n_table, remap, m);
    return hipGetLastError();
}

}  // namespace pool
