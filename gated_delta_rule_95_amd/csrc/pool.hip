// Pools of states: slots taken, freed and moved on the device.
//
// One workgroup plans (the free slots' ranks and the rows' ranks are running
// counts over at most 2^24 bytes), and a second launch moves the bytes.  A plan
// of 1000 slots takes 3 us, the latency of its loads and counts; copies are
// bound by HBM (32 copies of 8 slots of 4 MB: 168 MB in 28.6 us, 5.9 TB/s).
#include "kda_device.h"
#include "pool_launch.h"

namespace pool {
namespace {

constexpr int PT = 1024;                 // threads of a plan
constexpr int CT = 256;                  // threads that copy
constexpr int kPools = 32;               // pools a launch
constexpr int kPiece = 16 * 4 * CT;      // bytes of a row that one workgroup moves at a time

// Exclusive rank of `x` among the workgroup's threads in order, and the
// total.  All threads call it; `s` holds PT / 64 + 1 counts.
__device__ __forceinline__ int rank_of(bool x, int *s, int &total)
{
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
    total = all;
    return before + __popcll(b & (((uint64_t)1 << lane) - 1));
}

__device__ __forceinline__ bool valid(const uint8_t *used, int n_slots, const int32_t *src, int i)
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
__global__ __launch_bounds__(PT) void pool_take_kernel(uint8_t *used, int n_slots, const int32_t *src, int n,
                                                       int32_t *dst)
{
    __shared__ int s[PT / 64];
    int nfree = 0, total;
    for (int base = 0; base < n_slots && nfree < n; base += PT) {
        const int j = base + threadIdx.x;
        const bool f = j < n_slots && !used[j];
        const int k = nfree + rank_of(f, s, total);
        if (f && k < n) dst[k] = j;
        nfree += total;
    }
    int before = 0;
    for (int base = 0; base < n; base += PT) {
        const int i = base + threadIdx.x;
        rank_of(i < n && valid(used, n_slots, src, i), s, total);
        before += total;
    }
    __syncthreads();
    for (int base = (n - 1) / PT * PT; base >= 0; base -= PT) {
        const int i = base + threadIdx.x;
        const bool v = i < n && valid(used, n_slots, src, i);
        int k = rank_of(v, s, total);
        before -= total;
        k += before;
        const int to = v && k >= 0 && k < nfree ? dst[k] : -1;
        __syncthreads();
        if (i < n) dst[i] = to;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += PT) {
        const int j = dst[i];
        if (j >= 0 && j < n_slots) used[j] = 1;
    }
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
    int live = 0, total;
    for (int base = 0; base < n_slots; base += PT) {
        const int j = base + threadIdx.x;
        rank_of(j < n_slots && used[j], s, total);
        live += total;
    }
    int holes = 0, movers = 0;
    for (int base = 0; base < n_slots; base += PT) {
        const int j = base + threadIdx.x;
        const bool u = j < n_slots && used[j], hole = !u && j < live, mover = u && j >= live;
        const int kh = holes + rank_of(hole, s, total);
        holes += total;
        const int km = movers + rank_of(mover, s, total);
        movers += total;
        if (hole && kh < n_slots / 2) m.dst[kh] = j;
        if (mover && km < n_slots / 2) m.src[km] = j;
        if (j < n_slots) remap[j] = u ? j : -1;
    }
    // as many holes as movers, of n_slots in all
    movers = movers < n_slots / 2 ? movers : n_slots / 2;
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += PT) {
        const int j = m.src[k];
        if (j >= 0 && j < n_slots) remap[j] = m.dst[k];
    }
    for (int j = threadIdx.x; j < n_slots; j += PT) used[j] = j < live;
    if (threadIdx.x == 0) *m.count = movers;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n_table; i += PT) {
        const int j = table[i];
        if (j >= 0 && j < n_slots) table[i] = remap[j];
    }
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

// bytes (at most kPiece, a multiple of V's) from one row to another, or zeros.
// Whole pieces of 16-byte words are requested at once.  What is read may be
// read again (a fork's source by each of its copies: 32 copies of 8 slots of 4
// MB take 28.6 us, 42.2 with loads that bypass the caches), what is written is
// not.
template <typename V>
__device__ __forceinline__ void move_piece(const char *from, char *to, int bytes)
{
    const V *f = reinterpret_cast<const V *>(from);
    V *t = reinterpret_cast<V *>(to);
    constexpr int U = sizeof(V) == 16 ? kPiece / (16 * CT) : 1;
    if (U > 1 && bytes == kPiece) {
        V x[U] = {};
        if (from) {
#pragma unroll
            for (int k = 0; k < U; ++k) x[k] = f[threadIdx.x + k * CT];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) __builtin_nontemporal_store(x[k], t + threadIdx.x + k * CT);
        return;
    }
    for (int i = threadIdx.x; i < bytes / (int)sizeof(V); i += CT) t[i] = from ? f[i] : V{};
}

__global__ __launch_bounds__(CT) void pool_copy_kernel(CopyArgs a)
{
    const char *from = a.pool[blockIdx.y].from;
    char *to = a.pool[blockIdx.y].to;
    const size_t row = a.pool[blockIdx.y].row;
    const int64_t pieces = (row + kPiece - 1) / kPiece;
    int n = a.pairs.n;
    if (a.pairs.count) n = *a.pairs.count < n ? *a.pairs.count : n;
    const size_t odd = reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to) | row;
    for (int64_t unit = blockIdx.x; unit < n * pieces; unit += gridDim.x) {
        const int64_t i = unit / pieces, at = (unit - i * pieces) * kPiece;
        const int d = a.pairs.dst[i], f = from ? a.pairs.src[i] : 0;
        if (d < 0 || d >= a.pairs.to_slots || f < 0 || (from && f >= a.pairs.from_slots)) continue;
        const char *p = from ? from + (size_t)f * row + at : nullptr;
        char *q = to + (size_t)d * row + at;
        const int bytes = row - at < (size_t)kPiece ? (int)(row - at) : kPiece;
        if (odd % 16 == 0) move_piece<u32x4>(p, q, bytes);
        else if (odd % 4 == 0) move_piece<uint32_t>(p, q, bytes);
        else move_piece<uint8_t>(p, q, bytes);
    }
}

}  // namespace

hipError_t launch_copy(const pool_rows *from, const pool_rows *to, int32_t n_pools, const Pairs &pairs,
                       hipStream_t s)
{
    for (int first = 0; first < n_pools; first += kPools) {
        CopyArgs a{};
        a.pairs = pairs;
        int k = 0;
        int64_t units = 1;
        for (; k < kPools && first + k < n_pools; ++k) {
            const pool_rows &t = to[first + k];
            a.pool[k].from = from ? static_cast<const char *>(from[first + k].base) : nullptr;
            a.pool[k].to = static_cast<char *>(t.base);
            a.pool[k].row = t.row_bytes;
            const int64_t u = (int64_t)((t.row_bytes + kPiece - 1) / kPiece) * pairs.n;
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

hipError_t launch_take(uint8_t *used, int32_t n_slots, const int32_t *src, int32_t n, int32_t *dst, hipStream_t s)
{
    hipLaunchKernelGGL(pool_take_kernel, dim3(1), dim3(PT), 0, s, used, n_slots, src, n, dst);
    return hipGetLastError();
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
