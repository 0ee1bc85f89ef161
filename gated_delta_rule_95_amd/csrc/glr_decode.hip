// Gated linear recurrence, decode: one token of each request, the state
// updated in place in a pool.  A thread has V neighbouring channels of one
// request, a workgroup part of a request's row: inputs and states are read
// once and written once.  256 requests of 8192 channels, gated, bf16: 33.6 MB
// in 7.4 us (4.5 TB/s, launch included); one request of 4096: 2.6 us, its
// latency.  (With 64 or 256 threads a workgroup 7.9 us, one channel a thread
// 8.4.)
#include "glr_tiles.h"

namespace glr {
namespace {

constexpr int NT = 128;

template <typename T, bool GATED, int V>
__global__ __launch_bounds__(NT) void glr_decode_kernel(DecodeArgs a)
{
    typedef Row<T, V> R;
    typedef Row<float, V> RF;
    const int c = (blockIdx.x * NT + threadIdx.x) * V, D = a.D;
    if (c >= D) return;
    for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
        const int slot = a.slots ? a.slots[n] : n;
        const int64_t at = (int64_t)n * D + c;
        float h[V] = {};
        if (slot >= 0 && slot < a.n_slots) {
            float *S = a.S + (int64_t)slot * D + c;
            const typename R::raw x = ld<V>(static_cast<const T *>(a.x) + at);
            const typename RF::raw s = ld<V>(S);
            if constexpr (GATED) {
                const typename R::raw r = ld<V>(static_cast<const T *>(a.r) + at), i = ld<V>(static_cast<const T *>(a.i) + at);
                const typename RF::raw rate = ld<V>(a.rate + c);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const Gates g = gates<false>(R::get(r, j), R::get(i, j), -RF::get(rate, j));
                    h[j] = __builtin_fmaf(g.a, RF::get(s, j), g.b * R::get(x, j));
                }
            } else {
                const typename RF::raw g = ld<V>(a.g + at);
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = __builtin_fmaf(decay(RF::get(g, j)), RF::get(s, j), R::get(x, j));
            }
            st<V>(S, h);
        }
        st<V>(static_cast<T *>(a.h) + at, h);
    }
}

template <typename T, bool GATED, int V>
void launch_v(const DecodeArgs &a)
{
    const dim3 grid((a.D + NT * V - 1) / (NT * V), a.N < 65535 ? a.N : 65535);
    hipLaunchKernelGGL((glr_decode_kernel<T, GATED, V>), grid, dim3(NT), 0, a.stream, a);
}

template <typename T, bool GATED>
void launch_t(const DecodeArgs &a)
{
    // four channels a thread where every row of every tensor starts on four
    const uintptr_t in = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) |
                         reinterpret_cast<uintptr_t>(a.i) | reinterpret_cast<uintptr_t>(a.h);
    const uintptr_t st = reinterpret_cast<uintptr_t>(a.g) | reinterpret_cast<uintptr_t>(a.rate) | reinterpret_cast<uintptr_t>(a.S);
    if (a.D % 4 == 0 && in % (4 * sizeof(T)) == 0 && st % 16 == 0) launch_v<T, GATED, 4>(a);
    else launch_v<T, GATED, 1>(a);
}

}  // namespace

hipError_t launch_decode(const DecodeArgs &a)
{
    if (a.bf16) a.gated ? launch_t<bf16, true>(a) : launch_t<bf16, false>(a);
    else a.gated ? launch_t<float, true>(a) : launch_t<float, false>(a);
    return hipGetLastError();
}

}  // namespace glr
