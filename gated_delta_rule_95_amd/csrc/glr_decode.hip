// Gated linear recurrence, decode: one token of each request, the state
// updated in place in a pool.
#include "glr_device.h"

namespace glr {
namespace {

constexpr int NT = 256;

template <typename T, bool GATED>
__global__ __launch_bounds__(NT) void glr_decode_kernel(DecodeArgs a)
{
    const int c = blockIdx.x * NT + threadIdx.x, D = a.D;
    if (c >= D) return;
    for (int n = blockIdx.y; n < a.N; n += gridDim.y) {
        const int slot = a.slots ? a.slots[n] : n;
        const int64_t at = (int64_t)n * D + c;
        float h = 0.f;
        if (slot >= 0 && slot < a.n_slots) {
            float *S = a.S + (int64_t)slot * D + c;
            const float xv = kda::Elem<T>::ld(static_cast<const T *>(a.x) + at);
            if (GATED) {
                const Gates g = gates<false>(kda::Elem<T>::ld(static_cast<const T *>(a.r) + at),
                                      kda::Elem<T>::ld(static_cast<const T *>(a.i) + at), -a.rate[c]);
                h = __builtin_fmaf(g.a, *S, g.b * xv);
            } else
                h = __builtin_fmaf(decay(a.g[at]), *S, xv);
            *S = h;
        }
        kda::Elem<T>::st(static_cast<T *>(a.h) + at, h);
    }
}

template <typename T>
void launch_t(const DecodeArgs &a)
{
    const dim3 grid((a.D + NT - 1) / NT, a.N < 65535 ? a.N : 65535);
    if (a.gated) hipLaunchKernelGGL((glr_decode_kernel<T, true>), grid, dim3(NT), 0, a.stream, a);
    else hipLaunchKernelGGL((glr_decode_kernel<T, false>), grid, dim3(NT), 0, a.stream, a);
}

}  // namespace

hipError_t launch_decode(const DecodeArgs &a)
{
    if (a.bf16) launch_t<bf16>(a);
    else launch_t<float>(a);
    return hipGetLastError();
}

}  // namespace glr
