// Gated linear recurrence, forward: one thread per (sequence, channel), token
// after token.
#include "glr_device.h"

namespace glr {
namespace {

constexpr int NT = 64;

template <typename T, bool GATED>
__global__ __launch_bounds__(NT) void glr_scan_kernel(Args a)
{
    const int c = blockIdx.x * NT + threadIdx.x, D = a.D;
    if (c >= D) return;
    const gdr::SeqArgs sa = seq_args(a);
    const T *x = static_cast<const T *>(a.x), *rp = static_cast<const T *>(a.r), *ip = static_cast<const T *>(a.i);
    T *out = static_cast<T *>(a.h);
    for (int n = blockIdx.y; n < a.n_seqs; n += gridDim.y) {
        const gdr::Seq s = gdr::seq_of(sa, n);
        float h = a.h0 ? a.h0[(int64_t)n * D + c] : 0.f;
        const float nr = GATED && s.len ? -a.rate[c] : 0.f;
        for (int t = s.bos; t < s.bos + s.len; ++t) {
            const int64_t at = (int64_t)t * D + c;
            if (a.kept && t % kKept == 0) a.kept[(int64_t)(t / kKept) * D + c] = h;
            const float xv = kda::Elem<T>::ld(x + at);
            if (GATED) {
                const Gates gt = gates(kda::Elem<T>::ld(rp + at), kda::Elem<T>::ld(ip + at), nr);
                h = __builtin_fmaf(gt.a, h, gt.b * xv);
            } else
                h = __builtin_fmaf(decay(a.g[at]), h, xv);
            if (out) kda::Elem<T>::st(out + at, h);
        }
        if (a.h_T) a.h_T[(int64_t)n * D + c] = h;
    }
}

template <typename T>
void launch_t(const Args &a)
{
    const dim3 grid((a.D + NT - 1) / NT, a.n_seqs < 65535 ? a.n_seqs : 65535);
    if (a.gated) hipLaunchKernelGGL((glr_scan_kernel<T, true>), grid, dim3(NT), 0, a.stream, a);
    else hipLaunchKernelGGL((glr_scan_kernel<T, false>), grid, dim3(NT), 0, a.stream, a);
}

}  // namespace

size_t fwd_workspace(int64_t, int32_t) { return 0; }

hipError_t launch_fwd(const Args &a)
{
    if (a.bf16) launch_t<bf16>(a);
    else launch_t<float>(a);
    return hipGetLastError();
}

}  // namespace glr
