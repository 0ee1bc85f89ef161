// Gated linear recurrence, backward: one thread per (sequence, channel); the
// states of 64 tokens formed again from the kept ones, then the tokens from
// the last to the first.
#include "glr_device.h"

namespace glr {
namespace {

constexpr int NT = 64;

template <typename T, bool GATED>
__global__ __launch_bounds__(NT) void glr_grad_kernel(Args a)
{
    const int c = blockIdx.x * NT + threadIdx.x, D = a.D;
    if (c >= D) return;
    const gdr::SeqArgs sa = seq_args(a);
    const T *x = static_cast<const T *>(a.x), *rp = static_cast<const T *>(a.r), *ip = static_cast<const T *>(a.i);
    const T *dh = static_cast<const T *>(a.dh);
    const float nr = GATED && a.n_tokens ? -a.rate[c] : 0.f;
    double drate = 0;
    for (int n = 0; n < a.n_seqs; ++n) {
        const gdr::Seq s = gdr::seq_of(sa, n);
        float M = a.dh_T ? a.dh_T[(int64_t)n * D + c] : 0.f;
        for (int end = s.bos + s.len; end > s.bos;) {
            const int first = (end - 1) / kKept * kKept;
            const int bos = first > s.bos ? first : s.bos;
            float h = bos > s.bos ? a.kept[(int64_t)(bos / kKept) * D + c] : a.h0 ? a.h0[(int64_t)n * D + c] : 0.f;
            float ah[kKept];
            for (int t = bos; t < end; ++t) {
                const int64_t at = (int64_t)t * D + c;
                const float xv = kda::Elem<T>::ld(x + at);
                float al, u = xv;
                if (GATED) {
                    const Gates gt = gates(kda::Elem<T>::ld(rp + at), kda::Elem<T>::ld(ip + at), nr);
                    al = gt.a;
                    u = gt.b * xv;
                } else
                    al = decay(a.g[at]);
                ah[t - bos] = al * h;
                h = ah[t - bos] + u;
            }
            for (int t = end - 1; t >= bos; --t) {
                const int64_t at = (int64_t)t * D + c;
                const float xv = kda::Elem<T>::ld(x + at), L = kda::Elem<T>::ld(dh + at) + M;
                if (GATED) {
                    const GateGrads q = gate_grads(kda::Elem<T>::ld(rp + at), kda::Elem<T>::ld(ip + at), nr);
                    const float dg = L * (ah[t - bos] - q.c * xv), dx = L * q.b;
                    kda::Elem<T>::st(static_cast<T *>(a.dx) + at, dx);
                    kda::Elem<T>::st(static_cast<T *>(a.di) + at, dx * xv * q.rest_i);
                    kda::Elem<T>::st(static_cast<T *>(a.dr) + at, dg * q.q);
                    drate -= (double)(dg * q.s_r);
                    M = q.a * L;
                } else {
                    kda::Elem<T>::st(static_cast<T *>(a.dx) + at, L);
                    a.dg[at] = L * ah[t - bos];
                    M = decay(a.g[at]) * L;
                }
            }
            end = bos;
        }
        if (a.dh0) a.dh0[(int64_t)n * D + c] = M;
    }
    if (GATED) a.drate[c] = (float)drate;
}

template <typename T>
void launch_t(const Args &a)
{
    const dim3 grid((a.D + NT - 1) / NT);
    if (a.gated) hipLaunchKernelGGL((glr_grad_kernel<T, true>), grid, dim3(NT), 0, a.stream, a);
    else hipLaunchKernelGGL((glr_grad_kernel<T, false>), grid, dim3(NT), 0, a.stream, a);
}

}  // namespace

static size_t kept_part(int64_t n_tokens, int32_t D)
{
    return ((size_t)((n_tokens + kKept - 1) / kKept) * D * 4 + 255) & ~(size_t)255;
}

size_t bwd_workspace(int64_t n_tokens, int32_t D)
{
    return kept_part(n_tokens, D) + fwd_workspace(n_tokens, D);
}

hipError_t launch_bwd(const Args &arg)
{
    Args a = arg;
    if (!a.kept && a.n_tokens) {
        a.kept = static_cast<float *>(a.ws);
        Args f = a;
        f.h = nullptr;
        f.h_T = nullptr;
        f.ws = static_cast<char *>(a.ws) + kept_part(a.n_tokens, a.D);
        const hipError_t e = launch_fwd(f);
        if (e != hipSuccess) return e;
    }
    if (a.bf16) launch_t<bf16>(a);
    else launch_t<float>(a);
    return hipGetLastError();
}

}  // namespace glr
