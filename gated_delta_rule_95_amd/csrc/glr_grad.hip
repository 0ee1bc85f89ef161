// Gated linear recurrence, backward.
//
// The forward's tiles the other way round: 64 tokens by 64 V channels, each of
// eight waves eight tokens in registers.  Two maps come out of a wave: of the
// state, forwards, which starts from the state that the forward kept before
// the tile, and of the cotangent M_t = a_t L_t, L_t = dh_t + M_{t+1},
// backwards, which is chained from tile to tile as the forward's state is.
// Then every wave runs its tokens up once more for a_t h_{t-1} and down once
// for L_t and the gradients.  Inputs are read once and gradients written
// once; the rate's gradient, a sum over all tokens, goes through one row a
// tile, summed up in order by a second launch.
#include "glr_tiles.h"

namespace glr {
namespace {

constexpr int NW = 8, K = 8, C = NW * K, NT = NW * WAVE;
static_assert(C == kKept, "a tile starts from a kept state");

template <typename T, bool GATED, int V>
__global__ __launch_bounds__(NT) void glr_grad_kernel(Args a, Chain chain, float *part)
{
    typedef Row<T, V> R;
    typedef Row<float, V> RF;
    __shared__ int s_idx, s_first[C], s_last[C];
    __shared__ Map s_up[NW][WAVE * V], s_down[NW][WAVE * V];
    __shared__ float s_in[WAVE * V];
    const int tid = threadIdx.x, lane = tid % WAVE, w = __builtin_amdgcn_readfirstlane(tid / WAVE), D = a.D;
    const gdr::SeqArgs sa = seq_args(a);
    if (tid == 0) s_idx = chain.ticket ? (int)atomicAdd(chain.ticket, 1u) : (int)blockIdx.x;
    if (tid < C) s_first[tid] = s_last[tid] = -1;
    const int total = total_tokens(sa);
    __syncthreads();
    const int idx = __builtin_amdgcn_readfirstlane(s_idx);
    if (idx >= chain.tiles * chain.blocks) {
        empty_states(sa, idx - chain.tiles * chain.blocks, D, a.dh_T, a.dh0, NT);
        return;
    }
    const int order = idx / chain.blocks, tile = chain.tiles - 1 - order, t0 = tile * C;
    if (t0 >= total) return;
    const int count = total - t0 < C ? total - t0 : C;
    const int c = (idx - order * chain.blocks) * WAVE * V + lane * V;
    const bool active = c < D;
    const int cc = active ? c : 0;
    const int tw = t0 + w * K, mine = count - w * K < 0 ? 0 : count - w * K < K ? count - w * K : K;

    typename R::raw rx[K], rr[K], ri[K], rd[K];
    typename RF::raw rg[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t row = (int64_t)(k < mine ? tw + k : t0) * D;
        rx[k] = R::ld(static_cast<const T *>(a.x) + row + cc);
        if constexpr (GATED) {
            rr[k] = R::ld(static_cast<const T *>(a.r) + row + cc);
            ri[k] = R::ld(static_cast<const T *>(a.i) + row + cc);
        } else
            rg[k] = RF::ld(a.g + row + cc);
        rd[k] = R::ld(static_cast<const T *>(a.dh) + row + cc);
    }
    float nr[V], h[V];
    if constexpr (GATED) {
        const typename RF::raw rate = RF::ld(a.rate + cc);
#pragma unroll
        for (int j = 0; j < V; ++j) nr[j] = -RF::get(rate, j);
    }
    const typename RF::raw left = RF::ld(a.kept + (int64_t)tile * D + cc);
    if (w == 0) mark_borders(sa, t0, C, lane, s_first, s_last);
    __syncthreads();
    const uint64_t starts = __ballot(lane < K && s_first[w * K + lane % K] >= 0);
    const uint64_t ends = __ballot(lane < K && s_last[w * K + lane % K] >= 0);
    const bool plain = starts == 0 && ends == 0 && mine == K;

    // u: the token's input; gated, of h's derivatives: b by x, e by i over L,
    // and with w = a h_{t-1}: (w - cx) q by r, (w - cx) s by -rate
    float al[K][V], u[K][V], d[K][V], b[K][V], e[K][V], cx[K][V], q[K][V], s[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float x = R::get(rx[k], j);
            d[k][j] = R::get(rd[k], j);
            if constexpr (GATED) {
                const GateGrads g = gate_grads(R::get(rr[k], j), R::get(ri[k], j), nr[j]);
                al[k][j] = g.a;
                b[k][j] = g.b;
                u[k][j] = g.b * x;
                e[k][j] = u[k][j] * g.rest_i;
                cx[k][j] = g.c * x;
                q[k][j] = g.q;
                s[k][j] = g.s_r;
            } else {
                al[k][j] = decay(RF::get(rg[k], j));
                u[k][j] = x;
            }
        }
    Map up[V], down[V];
#pragma unroll
    for (int j = 0; j < V; ++j) up[j] = down[j] = Map{1.f, 0.f};
    // a start's input holds what comes of the state before the sequence, a
    // last token's cotangent what comes of the state behind it
    if (!plain) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k < mine) {
                if (a.dh_T && (ends >> k & 1)) {
                    const int n = __builtin_amdgcn_readfirstlane(s_last[w * K + k]);
                    const typename RF::raw t = RF::ld(a.dh_T + (int64_t)n * D + cc);
#pragma unroll
                    for (int j = 0; j < V; ++j) d[k][j] += RF::get(t, j);
                }
                const bool start = starts >> k & 1;
                float h0[V] = {};
                if (start && a.h0) {
                    const int n = __builtin_amdgcn_readfirstlane(s_first[w * K + k]);
                    const typename RF::raw t = RF::ld(a.h0 + (int64_t)n * D + cc);
#pragma unroll
                    for (int j = 0; j < V; ++j) h0[j] = RF::get(t, j);
                }
#pragma unroll
                for (int j = 0; j < V; ++j)
                    up[j] = start ? Map{kForget, __builtin_fmaf(al[k][j], h0[j], u[k][j])}
                                  : Map{up[j].A * al[k][j], __builtin_fmaf(al[k][j], up[j].B, u[k][j])};
            }
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k)
            if (k < mine) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    down[j] = starts >> k & 1 ? Map{kForget, 0.f}
                                              : Map{down[j].A * al[k][j], al[k][j] * (d[k][j] + down[j].B)};
            }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) up[j] = Map{up[j].A * al[k][j], __builtin_fmaf(al[k][j], up[j].B, u[k][j])};
#pragma unroll
        for (int k = K - 1; k >= 0; --k)
#pragma unroll
            for (int j = 0; j < V; ++j) down[j].B = al[k][j] * (d[k][j] + down[j].B);
#pragma unroll
        for (int j = 0; j < V; ++j) down[j].A = up[j].A;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s_up[w][lane * V + j] = up[j];
        s_down[w][lane * V + j] = down[j];
    }
    __syncthreads();

    if (w == 0) {
        Map m[V];
        float in[V];
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = s_down[NW - 1][lane * V + j];
#pragma unroll
        for (int i = NW - 2; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = after(s_down[i][lane * V + j], m[j]);
        const bool more = chain.ticket && tile > 0;
        const bool alone = t0 + C >= total || s_last[C - 1] >= 0;
        uint64_t *p = chain.words + (int64_t)tile * D + cc;
        if (alone) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                in[j] = 0.f;
                if (more && active) put(p + j, Map{kForget, m[j].B});
            }
        } else {
            if (more && active)
#pragma unroll
                for (int j = 0; j < V; ++j) put(p + j, m[j]);
            look_back<V>(p + D, D, (total - 1) / C - tile, active, in);
            if (more && active)
#pragma unroll
                for (int j = 0; j < V; ++j) put(p + j, Map{kForget, m[j](in[j])});
        }
#pragma unroll
        for (int j = 0; j < V; ++j) s_in[lane * V + j] = in[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        h[j] = RF::get(left, j);
        for (int i = 0; i < w; ++i) h[j] = s_up[i][lane * V + j](h[j]);
    }
    // cx becomes w - cx (plain: w)
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (starts >> k & 1) {
            typename RF::raw t{};
            if (a.h0) {
                const int n = __builtin_amdgcn_readfirstlane(s_first[w * K + k]);
                t = RF::ld(a.h0 + (int64_t)n * D + cc);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = RF::get(t, j);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float ah = al[k][j] * h[j];
            h[j] = ah + u[k][j];
            cx[k][j] = GATED ? ah - cx[k][j] : ah;
        }
    }
    __syncthreads();

    float M[V], rate[V] = {};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        M[j] = s_in[lane * V + j];
        for (int i = NW - 1; i > w; --i) M[j] = s_down[i][lane * V + j](M[j]);
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        if (k >= mine) continue;
        const int64_t at = (int64_t)(tw + k) * D + c;
        float L[V], dr[V], di[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            L[j] = d[k][j] + M[j];
            M[j] = al[k][j] * L[j];
            if constexpr (GATED) {
                const float dg = L[j] * cx[k][j];
                dr[j] = dg * q[k][j];
                rate[j] = __builtin_fmaf(-dg, s[k][j], rate[j]);
                di[j] = L[j] * e[k][j];
                L[j] *= b[k][j];
            } else
                dr[j] = L[j] * cx[k][j];
        }
        if (active) {
            R::st(static_cast<T *>(a.dx) + at, L);
            if constexpr (GATED) {
                R::st(static_cast<T *>(a.dr) + at, dr);
                R::st(static_cast<T *>(a.di) + at, di);
            } else
                RF::st(a.dg + at, dr);
        }
        if (starts >> k & 1) {
            if (a.dh0 && active) {
                const int n = __builtin_amdgcn_readfirstlane(s_first[w * K + k]);
                RF::st(a.dh0 + (int64_t)n * D + c, M);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) M[j] = 0.f;
        }
    }
    if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < V; ++j) s_up[w][lane * V + j].B = rate[j];
        __syncthreads();
        if (w == 0 && active) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                for (int i = 1; i < NW; ++i) rate[j] += s_up[i][lane * V + j].B;
            RF::st(part + (int64_t)tile * D + c, rate);
        }
    }
}

// drate: the tiles' rows, each wave every 16th of them, in 64 bits
constexpr int RW = 16;
__global__ __launch_bounds__(RW * WAVE) void glr_rate_kernel(Args a, const float *part)
{
    __shared__ double s_sum[RW][WAVE];
    const int lane = threadIdx.x % WAVE, w = threadIdx.x / WAVE, c = blockIdx.x * WAVE + lane;
    const int tiles = (total_tokens(seq_args(a)) + C - 1) / C;
    double sum = 0;
    if (c < a.D)
        for (int t = w; t < tiles; t += RW) sum += (double)part[(int64_t)t * a.D + c];
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w == 0 && c < a.D) {
        for (int i = 1; i < RW; ++i) sum += s_sum[i][lane];
        a.drate[c] = (float)sum;
    }
}

int64_t tiles_of(int64_t n_tokens) { return (n_tokens + C - 1) / C; }
size_t rows_bytes(int64_t n_tokens, int32_t D)          // one fp32 row a tile
{
    return ((size_t)tiles_of(n_tokens) * D * 4 + 255) & ~(size_t)255;
}

template <typename T, bool GATED>
void launch_v(const Args &a, const Chain &ch, float *part, int64_t groups, int V, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)ch.tiles * ch.blocks + groups));
    if (V == 2) hipLaunchKernelGGL((glr_grad_kernel<T, GATED, 2>), grid, dim3(NT), 0, s, a, ch, part);
    else hipLaunchKernelGGL((glr_grad_kernel<T, GATED, 1>), grid, dim3(NT), 0, s, a, ch, part);
}

}  // namespace

// kept states (where they are formed again), the tiles' shares of drate, the
// chain (the forward's first, which is never longer)
size_t bwd_workspace(int64_t n_tokens, int32_t D)
{
    return 2 * rows_bytes(n_tokens, D) + chain_bytes(tiles_of(n_tokens), D);
}

hipError_t launch_bwd(const Args &arg)
{
    Args a = arg;
    const size_t rows = rows_bytes(a.n_tokens, a.D);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + rows);
    void *chain = static_cast<char *>(a.ws) + 2 * rows;
    hipError_t e;
    if (!a.kept && a.n_tokens) {
        a.kept = static_cast<float *>(a.ws);
        Args f = a;
        f.h = nullptr;
        f.h_T = nullptr;
        f.ws = chain;
        if ((e = launch_fwd(f)) != hipSuccess) return e;
    }
    const int V = pairs(a) ? 2 : 1;
    const Chain ch = make_chain(chain, (int)tiles_of(a.n_tokens), (a.D + WAVE * V - 1) / (WAVE * V));
    const int64_t groups = empty_groups(a, a.dh0);
    if ((int64_t)ch.tiles * ch.blocks + groups) {
        if ((e = clear_chain(ch, a.D, a.stream)) != hipSuccess) return e;
        if (a.bf16) a.gated ? launch_v<bf16, true>(a, ch, part, groups, V, a.stream) : launch_v<bf16, false>(a, ch, part, groups, V, a.stream);
        else a.gated ? launch_v<float, true>(a, ch, part, groups, V, a.stream) : launch_v<float, false>(a, ch, part, groups, V, a.stream);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.gated) {
        hipLaunchKernelGGL(glr_rate_kernel, dim3((unsigned)((a.D + WAVE - 1) / WAVE)), dim3(RW * WAVE), 0, a.stream, a, part);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace glr
