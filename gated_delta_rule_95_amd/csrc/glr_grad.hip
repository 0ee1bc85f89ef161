// Gated linear recurrence, backward.
//
// The forward's tiles the other way round: 64 tokens (gated, with pairs of
// channels: 32) by 64 V channels, eight tokens a wave in registers.  Two maps
// come out of a wave: of the state, forwards, which starts from the state that
// the forward kept before the tile, and of the cotangent M_t = a_t L_t, L_t =
// dh_t + M_{t+1}, backwards, which is chained from tile to tile as the
// forward's state is.  Then every wave runs its tokens up once more for a_t
// h_{t-1} and down once for L_t and the gradients.  Inputs are read once and
// gradients written once; the rate's gradient, a sum over all tokens, goes
// through one row a tile, summed up in order by a second launch.
//
// Plain, bf16, 20011 tokens of 4096 channels: 1.15 GB in 191 us, 6.0 TB/s.
// Gated, the same size: 1.15 GB in 256 us; a token and channel is 62 vector
// instructions (54% of the time) and eight numbers, which with two channels a lane
// take 149 registers once two of them are laid aside in the LDS: three
// workgroups of four waves a compute unit, whose phases overlap in part.  (Four
// tokens a wave, eight waves: 85 registers and two workgroups, 333 us; made to
// fit three, 297; then, three of four waves took 272.)
//
// A token at a border loads the state before it and the cotangent behind it
// where it wants them, twice each, and the second time behind its neighbours'
// stores: 20011 sequences of one token with states, gated, take 684 us for 2.1
// GB, twice what the bytes take.
#include "glr_tiles.h"

namespace glr {
namespace {

constexpr int K = kGradTokens;

template <typename T, bool GATED, int V>
__global__ __launch_bounds__(grad_waves(GATED, V) * WAVE) void glr_grad_kernel(Args a, Chain chain, float *part)
{
    constexpr int NW = grad_waves(GATED, V), C = grad_tile(GATED, V), NT = NW * WAVE;
    typedef Row<T, V> R;
    typedef Row<float, V> RF;
    __shared__ int s_tile, s_first[C], s_last[C];
    __shared__ Map s_up[NW - 1][WAVE * V], s_down[NW][WAVE * V];
    __shared__ float s_in[WAVE * V], s_late[GATED ? K : 1][2][V][NT];
    const int tid = threadIdx.x, lane = tid % WAVE, w = __builtin_amdgcn_readfirstlane(tid / WAVE), D = a.D;
    const gdr::SeqArgs sa = seq_args(a);
    const int total = total_tokens(sa);
    const int idx = blockIdx.x;
    if (idx >= chain.tiles * chain.blocks) {
        empty_states(sa, idx - chain.tiles * chain.blocks, D, a.dh_T, a.dh0, NT);
        return;
    }
    const int block = block_of(chain, idx);
    if (tid == 0) s_tile = take(chain, block);
    const Edges few = few_edges(sa, lane);
    if (tid < C) s_first[tid] = s_last[tid] = -1;
    __syncthreads();
    const int taken = __builtin_amdgcn_readfirstlane(s_tile);
    const int tile = chain.tiles - 1 - taken, t0 = tile * C, c = block * WAVE * V + lane * V;
    const bool active = c < D;
    const int cc = active ? c : 0;
    uint64_t *const p = chain.words + (int64_t)tile * chain.pitch + block * (WAVE * V) + lane;
    const bool more = tile > 0;
    if (t0 >= total) {
        if (more) put_nothing<V>(p, active);
        return;
    }
    const int count = total - t0 < C ? total - t0 : C;
    const int tw = t0 + w * K, mine = count - w * K < 0 ? 0 : count - w * K < K ? count - w * K : K;

    const unsigned ct = active ? c * (unsigned)sizeof(T) : kNowhere, cf = active ? c * 4u : kNowhere;
    const Rows<T, V> bx(a.x, tw, mine, D), br(a.r, tw, GATED ? mine : 0, D), bi(a.i, tw, GATED ? mine : 0, D),
        bdh(a.dh, tw, mine, D);
    const Rows<float, V> bg(a.g, tw, GATED ? 0 : mine, D);

    typename R::raw rx[K], rr[K], ri[K], rd[K];
    typename RF::raw rg[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        rx[k] = bx.ld(k, ct);
        if constexpr (GATED) {
            rr[k] = br.ld(k, ct);
            ri[k] = bi.ld(k, ct);
        } else
            rg[k] = bg.ld(k, cf);
        rd[k] = bdh.ld(k, ct);
    }
    float nr[V], h[V];
    if constexpr (GATED) {
        const typename RF::raw rate = ld<V>(a.rate + cc);
#pragma unroll
        for (int j = 0; j < V; ++j) nr[j] = -RF::get(rate, j);
    }
    const typename RF::raw left = ld<V>(a.kept + (int64_t)(t0 / kKept) * D + cc);
    if (w == 0) mark_borders(Lane{lane}, sa, [&](int) { return few; }, t0, C, s_first, s_last);
    __syncthreads();
    const uint64_t starts = __ballot(lane < K && s_first[w * K + lane % K] >= 0);
    const uint64_t ends = __ballot(lane < K && s_last[w * K + lane % K] >= 0);
    const bool plain = starts == 0 && ends == 0 && mine == K;

    // u: the token's input; gated, of h's derivatives: b by x, e by i over L,
    // and with w = a h_{t-1}: (w - cx) q by r, (w - cx) s by -rate
    float al[K][V], u[K][V], b[K][V], cx[K][V], s[K][V];
    const auto form = [&](auto near) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float x = R::get(rx[k], j);
                if constexpr (GATED) {
                    const GateGrads g = gate_grads<decltype(near)::value>(R::get(rr[k], j), R::get(ri[k], j), nr[j]);
                    al[k][j] = g.a;
                    b[k][j] = g.b;
                    u[k][j] = g.b * x;
                    s_late[k][0][j][tid] = u[k][j] * g.rest_i;
                    cx[k][j] = g.c * x;
                    s_late[k][1][j][tid] = g.q;
                    s[k][j] = g.s_r;
                } else {
                    al[k][j] = decay(RF::get(rg[k], j));
                    u[k][j] = x;
                }
            }
    };
    if (GATED && all_near<V>(nr)) form(std::true_type{});
    else form(std::false_type{});
    Map up[V], down[V];
#pragma unroll
    for (int j = 0; j < V; ++j) up[j] = down[j] = Map{1.f, 0.f};
    // what comes into a sequence's last token from behind is dh_T (0 without
    // one), what leaves its first token goes to dh0 and no further
    const auto behind = [&](int k, float *M) {
        typename RF::raw t{};
        if (a.dh_T) {
            const int n = __builtin_amdgcn_readfirstlane(s_last[w * K + k]);
            t = ld<V>(a.dh_T + (int64_t)n * D + cc);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) M[j] = RF::get(t, j);
    };
    const auto before = [&](int k, float *H) {
        typename RF::raw t{};
        if (a.h0) {
            const int n = __builtin_amdgcn_readfirstlane(s_first[w * K + k]);
            t = ld<V>(a.h0 + (int64_t)n * D + cc);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) H[j] = RF::get(t, j);
    };
    if (!plain) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k >= mine) continue;
            if (starts >> k & 1) {
                float H[V];
                before(k, H);
#pragma unroll
                for (int j = 0; j < V; ++j) up[j] = Map{kForget, H[j]};
            }
#pragma unroll
            for (int j = 0; j < V; ++j) up[j] = Map{up[j].A * al[k][j], __builtin_fmaf(al[k][j], up[j].B, u[k][j])};
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            if (k >= mine) continue;
            if (ends >> k & 1) {
                float M[V];
                behind(k, M);
#pragma unroll
                for (int j = 0; j < V; ++j) down[j] = Map{kForget, M[j]};
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
                down[j] = starts >> k & 1 ? Map{kForget, 0.f}
                                          : Map{down[j].A * al[k][j], al[k][j] * (R::get(rd[k], j) + down[j].B)};
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) up[j] = Map{up[j].A * al[k][j], __builtin_fmaf(al[k][j], up[j].B, u[k][j])};
#pragma unroll
        for (int k = K - 1; k >= 0; --k)
#pragma unroll
            for (int j = 0; j < V; ++j) down[j].B = al[k][j] * (R::get(rd[k], j) + down[j].B);
#pragma unroll
        for (int j = 0; j < V; ++j) down[j].A = up[j].A;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (w < NW - 1) s_up[w][lane * V + j] = up[j];
        s_down[w][lane * V + j] = down[j];
    }
    __syncthreads();

    // the tile's map of the cotangent: wave 0 stores it for the tiles before
    // this one as soon as it is there
    const bool alone = t0 + C >= total || s_last[C - 1] >= 0;
    Map t[V];
    if (w == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = s_down[NW - 1][lane * V + j];
#pragma unroll
        for (int i = NW - 2; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < V; ++j) t[j] = after(s_down[i][lane * V + j], t[j]);
        if (more && active)
#pragma unroll
            for (int j = 0; j < V; ++j) put(p + j * kLanes, alone ? Map{kForget, t[j].B} : t[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        h[j] = RF::get(left, j);
        for (int i = 0; i < w; ++i) h[j] = s_up[i][lane * V + j](h[j]);
    }
    // cx becomes w - cx (plain: w).  (Here and below the waves without a border
    // have code of their own: a load in a branch would make every token wait
    // for the stores before it.)
    const auto ascend = [&](auto borders) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (decltype(borders)::value && (starts >> k & 1)) before(k, h);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float ah = al[k][j] * h[j];
                h[j] = ah + u[k][j];
                cx[k][j] = GATED ? ah - cx[k][j] : ah;
            }
        }
    };
    if (plain) ascend(std::false_type{});
    else ascend(std::true_type{});
    if (w == 0) {
        float in[V] = {};
        if (!alone) {
            look_back<8 / V, V>(p + chain.pitch, chain.pitch, chain.tiles - 1 - tile, active, in);
            if (more && active)
#pragma unroll
                for (int j = 0; j < V; ++j) put(p + j * kLanes, Map{kForget, t[j](in[j])});
        }
#pragma unroll
        for (int j = 0; j < V; ++j) s_in[lane * V + j] = in[j];
    }
    __syncthreads();

    const Rows<T, V> bdx(a.dx, tw, mine, D), bdr(a.dr, tw, GATED ? mine : 0, D), bdi(a.di, tw, GATED ? mine : 0, D);
    const Rows<float, V> bdg(a.dg, tw, GATED ? 0 : mine, D);
    float M[V], rate[V] = {};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        M[j] = s_in[lane * V + j];
        for (int i = NW - 1; i > w; --i) M[j] = s_down[i][lane * V + j](M[j]);
    }
    const auto descend = [&](auto borders) {
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            if (decltype(borders)::value && k >= mine) continue;
            if (decltype(borders)::value && (ends >> k & 1)) behind(k, M);
            float L[V], dr[V], di[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                L[j] = R::get(rd[k], j) + M[j];
                M[j] = al[k][j] * L[j];
                if constexpr (GATED) {
                    const float dg = L[j] * cx[k][j];
                    dr[j] = dg * s_late[k][1][j][tid];
                    rate[j] = __builtin_fmaf(-dg, s[k][j], rate[j]);
                    di[j] = L[j] * s_late[k][0][j][tid];
                    L[j] *= b[k][j];
                } else
                    dr[j] = L[j] * cx[k][j];
            }
            bdx.st(k, ct, L);
            if constexpr (GATED) {
                bdr.st(k, ct, dr);
                bdi.st(k, ct, di);
            } else
                bdg.st(k, cf, dr);
            if (decltype(borders)::value && (starts >> k & 1)) {
                if (a.dh0 && active) {
                    const int n = __builtin_amdgcn_readfirstlane(s_first[w * K + k]);
                    st<V>(a.dh0 + (int64_t)n * D + c, M);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) M[j] = 0.f;
            }
        }
    };
    if (plain) descend(std::false_type{});
    else descend(std::true_type{});
    if constexpr (GATED) {
        // a wave is done with what it laid aside, and all are with the maps of the state
        float (*s_rate)[WAVE * V] = reinterpret_cast<float (*)[WAVE * V]>(&s_up[0][0]);
        static_assert(sizeof(s_up) >= NW * WAVE * V * sizeof(float), "room for the rates");
#pragma unroll
        for (int j = 0; j < V; ++j) s_rate[w][lane * V + j] = rate[j];
        __syncthreads();
        if (w == 0 && active) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                for (int i = 1; i < NW; ++i) rate[j] += s_rate[i][lane * V + j];
            st<V>(part + (int64_t)tile * D + c, rate);
        }
    }
}

// drate: the tiles' rows, each wave every 16th of them, in 64 bits
constexpr int RW = 16;
__global__ __launch_bounds__(RW * WAVE) void glr_rate_kernel(Args a, const float *part, int C)
{
    __shared__ double s_sum[RW][WAVE];
    const int lane = threadIdx.x % WAVE, w = threadIdx.x / WAVE, c = blockIdx.x * WAVE + lane;
    const int tiles = (total_tokens(seq_args(a)) + C - 1) / C;
    double sum = 0;
    if (c < a.D)
#pragma unroll 8
        for (int t = w; t < tiles; t += RW) sum += (double)part[(int64_t)t * a.D + c];
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w == 0 && c < a.D) {
        for (int i = 1; i < RW; ++i) sum += s_sum[i][lane];
        a.drate[c] = (float)sum;
    }
}

template <typename T, bool GATED>
void launch_v(const Args &a, const Chain &ch, float *part, int V, hipStream_t s)
{
    const dim3 grid((unsigned)ch.items);
    if constexpr (kPairs<T, GATED>)
        if (V == 2) {
            hipLaunchKernelGGL((glr_grad_kernel<T, GATED, 2>), grid, dim3(grad_waves(GATED, 2) * WAVE), 0, s, a, ch, part);
            return;
        }
    hipLaunchKernelGGL((glr_grad_kernel<T, GATED, 1>), grid, dim3(grad_waves(GATED, 1) * WAVE), 0, s, a, ch, part);
}

}  // namespace

hipError_t launch_bwd(const Args &arg)
{
    Args a = arg;
    const GradParts w(a);
    hipError_t e;
    if (!a.kept && a.n_tokens) {
        a.kept = w.kept;
        Args f = a;
        f.h = nullptr;
        f.h_T = nullptr;
        f.ws = w.chain;
        if ((e = launch_fwd(f)) != hipSuccess) return e;
    }
    const Plan p = plan_grad(a, w.chain);
    if (p.chain.items) {
        if ((e = clear_chain(p.chain, a.stream)) != hipSuccess) return e;
        if (a.bf16)
            a.gated ? launch_v<bf16, true>(a, p.chain, w.part, p.V, a.stream)
                    : launch_v<bf16, false>(a, p.chain, w.part, p.V, a.stream);
        else
            a.gated ? launch_v<float, true>(a, p.chain, w.part, p.V, a.stream)
                    : launch_v<float, false>(a, p.chain, w.part, p.V, a.stream);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!a.gated) return hipSuccess;
    hipLaunchKernelGGL(glr_rate_kernel, dim3((unsigned)blocks_of(a.D, 1)), dim3(RW * WAVE), 0, a.stream, a, w.part,
                       grad_tile(true, p.V));
    return hipGetLastError();
}

}  // namespace glr
