// Gated delta rule token by token in fp32: the forward, the forward that
// keeps states for the backward, and the reverse sweep.  Right for every
// type and head size.
//
// Columns of the state evolve independently, so a wave owns 16 columns and
// all rows of S in registers: lane (c, r) = (lane % 16, lane / 16) holds rows
// 16 t + 4 r + e of column c.  Per token the two column sums S'^T k and
// S'^T q are taken together (o = S'^T q + u (k . q)), each over a lane's own
// rows and then over the four row groups by two register swaps.
#include "gdr_device.h"

namespace gdr {
namespace {

constexpr int TT = 16;               // tokens staged at a time

enum { FWD = 0, KEEP = 1, SWEEP = 2 };

template <typename TI, int DK, int DV>
struct Shape {
    static constexpr int NW = DV / 16 < 4 ? DV / 16 : 4;
    static constexpr int NT = NW * WAVE;
    static constexpr int BV = 16 * NW;
};

// MODE FWD: writes o and S_T.  KEEP: the state before every token of index
// 0, C, 2C, ... of its sequence to Sc[slot], and R_t = v_t - S'^T k_t.
// SWEEP: from the last token to the first with the cotangent L of the state,
//     L += scale q_t dO_t^T;  Ub_t = L^T k_t;  L = exp(g_t) (L - k_t (beta_t Ub_t)^T),
// writing dv = beta Ub, Ub, L behind the last token of every chunk (Lc) and
// dS0.
template <typename TI, int DK, int DV, int MODE>
__global__ __launch_bounds__((Shape<TI, DK, DV>::NT))
void gdr_recurrent_kernel(Args a, int C)
{
    using Sh = Shape<TI, DK, DV>;
    using TO = typename OutOf<TI>::type;
    constexpr int RT = DK / 16;      // row tiles: four rows of each per lane
    constexpr int CB = DV / Sh::BV;
    __shared__ __align__(16) float s_k[TT][DK], s_q[TT][DK], s_v[TT][Sh::BV];
    __shared__ float s_a[TT], s_b[TT], s_kq[TT];
    const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
    const int c = lane % 16, r = lane / 16;
    const int64_t chain = blockIdx.x / CB;
    const int cb = blockIdx.x % CB;
    const int n = (int)(chain / a.Hv), hv = (int)(chain % a.Hv), hk = hv / (a.Hv / a.Hk);
    const Seq sq = seq_of(a.seq, n);
    const int col = cb * Sh::BV + 16 * wave + c;
    const auto Q = src<TI>(a.q, a.qe), K = src<TI>(a.k, a.ke), V = src<TI>(a.v, a.ve);
    const auto G = src<TO>(a.dO, nullptr);
    const int64_t st = (chain * DK) * DV + col;
    const float *init = MODE == SWEEP ? a.dS_T : a.S0;
    f32x4 S[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[t][e] = init ? init[st + (int64_t)(16 * t + 4 * r + e) * DV] : 0.f;

    const int tiles = (sq.len + TT - 1) / TT;
    for (int tile = 0; tile < tiles; ++tile) {
        const int t0 = (MODE == SWEEP ? tiles - 1 - tile : tile) * TT;
        const int nt = sq.len - t0 < TT ? sq.len - t0 : TT;
        __syncthreads();
        for (int i = tid; i < TT * DK / 4; i += Sh::NT) {
            const int t = i / (DK / 4), ch = 4 * (i % (DK / 4));
            f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qq = kk;
            if (t < nt) {
                const int64_t row = (int64_t)(sq.bos + t0 + t) * a.Hk + hk;
                kk = K.ld4(row, DK, ch);
                if (MODE != KEEP) qq = Q.ld4(row, DK, ch);
            }
            *reinterpret_cast<f32x4 *>(&s_k[t][ch]) = kk;
            *reinterpret_cast<f32x4 *>(&s_q[t][ch]) = qq;
        }
        for (int i = tid; i < TT * Sh::BV / 4; i += Sh::NT) {
            const int t = i / (Sh::BV / 4), x = 4 * (i % (Sh::BV / 4));
            f32x4 vv = {0.f, 0.f, 0.f, 0.f};
            if (t < nt) {
                const int64_t row = (int64_t)(sq.bos + t0 + t) * a.Hv + hv;
                if constexpr (MODE == SWEEP) vv = G.ld4(row, DV, cb * Sh::BV + x);
                else vv = V.ld4(row, DV, cb * Sh::BV + x);
            }
            *reinterpret_cast<f32x4 *>(&s_v[t][x]) = vv;
        }
        if (tid < TT) {
            const bool in = tid < nt;
            const int64_t row = (int64_t)(sq.bos + t0 + (in ? tid : 0)) * a.Hv + hv;
            s_a[tid] = in ? kda::fast_exp2(floor_g(a.g[row]) * LOG2E) : 1.f;
            s_b[tid] = in ? a.beta[row] : 0.f;
        }
        __syncthreads();
        if (MODE == FWD) {           // k . q of every token: 16 lanes a token
            for (int t = tid / 16; t < TT; t += Sh::NT / 16) {
                float x = 0.f;
                for (int i = tid % 16; i < DK; i += 16) x += s_k[t][i] * s_q[t][i];
#pragma unroll
                for (int m = 1; m < 16; m *= 2) x += __shfl_xor(x, m);
                if (tid % 16 == 0) s_kq[t] = x;
            }
            __syncthreads();
        }
        for (int i = 0; i < nt; ++i) {
            const int t = MODE == SWEEP ? nt - 1 - i : i;
            const int pos = t0 + t;
            const int64_t row = (int64_t)(sq.bos + pos) * a.Hv + hv;
            const float al = s_a[t], be = s_b[t], x = s_v[t][16 * wave + c];
            const int64_t slot = sq.bos / C + n + pos / C;
            const int64_t cst = ((slot * a.Hv + hv) * DK) * DV + col;
            if (MODE == KEEP && pos % C == 0) {
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a.Sc[cst + (int64_t)(16 * m + 4 * r + e) * DV] = S[m][e];
            }
            if (MODE == SWEEP && (pos % C == C - 1 || pos == sq.len - 1)) {
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a.Lc[cst + (int64_t)(16 * m + 4 * r + e) * DV] = S[m][e];
            }
            // four partial sums each: one would be a chain of d_k / 4 dependent adds
            f32x4 pk4 = {0.f, 0.f, 0.f, 0.f}, pq4 = pk4;
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                const f32x4 kk = *reinterpret_cast<const f32x4 *>(&s_k[t][16 * m + 4 * r]);
                const f32x4 qq = *reinterpret_cast<const f32x4 *>(&s_q[t][16 * m + 4 * r]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (MODE == SWEEP) S[m][e] += (a.scale * x) * qq[e];
                    else S[m][e] *= al;
                    pk4[e] += S[m][e] * kk[e];
                    if (MODE == FWD) pq4[e] += S[m][e] * qq[e];
                }
            }
            const float pk = sum_groups((pk4[0] + pk4[1]) + (pk4[2] + pk4[3]));
            float u;
            if (MODE == SWEEP) {
                u = -be * pk;
                if (r == 0) {
                    kda::Elem<TO>::st((TO *)a.dval + row * DV + col, be * pk);
                    a.Ub[row * DV + col] = pk;
                }
            } else {
                const float res = x - pk;
                u = be * res;
                if (MODE == KEEP && r == 0) a.R[row * DV + col] = res;
            }
            if (MODE == FWD) {
                const float pq = sum_groups((pq4[0] + pq4[1]) + (pq4[2] + pq4[3]));
                if (r == 0)
                    kda::Elem<TO>::st((TO *)a.o + row * DV + col, a.scale * (pq + u * s_kq[t]));
            }
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                const f32x4 kk = *reinterpret_cast<const f32x4 *>(&s_k[t][16 * m + 4 * r]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[m][e] += kk[e] * u;
                    if (MODE == SWEEP) S[m][e] *= al;
                }
            }
        }
    }
    float *out = MODE == FWD ? a.S_T : MODE == SWEEP ? a.dS0 : nullptr;
    if (out) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[st + (int64_t)(16 * t + 4 * r + e) * DV] = S[t][e];
    }
}

template <typename TI, int DK, int DV>
hipError_t launch_t(const Args &a, int mode, int C)
{
    using Sh = Shape<TI, DK, DV>;
    const int64_t blocks = (int64_t)a.seq.n_seqs * a.Hv * (DV / Sh::BV);
    if (blocks * Sh::NT >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    const dim3 grid((unsigned)blocks), block(Sh::NT);
    if (mode == FWD) {
        if constexpr (std::is_same<TI, e4m3>::value) return hipErrorInvalidValue;
        else hipLaunchKernelGGL((gdr_recurrent_kernel<TI, DK, DV, FWD>), grid, block, 0, a.stream, a, C);
    } else if (mode == KEEP)
        hipLaunchKernelGGL((gdr_recurrent_kernel<TI, DK, DV, KEEP>), grid, block, 0, a.stream, a, C);
    else
        hipLaunchKernelGGL((gdr_recurrent_kernel<TI, DK, DV, SWEEP>), grid, block, 0, a.stream, a, C);
    return hipGetLastError();
}

template <typename TI>
hipError_t dispatch(const Args &a, int mode, int C)
{
#define GDR_CASE(DK_, DV_) if (a.dk == DK_ && a.dv == DV_) return launch_t<TI, DK_, DV_>(a, mode, C);
#define GDR_ROW(DK_) GDR_CASE(DK_, 16) GDR_CASE(DK_, 32) GDR_CASE(DK_, 64) GDR_CASE(DK_, 128)
    GDR_ROW(16) GDR_ROW(32) GDR_ROW(64) GDR_ROW(128)
#undef GDR_ROW
#undef GDR_CASE
    return hipErrorInvalidValue;
}

hipError_t run(const Args &a, int mode, int C)
{
    if (a.in == In::F32) return dispatch<float>(a, mode, C);
    if (a.in == In::BF16) return dispatch<bf16>(a, mode, C);
    return dispatch<e4m3>(a, mode, C);
}

}  // namespace

hipError_t launch_recurrent_fwd(const Args &a) { return run(a, FWD, 1 << 30); }
hipError_t launch_recurrent_keep(const Args &a, int C) { return run(a, KEEP, C); }
hipError_t launch_recurrent_sweep(const Args &a, int C) { return run(a, SWEEP, C); }

}  // namespace gdr
