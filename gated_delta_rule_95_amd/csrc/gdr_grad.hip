// Gated delta rule, backward: the gradients of one chunk from its entry
// state S, exit cotangent L, residuals R and cotangents Ub, all chunks in
// parallel.  With U = beta R, Yb = beta Ub, D_ij = exp(G_i - G_j):
//
//   dP = [i >= j] scale D (dO U^T)          dN = -[i > j] D (Yb U^T)
//   dq = scale e^G dO S^T + dP K
//   dk = -e^G Yb S^T + e^{G_C - G} U L^T + dP^T Q + (dN + dN^T) K
//   dbeta_i = Ub_i . R_i
//   dg_t = sum_{i >= t} a_i + sum_{i < t} b_i + e^{G_C} <L, S> + sum_{j < t <= i} E_ij
//     a_i = q_i . (scale e^G dO S^T)_i - k_i . (e^G Yb S^T)_i
//     b_i = k_i . (e^{G_C - G} U L^T)_i,   E = dP (Q K^T) + dN (K K^T), i > j
//
// Every term of dg carries the decays it passes through, so none cancels
// against another however fast the decay is.
//
// Bound by latency: a workgroup passes through the phases above once for each
// value head, with some tens of products a wave in each.  fp32, 600 tokens, 4
// value heads of 32 x 64: 23.5 us for 40 workgroups.
#include "gdr_device.h"

namespace gdr {
namespace {

__device__ __forceinline__ f32x4 mma4(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// fp32 on the fp32 matrix cores (16x16x4): lane (n, g) = (lane % 16, lane / 16)
// takes contraction index 4 g + i at step i, so both operands of a product
// of row-major tiles are 16-byte reads of a row.
constexpr int C32 = kRecurrentChunk;
static_assert(C32 == 32, "the lane layouts below");

template <typename TI, int DK, int DV>
struct alignas(16) GradSmem {
    float q[C32][DK + 4], k[C32][DK + 4];
    float dO[C32][DV + 4], U[C32][DV + 4], Yb[C32][DV + 4];
    float dP[C32][C32 + 4], dN[C32][C32 + 4], qk[C32][C32 + 4], kk[C32][C32 + 4];
    double G[C32];
    float eG[C32], eR[C32], a[4][C32], b[4][C32], ls[4];
};

template <typename TI, int DK, int DV>
__global__ __launch_bounds__(256)
void gdr_grad_kernel(Args a)
{
    using TO = typename OutOf<TI>::type;
    constexpr int C = C32;
    __shared__ GradSmem<TI, DK, DV> s;
    const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
    const int ln = lane % 16, lg = lane / 16;
    const int64_t slot = blockIdx.x / a.Hk;
    const int hk = blockIdx.x % a.Hk, grp = a.Hv / a.Hk;
    int n, c;
    if (!find_chunk(a.seq, slot, C, n, c)) return;
    const Seq sq = seq_of(a.seq, n);
    const int tok = sq.bos + c * C;
    const int nt = sq.len - c * C < C ? sq.len - c * C : C;
    const auto Q = src<TI>(a.q, a.qe), K = src<TI>(a.k, a.ke);
    const auto O = src<TO>(a.dO, nullptr);
    for (int i = tid; i < C * DK / 4; i += 256) {
        const int t = i / (DK / 4), ch = 4 * (i % (DK / 4));
        f32x4 qq = {0.f, 0.f, 0.f, 0.f}, kk = qq;
        if (t < nt) {
            const int64_t row = (int64_t)(tok + t) * a.Hk + hk;
            qq = Q.ld4(row, DK, ch);
            kk = K.ld4(row, DK, ch);
        }
        *reinterpret_cast<f32x4 *>(&s.q[t][ch]) = qq;
        *reinterpret_cast<f32x4 *>(&s.k[t][ch]) = kk;
    }
    constexpr int MT = (DK / 16 + 3) / 4;      // channel tiles per wave
    f32x4 dq[MT][2] = {}, dk[MT][2] = {};
    for (int h = 0; h < grp; ++h) {
        const int hv = hk * grp + h;
        __syncthreads();
        for (int i = tid; i < C * DV / 4; i += 256) {
            const int t = i / (DV / 4), x = 4 * (i % (DV / 4));
            f32x4 o = {0.f, 0.f, 0.f, 0.f}, u = o, y = o;
            if (t < nt) {
                const int64_t row = (int64_t)(tok + t) * a.Hv + hv;
                const float b = a.beta[row];
                o = O.ld4(row, DV, x);
                u = b * *reinterpret_cast<const f32x4 *>(a.R + row * DV + x);
                y = b * *reinterpret_cast<const f32x4 *>(a.Ub + row * DV + x);
            }
            *reinterpret_cast<f32x4 *>(&s.dO[t][x]) = o;
            *reinterpret_cast<f32x4 *>(&s.U[t][x]) = u;
            *reinterpret_cast<f32x4 *>(&s.Yb[t][x]) = y;
        }
        if (tid < C) {
            double x = tid < nt ? (double)floor_g(a.g[(int64_t)(tok + tid) * a.Hv + hv]) : 0.0;
#pragma unroll
            for (int m = 1; m < C; m *= 2) {
                const double y = __shfl_up(x, m);
                if (tid >= m) x += y;
            }
            s.G[tid] = x;
        }
        __syncthreads();
        if (tid < C) {
            s.eG[tid] = exp2_64(s.G[tid] * LOG2E64);
            s.eR[tid] = exp2_64((s.G[C - 1] - s.G[tid]) * LOG2E64);
        }
        // dbeta: eight threads a token
        {
            const int t = tid / 8;
            float x = 0.f;
            const int64_t row = (int64_t)(tok + t) * a.Hv + hv;
            if (t < nt)
                for (int i = tid % 8; i < DV; i += 8) x += a.R[row * DV + i] * a.Ub[row * DV + i];
#pragma unroll
            for (int m = 1; m < 8; m *= 2) x += __shfl_xor(x, m);
            if (t < nt && tid % 8 == 0) a.dbeta[row] = x;
        }
        // the four C x C products, one a wave
        {
            const float *A = wave == 0 ? &s.dO[0][0] : wave == 1 ? &s.Yb[0][0] : wave == 2 ? &s.q[0][0] : &s.k[0][0];
            const float *B = wave < 2 ? &s.U[0][0] : &s.k[0][0];
            const int D = wave < 2 ? DV : DK, ld = D + 4;
            float(*out)[C + 4] = wave == 0 ? s.dP : wave == 1 ? s.dN : wave == 2 ? s.qk : s.kk;
            for (int m = 0; m < 2; ++m)
                for (int nn = 0; nn <= m; ++nn) {
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                    for (int x = 0; x < D; x += 16) {
                        const f32x4 av = *reinterpret_cast<const f32x4 *>(A + (16 * m + ln) * ld + x + 4 * lg);
                        const f32x4 bv = *reinterpret_cast<const f32x4 *>(B + (16 * nn + ln) * ld + x + 4 * lg);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc = mma4(av[i], bv[i], acc);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) out[16 * m + 4 * lg + i][16 * nn + ln] = acc[i];
                }
        }
        __syncthreads();
        for (int x = tid; x < C * C; x += 256) {
            const int i = x / C, j = x % C;
            float p = 0.f, nn = 0.f, e = 0.f;
            if (i >= j) {
                const float d = exp2_64((s.G[i] - s.G[j]) * LOG2E64);
                p = a.scale * d * s.dP[i][j];
                if (i > j) {
                    nn = -d * s.dN[i][j];
                    e = p * s.qk[i][j] + nn * s.kk[i][j];
                }
            }
            s.dP[i][j] = p;
            s.dN[i][j] = nn;
            s.qk[i][j] = e;
        }
        __syncthreads();
        // channel tiles: products with the state and its cotangent, then
        // with the rows of the chunk
        const int64_t st = ((slot * a.Hv + hv) * DK) * DV;
        float ra[2][4] = {}, rb[2][4] = {}, ls = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int ch = 16 * (wave + 4 * m);
            if (ch < DK) {
                f32x4 x1[2] = {}, x2[2] = {}, x3[2] = {};
                for (int x = 0; x < DV; x += 16) {
                    const int64_t at = st + (int64_t)(ch + ln) * DV + x + 4 * lg;
                    const f32x4 sv = *reinterpret_cast<const f32x4 *>(a.Sc + at);
                    const f32x4 lv = *reinterpret_cast<const f32x4 *>(a.Lc + at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) ls += sv[i] * lv[i];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const f32x4 o = *reinterpret_cast<const f32x4 *>(&s.dO[16 * t + ln][x + 4 * lg]);
                        const f32x4 y = *reinterpret_cast<const f32x4 *>(&s.Yb[16 * t + ln][x + 4 * lg]);
                        const f32x4 u = *reinterpret_cast<const f32x4 *>(&s.U[16 * t + ln][x + 4 * lg]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x1[t] = mma4(o[i], sv[i], x1[t]);
                            x2[t] = mma4(y[i], sv[i], x2[t]);
                            x3[t] = mma4(u[i], lv[i], x3[t]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 16 * t + 4 * lg + i;
                        const float qv = s.q[row][ch + ln], kv = s.k[row][ch + ln];
                        const float d1 = a.scale * s.eG[row] * x1[t][i], d2 = s.eG[row] * x2[t][i];
                        const float d3 = s.eR[row] * x3[t][i];
                        ra[t][i] += qv * d1 - kv * d2;
                        rb[t][i] += kv * d3;
                        dq[m][t][i] += d1;
                        dk[m][t][i] += d3 - d2;
                    }
                for (int x = 0; x < C; x += 16) {
                    float kb[4], qb[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        kb[i] = s.k[x + 4 * lg + i][ch + ln];
                        qb[i] = s.q[x + 4 * lg + i][ch + ln];
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 16 * t + ln, j = x + 4 * lg + i;
                            dq[m][t] = mma4(s.dP[row][j], kb[i], dq[m][t]);
                            dk[m][t] = mma4(s.dP[j][row], qb[i], dk[m][t]);
                            dk[m][t] = mma4(s.dN[row][j] + s.dN[j][row], kb[i], dk[m][t]);
                        }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = ra[t][i], y = rb[t][i];
#pragma unroll
                for (int m = 1; m < 16; m *= 2) {
                    x += __shfl_xor(x, m);
                    y += __shfl_xor(y, m);
                }
                if (ln == 0) {
                    s.a[wave][16 * t + 4 * lg + i] = x;
                    s.b[wave][16 * t + 4 * lg + i] = y;
                }
            }
#pragma unroll
        for (int m = 1; m < 64; m *= 2) ls += __shfl_xor(ls, m);
        if (lane == 0) s.ls[wave] = ls;
        __syncthreads();
        {
            // eight threads a token, each every eighth row
            const int t = tid / 8;
            float x = 0.f;
#pragma unroll
            for (int i0 = 0; i0 < C; i0 += 8) {
                const int i = i0 + tid % 8;
#pragma unroll
                for (int w = 0; w < 4; ++w) x += i >= t ? s.a[w][i] : s.b[w][i];
                if (i >= t)
                    for (int j = 0; j < t; ++j) x += s.qk[i][j];
            }
#pragma unroll
            for (int m = 1; m < 8; m *= 2) x += __shfl_xor(x, m);
            if (tid % 8 == 0 && t < nt)
                a.dg[(int64_t)(tok + t) * a.Hv + hv] =
                    x + exp2_64(s.G[C - 1] * LOG2E64) * (s.ls[0] + s.ls[1] + s.ls[2] + s.ls[3]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int ch = 16 * (wave + 4 * m) + ln;
        if (ch < DK)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * t + 4 * lg + i;
                    if (row < nt) {
                        const int64_t at = ((int64_t)(tok + row) * a.Hk + hk) * DK + ch;
                        kda::Elem<TO>::st((TO *)a.dq + at, dq[m][t][i]);
                        kda::Elem<TO>::st((TO *)a.dkey + at, dk[m][t][i]);
                    }
                }
    }
}

template <typename TI, int DK, int DV>
hipError_t launch_t(const Args &a)
{
    const int64_t blocks = bwd_slots(a.seq.n_seqs, a.seq.n_tokens, C32) * a.Hk;
    if (blocks * 256 >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    hipLaunchKernelGGL((gdr_grad_kernel<TI, DK, DV>), dim3((unsigned)blocks), dim3(256), 0,
                       a.stream, a);
    return hipGetLastError();
}

template <typename TI>
hipError_t dispatch(const Args &a)
{
#define GDR_CASE(DK_, DV_) if (a.dk == DK_ && a.dv == DV_) return launch_t<TI, DK_, DV_>(a);
#define GDR_ROW(DK_) GDR_CASE(DK_, 16) GDR_CASE(DK_, 32) GDR_CASE(DK_, 64) GDR_CASE(DK_, 128)
    GDR_ROW(16) GDR_ROW(32) GDR_ROW(64) GDR_ROW(128)
#undef GDR_ROW
#undef GDR_CASE
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_grad32(const Args &a)
{
    if (a.in == In::F32) return dispatch<float>(a);
    if (a.in == In::BF16) return dispatch<bf16>(a);
    return dispatch<e4m3>(a);
}

}  // namespace gdr
