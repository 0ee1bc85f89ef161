// Gated delta rule in chunks of 64 tokens on the matrix cores (bf16 or 8-bit
// inputs, d_k and d_v of 64 or 128): the forward, the forward that keeps
// states for the backward, and the reverse sweep.
//
// Forward, with G the inclusive cumsum of g in the chunk, D_ij = e^{G_i - G_j},
// N_ij = [i > j] D_ij k_i.k_j, b = beta:
//     Y = V - e^G K S;   (I + N diag(b)) R = Y;   O = scale e^G Q S + P R
//     S <- e^{G_C} S + K^T (b e^{G_C - G} R),     P_ij = [i >= j] scale D_ij b_j q_i.k_j
// Reverse, with L the cotangent of the state behind the chunk:
//     F = P0^T dO + e^{G_C - G} K L;   (I + (diag(b) N)^T) Ub = F;   dV = b Ub
//     L <- e^{G_C} L + Q^T (scale e^G dO) - K^T (e^G b Ub),   P0: P without b_j
//
// One workgroup runs a (sequence, value head, 64 state columns) chain.  Four
// consumer waves hold 16 columns of S (L) each in registers, in the matrix
// cores' result layout, and never exchange anything: every operand they
// multiply from the right is one of their own results.  The triangular system
// is solved by substitution over four blocks of 16 tokens with the diagonal
// blocks inverted (so it is as stable as substitution is: keys may repeat).
// Four producer waves build the next chunk's left operands in the other half
// of the LDS meanwhile; one barrier a chunk.  Producer w forms row w of the
// tiles of K K^T and row 3 - w of K Q^T straight from global loads in operand
// layout, five tiles each, and inverts diagonal block w by itself: no
// exchange among producers either.
#include "gdr_chunk.h"

namespace gdr {
namespace {

constexpr int C = 64;
enum { FWD = 0, KEEP = 1, SWEEP = 2 };

// a 16 x 16 left operand in three parts, lane order: lane (ln, lg) has row
// ln, columns 4 lg .. 4 lg + 3
struct Block {
    u32x2 p[3][WAVE];
};

template <int DK, int NC, int MODE>
struct Stage {
    static constexpr int LK = DK + 16;           // odd multiples of 32 bytes: no bank conflicts
    static constexpr int LV = 16 * NC + 16;
    bf16 K[C][LK], Q[C][LK], V[C][LV];           // V: v, or dO in the sweep
    // operands of 1 KiB in lane order
    bf16x8 P[2][MODE == KEEP ? 1 : 6][WAVE];   // [part][0, 1, 2a, 2b, 3a, 3b]
    bf16x8 Apair[2][3][WAVE];                    // a block of rows against two of columns
    Block Aone[2], T[4];                         // block against block; inverted diagonal blocks
    float eG[C], eR[C];                          // e^G; b e^{G_C - G} (sweep: e^{G_C - G})
    float beta[C];
    float gamma;
};

template <int DK, int NC, int MODE>
struct alignas(16) Smem {
    Stage<DK, NC, MODE> st[2];
    float G[4][3][C];                            // per producer: G hi, G lo, beta
};

// scalar pieces of a lane's four rows of token block t
__device__ __forceinline__ f32x4 ld4f(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
template <typename TI, int DK, int NC, int MODE>
struct Producer {
    using R = Rows<TI>;
    static constexpr int KS = DK / 32;
    static constexpr int VL = NC / 2;            // 16-byte loads of V a thread
    static constexpr bool SW = MODE == SWEEP;
    // operand rows: K blocks, and in the sweep Q blocks; the lane blocks
    typename R::raw_t kb[4][KS], qb[SW ? 4 : 1][KS], kw[KS], xw[KS];
    u32x4 v[VL > 0 ? VL : 1];
    typename Rows<TI>::raw_t v8[VL > 0 ? VL : 1];
    float g, beta;

    // requests chunk inputs: n rows from token tok
    __device__ __forceinline__ void load(const Args &a, int64_t tok, int n, int hk, int hv, int col,
                                         int w, int ln, int lg, int ptid)
    {
        const R K(a.k, a.ke, tok, n, a.Hk, hk, DK), Q(a.q, a.qe, tok, n, a.Hk, hk, DK);
        const int hi = w > 3 - w ? w : 3 - w;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int c = 32 * s + 8 * lg;
            kw[s] = K.raw(16 * w + ln, c);
            if constexpr (SW) {
                xw[s] = K.raw(16 * (3 - w) + ln, c);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b >= w) kb[b][s] = K.raw(16 * b + ln, c);
                    if (b >= 3 - w) qb[b][s] = Q.raw(16 * b + ln, c);
                }
            } else {
                if constexpr (MODE == FWD) xw[s] = Q.raw(16 * (3 - w) + ln, c);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (b <= (MODE == FWD ? hi : w)) kb[b][s] = K.raw(16 * b + ln, c);
            }
        }
        const int row = ptid / 4, cv = col + (ptid % 4) * (4 * NC);
        if constexpr (SW) {
            const Rows<bf16> V(a.dO, nullptr, tok, n, a.Hv, hv, a.dv);
#pragma unroll
            for (int i = 0; i < VL; ++i) v[i] = V.raw(row, cv + 8 * i);
        } else {
            const R V(a.v, a.ve, tok, n, a.Hv, hv, a.dv);
#pragma unroll
            for (int i = 0; i < VL; ++i) v8[i] = V.raw(row, cv + 8 * i);
        }
        const int lane = ln + 16 * lg;
        const rsrc_t rg = make_rsrc(a.g + tok * a.Hv, n * a.Hv * 4), rb = make_rsrc(a.beta + tok * a.Hv, n * a.Hv * 4);
        g = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rg, (lane * a.Hv + hv) * 4, 0, 0));
        beta = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rb, (lane * a.Hv + hv) * 4, 0, 0));
    }

    // A operands in three parts from a lane's four values of one tile
    static __device__ __forceinline__ void put_block(Block &t, int lane, f32x4 x, const Eye &eye)
    {
        u32x2 h, m, l;
        split_half(x, eye, h, m, l);
        t.p[0][lane] = h;
        t.p[1][lane] = m;
        t.p[2][lane] = l;
    }
    static __device__ __forceinline__ void put_side(bf16x8 (*t)[WAVE], int lane, int side, f32x4 x, const Eye &eye)
    {
        u32x2 p[3];
        split_half(x, eye, p[0], p[1], p[2]);
#pragma unroll
        for (int i = 0; i < 3; ++i) reinterpret_cast<u32x2 *>(&t[i][lane])[side] = p[i];
    }

    // builds the stage; `next` requests the chunk after it once the
    // registers of this one are free
    template <typename F>
    __device__ __forceinline__ void build(Stage<DK, NC, MODE> &st, float (*gp)[C], const Eye &eye, float scale,
                                          int w, int ln, int lg, int ptid, F next)
    {
        const int lane = ln + 16 * lg;
        // cumulative log2-decay in double, held as two floats
        double G = (double)floor_g(g) * (double)LOG2E;
#pragma unroll
        for (int d = 1; d < C; d *= 2) {
            const double y = __shfl_up(G, d);
            if (lane >= d) G += y;
        }
        const double Gend = __shfl(G, C - 1);
        const float gh = (float)G, gl = (float)(G - (double)gh);
        gp[0][lane] = gh;
        gp[1][lane] = gl;
        gp[2][lane] = beta;
        if (w == 0) {
            const float er = kda::fast_exp2((float)(Gend - G));
            st.eG[lane] = kda::fast_exp2((float)G);
            st.eR[lane] = SW ? er : er * beta;
            st.beta[lane] = beta;
            if (lane == 0) st.gamma = kda::fast_exp2((float)Gend);
        }
        // K and Q blocks to the stage, tile products
        f32x4 kk[4] = {}, kq[4] = {};
        bf16x8 kwf[KS], xwf[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            kwf[s] = R::bf(kw[s]);
            *reinterpret_cast<bf16x8 *>(&st.K[16 * w + ln][32 * s + 8 * lg]) = kwf[s];
            if constexpr (MODE != KEEP) xwf[s] = R::bf(xw[s]);
            if constexpr (MODE == FWD)
                *reinterpret_cast<bf16x8 *>(&st.Q[16 * (3 - w) + ln][32 * s + 8 * lg]) = xwf[s];
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const bool in_kk = SW ? b >= w : b <= w, in_kq = SW ? b >= 3 - w : b <= 3 - w;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (in_kk) kk[b] = mma(R::bf(kb[b][s]), kwf[s], kk[b]);
                if constexpr (MODE == FWD)
                    if (in_kq) kq[b] = mma(R::bf(kb[b][s]), xwf[s], kq[b]);
                if constexpr (SW)
                    if (in_kq) {
                        const bf16x8 qf = R::bf(qb[b][s]);
                        kq[b] = mma(qf, xwf[s], kq[b]);
                        if (b == 3 - w) *reinterpret_cast<bf16x8 *>(&st.Q[16 * b + ln][32 * s + 8 * lg]) = qf;
                    }
            }
        }
        {
            const int row = ptid / 4, c = (ptid % 4) * (4 * NC);
#pragma unroll
            for (int i = 0; i < VL; ++i)
                *reinterpret_cast<bf16x8 *>(&st.V[row][c + 8 * i]) = SW ? Rows<bf16>::bf(v[i]) : R::bf(v8[i]);
        }
        next();
        // tiles: lane token x = 16 (block) + ln, row tokens y = 16 b + 4 lg + e;
        // x is the later one in the forward, the earlier one in the sweep
        const float sgn = SW ? -1.f : 1.f;
        const int xk = 16 * w + ln, xq = 16 * (3 - w) + ln;
        f32x4 diag = {0.f, 0.f, 0.f, 0.f};
        const float ghk = gp[0][xk], glk = gp[1][xk], ghq = gp[0][xq], glq = gp[1][xq];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const bool in_kk = SW ? b >= w : b <= w, in_kq = SW ? b >= 3 - w : b <= 3 - w;
            const int y = 16 * b + 4 * lg;
            const f32x4 yh = ld4f(&gp[0][y]), yl = ld4f(&gp[1][y]), yb = ld4f(&gp[2][y]);
            if (in_kk) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool off = SW ? y + e > xk : y + e < xk;
                    const float d = kda::fast_exp2(sgn * ((ghk - yh[e]) + (glk - yl[e])));
                    x[e] = off ? d * yb[e] * kk[b][e] : 0.f;
                }
                if (b == w) {
                    diag = x;
                } else {
                    x = -x;
                    // forward: 1 <- 0, 3 <- 2 one block, 2 and 3 <- (0, 1);
                    // sweep: 2 <- 3, 0 <- 1 one block, 1 and 0 <- (2, 3)
                    if ((w ^ 1) == b) put_block(st.Aone[SW ? (w == 2 ? 0 : 1) : (w == 1 ? 0 : 1)], lane, x, eye);
                    else put_side(st.Apair[SW ? (w == 1 ? 0 : 1) : (w == 2 ? 0 : 1)], lane, b & 1, x, eye);
                }
            }
            if (MODE != KEEP && in_kq) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool in = SW ? y + e >= xq : y + e <= xq;
                    const float d = kda::fast_exp2(sgn * ((ghq - yh[e]) + (glq - yl[e])));
                    x[e] = in ? d * (SW ? scale : scale * yb[e]) * kq[b][e] : 0.f;
                }
                const int r = 3 - w, op = SW ? (r < 2 ? 2 * r + (b >> 1) : r + 2) : (r < 2 ? r : 2 * r - 2 + (b >> 1));
                u32x2 h, m, l;
                split_half(x, eye, h, m, l);
                reinterpret_cast<u32x2 *>(&st.P[0][op][lane])[b & 1] = h;
                reinterpret_cast<u32x2 *>(&st.P[1][op][lane])[b & 1] = m;
            }
        }
        // (I + A)^-1 of the diagonal block row by row: lane row i = ln solves
        // t (I + A) = e_i from the last column to the first (sweep: A is
        // upper triangular, from the first on)
        float *sc = reinterpret_cast<float *>(&st.T[w]);     // [column][row], 20 floats a column
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[(4 * lg + e) * 20 + ln] = diag[e];
        __builtin_amdgcn_wave_barrier();
        float t[16];
#pragma unroll
        for (int jj = 0; jj < 16; ++jj) {
            const int j = SW ? jj : 15 - jj;
            float acc = ln == j ? 1.f : 0.f;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
                if (SW ? 4 * k4 >= j : 4 * k4 + 3 <= j) continue;
                const f32x4 av = ld4f(&sc[j * 20 + 4 * k4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = 4 * k4 + e;
                    if (SW ? k < j : k > j) acc -= t[k] * av[e];
                }
            }
            t[j] = acc;
        }
        f32x4 tv;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            tv[e] = lg == 0 ? t[e] : lg == 1 ? t[4 + e] : lg == 2 ? t[8 + e] : t[12 + e];
        __builtin_amdgcn_wave_barrier();
        put_block(st.T[w], lane, tv, eye);
    }
};

// ---------------------------------------------------------------------------
// consumers
// ---------------------------------------------------------------------------
// channels of the state's row tiles: rows 4 lg + e of tiles 2 s and 2 s + 1 are
// the channels 32 s + 8 lg + e and + 4, so a pair's rows in one lane are the
// eight channels of one 16-byte operand read
__device__ __forceinline__ int channel(int t, int lg, int e) { return 32 * (t >> 1) + 8 * lg + 4 * (t & 1) + e; }

__device__ __forceinline__ f32x4 mul_block(const Block &t, int lane, const Half &b, f32x4 c)
{
    const u32x2 h = t.p[0][lane], m = t.p[1][lane], l = t.p[2][lane];
    c = mma(join(h, l), b.lh, c);
    c = mma(join(m, m), b.hm, c);
    return mma(join(h, h), b.hm, c);
}
__device__ __forceinline__ f32x4 mul_pair(const bf16x8 (*t)[WAVE], int lane, const Parts<3> &b, f32x4 c)
{
    const bf16x8 h = t[0][lane], m = t[1][lane], l = t[2][lane];
    c = mma(h, b.p[2], c);
    c = mma(l, b.p[0], c);
    c = mma(m, b.p[1], c);
    c = mma(m, b.p[0], c);
    c = mma(h, b.p[1], c);
    return mma(h, b.p[0], c);
}

template <typename TI, int DK, int NC, int MODE>
struct Consumer {
    static constexpr int RT = DK / 16, KS = DK / 32;
    using TO = bf16;
    f32x4 S[RT];

    // K^T or Q^T operand: channels of row tile ct against tokens 32 s ..
    static __device__ __forceinline__ bf16x8 transposed(const bf16 (*X)[Stage<DK, NC, MODE>::LK], int ct, int s, int ln, int lg)
    {
        const int c = 32 * (ct >> 1) + 8 * (ln & 3) + 4 * (ct & 1), r = 32 * s + 4 * lg + (ln >> 2);
        return join(lds_tr(&X[r][c]), lds_tr(&X[r + 16][c]));
    }

    __device__ __forceinline__ void forward(const Stage<DK, NC, MODE> &st, const Eye &eye, float scale, int w, int ln, int lg,
                                            rsrc_t out, int row_bytes, int head)
    {
        const int lane = ln + 16 * lg;
        f32x4 X[4] = {}, O[4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Parts<3> p = split_pair<3>(S[2 * s], S[2 * s + 1], eye);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                X[t] = mma_parts<3>(lds8(&st.K[16 * t + ln][32 * s + 8 * lg]), p, X[t]);
                if constexpr (MODE == FWD) O[t] = mma_parts<2>(lds8(&st.Q[16 * t + ln][32 * s + 8 * lg]), Parts<2>{{p.p[0], p.p[1]}}, O[t]);
            }
        }
        f32x4 R[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f32x4 v = widen(lds_tr(&st.V[16 * t + 4 * lg + (ln >> 2)][16 * w + 4 * (ln & 3)]));
            const f32x4 eg = ld4f(&st.eG[16 * t + 4 * lg]);
            R[t] = v - eg * X[t];
            if constexpr (MODE == FWD) O[t] *= scale * eg;
        }
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        u32x2 h, m, l;
        Half x = split_half(R[0], eye, h, m, l);
        R[0] = mul_block(st.T[0], lane, x, zero);
        x = split_half(R[0], eye, h, m, l);
        R[1] = mul_block(st.Aone[0], lane, x, R[1]);
        x = split_half(R[1], eye, h, m, l);
        R[1] = mul_block(st.T[1], lane, x, zero);
        const Parts<3> r01 = split_pair<3>(R[0], R[1], eye);
        R[2] = mul_pair(st.Apair[0], lane, r01, R[2]);
        R[3] = mul_pair(st.Apair[1], lane, r01, R[3]);
        x = split_half(R[2], eye, h, m, l);
        R[2] = mul_block(st.T[2], lane, x, zero);
        x = split_half(R[2], eye, h, m, l);
        R[3] = mul_block(st.Aone[1], lane, x, R[3]);
        x = split_half(R[3], eye, h, m, l);
        R[3] = mul_block(st.T[3], lane, x, zero);
        if constexpr (MODE == FWD) {
            const Parts<2> r23 = split_pair<2>(R[2], R[3], eye);
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                // operands 0, 1, 2a, 2b, 3a, 3b: rows 0, 1, 2, 2, 3, 3 against tokens 0-31 (2b, 3b: 32-63)
                const int t = i < 2 ? i : 1 + i / 2;
                const bool late = i == 3 || i == 5;
                const bf16x8 h = st.P[0][i][lane], m = st.P[1][i][lane];
                const bf16x8 rh = late ? r23.p[0] : r01.p[0], rm = late ? r23.p[1] : r01.p[1];
                O[t] = mma(m, rh, O[t]);
                O[t] = mma(h, rm, O[t]);
                O[t] = mma(h, rh, O[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int off = (16 * t + 4 * lg + e) * row_bytes + head;
                if constexpr (MODE == FWD)
                    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)O[t][e]), out, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(R[t][e]), out, off, 0, 0);
            }
        const float gam = st.gamma;
        Parts<3> u[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
            u[s] = split_pair<3>(ld4f(&st.eR[32 * s + 4 * lg]) * R[2 * s], ld4f(&st.eR[32 * s + 16 + 4 * lg]) * R[2 * s + 1], eye);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            S[t] *= gam;
#pragma unroll
            for (int s = 0; s < 2; ++s) S[t] = mma_parts<3>(transposed(st.K, t, s, ln, lg), u[s], S[t]);
        }
    }
};

// where a state column block starts for a lane; rows by channel()
template <int RT>
__device__ __forceinline__ void load_state(f32x4 *S, const float *p, int dv, int lg)
{
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t][e] = p ? p[(int64_t)channel(t, lg, e) * dv] : 0.f;
}
template <int RT>
__device__ __forceinline__ void store_state(const f32x4 *S, float *p, int dv, int lg)
{
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(int64_t)channel(t, lg, e) * dv] = S[t][e];
}

// Workgroups of one key head (its value heads' column blocks) share q and k:
// unit u of them runs on XCD u % 8 (workgroups go round the XCDs in order), so
// that the second and later reads hit that XCD's L2.
__device__ __forceinline__ bool my_chain(const Args &a, int per_unit, int &n, int &hk, int &j)
{
    const int64_t b = blockIdx.x, slot = b / 8;
    const int64_t u = (slot / per_unit) * 8 + b % 8;
    j = (int)(slot % per_unit);
    if (u >= (int64_t)a.seq.n_seqs * a.Hk) return false;
    n = (int)(u / a.Hk);
    hk = (int)(u % a.Hk);
    return true;
}

template <typename TI, int DK, int NC, int MODE>
__global__ __launch_bounds__((NC + 4) * WAVE)
void gdr_chunk_kernel(Args a)
{
    __shared__ Smem<DK, NC, MODE> sm;
    constexpr int BV = 16 * NC;
    const int CB = a.dv / BV, grp = a.Hv / a.Hk;
    int n, hk, j;
    if (!my_chain(a, grp * CB, n, hk, j)) return;
    const int hv = hk * grp + j / CB, col = (j % CB) * BV;
    const int tid = threadIdx.x, lane = tid % WAVE, ln = lane % 16, lg = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const Seq sq = seq_of(a.seq, n);
    const int bos = __builtin_amdgcn_readfirstlane(sq.bos), len = __builtin_amdgcn_readfirstlane(sq.len);
    const int chunks = (len + C - 1) / C;
    // tiles above the diagonal in the operand pairs stay zero
    for (int i = tid; i < (int)(sizeof(sm.st[0].P) / sizeof(bf16x8)); i += (NC + 4) * WAVE) {
        (&sm.st[0].P[0][0][0])[i] = bf16x8{};
        (&sm.st[1].P[0][0][0])[i] = bf16x8{};
    }
    __syncthreads();
    const Eye eye = make_eye(lane);
    const auto nrows = [&](int c) { return len - c * C < C ? len - c * C : C; };
    if (wave >= NC) {
        const int w = wave - NC, ptid = tid - NC * WAVE;
        Producer<TI, DK, NC, MODE> p;
        const auto request = [&](int c) {
            if (c < chunks) p.load(a, bos + (int64_t)c * C, nrows(c), hk, hv, col, w, ln, lg, ptid);
        };
        request(0);
        for (int c = 0; c < chunks; ++c) {
            p.build(sm.st[c & 1], sm.G[w], eye, a.scale, w, ln, lg, ptid, [&] { request(c + 1); });
            __syncthreads();
        }
    } else {
        Consumer<TI, DK, NC, MODE> q;
        const int64_t st = ((int64_t)n * a.Hv + hv) * DK * a.dv + col + 16 * wave + ln;
        load_state<DK / 16>(q.S, a.S0 ? a.S0 + st : nullptr, a.dv, lg);
        for (int c = 0; c < chunks; ++c) {
            __syncthreads();
            const int64_t tok = bos + (int64_t)c * C;
            const int es = MODE == FWD ? 2 : 4, rb = a.Hv * a.dv * es;
            char *base = MODE == FWD ? static_cast<char *>(a.o) : reinterpret_cast<char *>(a.R);
            if constexpr (MODE == KEEP) {
                const int64_t slot = bos / C + n + c;
                store_state<DK / 16>(q.S, a.Sc + (slot * a.Hv + hv) * DK * a.dv + col + 16 * wave + ln, a.dv, lg);
            }
            q.forward(sm.st[c & 1], eye, a.scale, wave, ln, lg, make_rsrc(base + tok * rb, nrows(c) * rb), rb,
                      (hv * a.dv + col + 16 * wave + ln) * es);
        }
        if (MODE == FWD && a.S_T) store_state<DK / 16>(q.S, a.S_T + st, a.dv, lg);
    }
}

template <typename TI, int DK, int NC, int MODE>
hipError_t launch_t(const Args &a)
{
    const int64_t units = (int64_t)a.seq.n_seqs * a.Hk;
    const int64_t blocks = (units + 7) / 8 * 8 * (a.Hv / a.Hk) * (a.dv / (16 * NC));
    constexpr int NT = (NC + 4) * WAVE;
    if (blocks * NT >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    static_assert(sizeof(Smem<DK, NC, MODE>) <= 160 * 1024, "LDS");
    hipLaunchKernelGGL((gdr_chunk_kernel<TI, DK, NC, MODE>), dim3((unsigned)blocks), dim3(NT), 0,
                       a.stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_fwd(const Args &a)
{
    return a.dk == 128 ? launch_t<bf16, 128, 4, FWD>(a) : launch_t<bf16, 64, 4, FWD>(a);
}

}  // namespace gdr
