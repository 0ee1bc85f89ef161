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
// is solved by substitution over two blocks of 32 tokens with the diagonal
// blocks inverted: 16 by 16 by substitution too, joined by one product (so it
// is as stable as substitution is: keys may repeat).  Four producer waves
// build the next chunk's left operands in the other half of the LDS meanwhile,
// two barriers a chunk: two of them form and invert a diagonal block of 32
// each, two the rest of K K^T and K Q^T, without a word among them.
//
// Bound by the chain of chunks: a chunk's products wait for one another, most
// of all in the substitution, and the matrix cores are busy for 48% of the
// forward's time (37% of the backward's two passes).  Forward, 4 sequences of
// 4096 tokens, 32 heads of 128 x 128: 262 us (1.6 TB/s of inputs, outputs and
// states; the consumers by themselves 183 us, the producers 178); 13 ragged
// sequences, 20011 tokens: 281 us (201 and 170).  Keeping forward and sweep of
// the former: 0.71 ms for 2.3 GB moved.  Operands straight from global memory
// in place of the LDS take twice the time (a load of 64 scattered pieces takes
// 900 cycles and more to issue).
//
// What only o sees, S, R and P in its products, is held in two bf16 parts, the
// products below 2^-16 left out: o is rounded to bf16 (2^-8) behind it, and its
// error stays that of the rounding (1.66e-3 of its norm, as in 32 bits
// throughout); 0.3% of its elements round to the other neighbour.  Three parts
// bring that to 0.02% and cost 8 to 10% (262 -> 288 and 284 -> 311 us); one part
// of S and R saves 5% and misses repeated keys by 4e-3.
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
    static constexpr int PP = MODE == SWEEP ? 3 : 2;
    bf16 K[C * DK], Q[C * DK];                   // by Swz
    // operands of 1 KiB in lane order
    bf16x8 P[PP][MODE == KEEP ? 1 : 6][WAVE];   // [part][0, 1, 2a, 2b, 3a, 3b]
    bf16x8 Apair[2][3][WAVE];                    // a block of rows against two of columns
    // inverted diagonal blocks of 32: the rows with one block of 16, those with two
    Block Tone[2];
    bf16x8 Tpair[2][3][WAVE];
    float eG[C], eR[C];                          // e^G; b e^{G_C - G} (sweep: e^{G_C - G})
    float eGs[C];                                // scale e^G
    float eGb[C], beta[C];                       // b e^G and b, in the sweep
    float gamma;
};

template <int NC>
struct Values {
    bf16 x[C][16 * NC + 8];
};

template <int DK, int NC, int MODE>
struct alignas(16) Smem {
    Stage<DK, NC, MODE> st[2];
    // v, or dO in the sweep: read before a chunk's first barrier and the next
    // written behind it, so one is enough (two measured 2% slower in a ragged
    // batch)
    Values<NC> V;
    float G[4][3][C];                            // per producer: G hi, G lo, beta
};

// scalar pieces of a lane's four rows of token block t
__device__ __forceinline__ f32x4 ld4f(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
__device__ __forceinline__ double last_lane(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, 63), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Producer W of four.  A tile pairs the lane tokens of one block of 16 with the
// row tokens of another, the lane's the later ones in the forward and the
// earlier ones in the sweep.
template <typename TI, int DK, int NC, int MODE, int W>
struct Producer {
    using R = Rows<TI>;
    using St = Stage<DK, NC, MODE>;
    static constexpr int KS = DK / 32;
    static constexpr int VL = NC / 2;            // 16-byte loads of V a thread
    static constexpr bool SW = MODE == SWEEP;
    static constexpr int PR = W / 2;             // odd waves: the diagonal block of 32 it inverts
    // odd waves: the blocks of 16 the off-diagonal tile pairs
    static constexpr int OL = SW ? 2 * PR : 2 * PR + 1, OR = SW ? 2 * PR + 1 : 2 * PR;
    // even waves: lane block and first row block of its half of the corner
    // (rows 2, 3 against 0, 1; sweep: 0, 1 against 2, 3), lane blocks of K Q^T
    static constexpr int CL = SW ? PR : 2 + PR, CR = SW ? 2 : 0;
    static constexpr int L0 = SW ? PR : 3 - PR, L1 = 3 - L0;
    static constexpr bool reaches(int lane, int row) { return SW ? row >= lane : row <= lane; }
    typename R::raw_t kw[KS], qw[KS];            // rows of K and Q, block W
    u32x4 v[VL];
    typename R::raw_t v8[VL];
    float g, beta;

    // requests chunk inputs: n rows from token tok
    __device__ __forceinline__ void load(const Args &a, int64_t tok, int n, int hk, int hv, int col,
                                         int ln, int lg, int ptid)
    {
        const typename R::at_t at = R::at(ln, a.Hk, hk, DK, 8 * lg);
        const R K(a.k, a.ke, tok + 16 * W, n - 16 * W, a.Hk, DK), Q(a.q, a.qe, tok + 16 * W, n - 16 * W, a.Hk, DK);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            kw[s] = K.raw(at, 32 * s);
            if (MODE != KEEP) qw[s] = Q.raw(at, 32 * s);
        }
        const int row = ptid / 4, cv = col + (ptid % 4) * (4 * NC);
        if constexpr (SW) {
            const Rows<bf16> V(a.dO, nullptr, tok, n, a.Hv, a.dv);
#pragma unroll
            for (int i = 0; i < VL; ++i) v[i] = V.raw(Rows<bf16>::at(row, a.Hv, hv, a.dv, cv), 8 * i);
        } else {
            const R V(a.v, a.ve, tok, n, a.Hv, a.dv);
#pragma unroll
            for (int i = 0; i < VL; ++i) v8[i] = V.raw(R::at(row, a.Hv, hv, a.dv, cv), 8 * i);
        }
        const int lane = ln + 16 * lg;
        const rsrc_t rg = make_rsrc(a.g + tok * a.Hv, n * a.Hv * 4), rb = make_rsrc(a.beta + tok * a.Hv, n * a.Hv * 4);
        g = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rg, (lane * a.Hv + hv) * 4, 0, 0));
        beta = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rb, (lane * a.Hv + hv) * 4, 0, 0));
    }

    // left operands in three parts from a lane's four values of one tile
    static __device__ __forceinline__ void put_block(Block &t, int lane, f32x4 x, const Eye &eye)
    {
        u32x2 p[3];
        split3(x, eye, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) t.p[i][lane] = p[i];
    }
    static __device__ __forceinline__ void put_side(bf16x8 (*t)[WAVE], int lane, int side, f32x4 x, const Eye &eye)
    {
        u32x2 p[3];
        split3(x, eye, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) reinterpret_cast<u32x2 *>(&t[i][lane])[side] = p[i];
    }
    // decays between lane token x and the row tokens y .. y + 3, times w.  The
    // exponent's sum rounds (|d| 2^-25 of the factor 2^d): such a factor stands
    // in a row beside the token's own, which has no decay.
    static __device__ __forceinline__ f32x4 decays(const float (*gp)[C], int x, int y, f32x4 w)
    {
        const float gh = gp[0][x], gl = gp[1][x];
        const f32x4 yh = ld4f(&gp[0][y]), yl = ld4f(&gp[1][y]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float d = (gh - yh[e]) + (gl - yl[e]);
            w[e] *= kda::fast_exp2(SW ? -d : d);
        }
        return w;
    }

    // (I + A)^-1 of a diagonal block of 32 from its tiles, into the stage
    static __device__ __forceinline__ void invert(St &st, f32x4 d0, f32x4 d1, f32x4 off, const Eye &eye, int ln, int lg)
    {
        const int lane = ln + 16 * lg;
        // three tiles of 16 x 16 floats where the operands go later
        float *sc = reinterpret_cast<float *>(st.Tpair[PR]), *s0 = sc, *s1 = sc + 256, *so = sc + 512;
        *reinterpret_cast<f32x4 *>(&s0[16 * ln + 4 * lg]) = d0;
        *reinterpret_cast<f32x4 *>(&s1[16 * ln + 4 * lg]) = d1;
        *reinterpret_cast<f32x4 *>(&so[16 * ln + 4 * lg]) = off;
        __builtin_amdgcn_wave_barrier();
        // Both blocks of 16 at once, one a half wave: lane row i = ln solves
        // t (I + A) = e_i, each entry when final taken out of those left (from
        // the last to the first; sweep: A is upper triangular, from the first
        // on).  Row j is read a step ahead.
        float *mine = sc + 256 * (lg >> 1);
        float t[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] = ln == j ? 1.f : 0.f;
        f32x4 av[4];
        const auto row = [&](int j, f32x4 *x) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)
                if (SW ? 4 * k4 + 3 > j : 4 * k4 < j) x[k4] = ld4f(&mine[16 * j + 4 * k4]);
        };
        row(SW ? 0 : 15, av);
#pragma unroll
        for (int jj = 0; jj < 15; ++jj) {
            const int j = SW ? jj : 15 - jj;
            f32x4 ahead[4];
            if (jj < 14) row(SW ? j + 1 : j - 1, ahead);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (SW ? k > j : k < j) t[k] -= t[j] * av[k / 4][k % 4];
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) av[k4] = ahead[k4];
            // The step's updates are independent of one another and made now:
            // left to itself the compiler gathers each entry's into a chain
            // at its end, with every row in registers.
            asm volatile("" : "+v"(t[0]), "+v"(t[1]), "+v"(t[2]), "+v"(t[3]), "+v"(t[4]), "+v"(t[5]), "+v"(t[6]), "+v"(t[7]));
            asm volatile("" : "+v"(t[8]), "+v"(t[9]), "+v"(t[10]), "+v"(t[11]), "+v"(t[12]), "+v"(t[13]), "+v"(t[14]), "+v"(t[15]));
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
            *reinterpret_cast<f32x4 *>(&mine[16 * ln + 4 * k4]) = f32x4{t[4 * k4], t[4 * k4 + 1], t[4 * k4 + 2], t[4 * k4 + 3]};
        asm volatile("" ::: "memory");
        // X = -T_L A T_R for the off-diagonal tile (lane block L, row block R),
        // transposed and on the fp32 matrix cores: W = A^T T_L^T, X^T = -T_R^T W
        const float *tr = OL % 2 ? s0 : s1;
        const f32x4 t0 = ld4f(&s0[16 * ln + 4 * lg]), t1 = ld4f(&s1[16 * ln + 4 * lg]);
        const f32x4 bl = OL % 2 ? t1 : t0;
        f32x4 w = {0.f, 0.f, 0.f, 0.f}, x = w;
        float ac[4], tc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ac[i] = so[16 * (4 * lg + i) + ln];
            tc[i] = tr[16 * (4 * lg + i) + ln];
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) w = __builtin_amdgcn_mfma_f32_16x16x4f32(ac[i], bl[i], w, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) x = __builtin_amdgcn_mfma_f32_16x16x4f32(tc[i], w[i], x, 0, 0, 0);
        put_block(st.Tone[PR], lane, SW ? t1 : t0, eye);
        put_side(st.Tpair[PR], lane, 0, SW ? t0 : -x, eye);
        put_side(st.Tpair[PR], lane, 1, SW ? -x : t1, eye);
    }

    // builds the stage; `next` requests the chunk after it once this one's
    // rows are in the stage
    template <typename F>
    __device__ __forceinline__ void build(St &st, Values<NC> &values, float (*gp)[C], const Eye &eye, float scale,
                                          int ln, int lg, int ptid, F next)
    {
        const int lane = ln + 16 * lg;
        // cumulative log2-decay in double, held as two floats
        const double G = scan64((double)floor_g(g) * LOG2E64), Gend = last_lane(G);
        const float gh = (float)G, gl = (float)(G - (double)gh);
        gp[0][lane] = gh;
        gp[1][lane] = gl;
        gp[2][lane] = beta;
        if constexpr (W == 0) {
            const float er = exp2_64(Gend - G);
            const float eg = exp2_two(gh, gl);
            st.eG[lane] = eg;
            st.eGs[lane] = scale * eg;
            st.eR[lane] = SW ? er : er * beta;
            if constexpr (SW) {
                st.eGb[lane] = beta * eg;
                st.beta[lane] = beta;
            }
            if (lane == 0) st.gamma = exp2_64(Gend);
        }
        // K and Q blocks to the stage
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int at = Swz<DK>::at(16 * W + ln, 32 * s + 8 * lg);
            *reinterpret_cast<bf16x8 *>(&st.K[at]) = R::bf(kw[s]);
            if constexpr (MODE != KEEP) *reinterpret_cast<bf16x8 *>(&st.Q[at]) = R::bf(qw[s]);
        }
        __syncthreads();                 // rows of the chunk are in the stage, and the values of the one before read
        {
            const int row = ptid / 4, c = (ptid % 4) * (4 * NC);
#pragma unroll
            for (int i = 0; i < VL; ++i)
                *reinterpret_cast<bf16x8 *>(&values.x[row][c + 8 * i]) = SW ? Rows<bf16>::bf(v[i]) : R::bf(v8[i]);
        }
        next();
        const auto rows = [&](const bf16 *x, int b, int s) { return lds8(&x[Swz<DK>::at(16 * b + ln, 32 * s + 8 * lg)]); };
        if constexpr (W % 2) {
            // the three tiles of the diagonal block of 32
            f32x4 d0 = {}, d1 = {}, off = {};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bf16x8 k0 = rows(st.K, 2 * PR, s), k1 = rows(st.K, 2 * PR + 1, s);
                d0 = mma(k0, k0, d0);
                d1 = mma(k1, k1, d1);
                off = SW ? mma(k1, k0, off) : mma(k0, k1, off);
            }
            const int x0 = 32 * PR + ln, y0 = 32 * PR + 4 * lg;
            const f32x4 b0 = ld4f(&gp[2][y0]), b1 = ld4f(&gp[2][y0 + 16]);
            d0 = decays(gp, x0, y0, b0 * d0);
            d1 = decays(gp, x0 + 16, y0 + 16, b1 * d1);
            off = decays(gp, 16 * OL + ln, 16 * OR + 4 * lg, (SW ? b1 : b0) * off);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(SW ? 4 * lg + e > ln : 4 * lg + e < ln)) d0[e] = d1[e] = 0.f;
            invert(st, d0, d1, off, eye, ln, lg);
        } else {
            // two tiles of the corner and five of K Q^T
            f32x4 kk[2] = {}, q0[4] = {}, q1[4] = {};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const bf16x8 kl = rows(st.K, CL, s);
                bf16x8 l0 = {}, l1 = {};
                if constexpr (MODE != KEEP) {
                    l0 = rows(SW ? st.K : st.Q, L0, s);
                    l1 = rows(SW ? st.K : st.Q, L1, s);
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const bool corner = b == CR || b == CR + 1, any = MODE != KEEP && (reaches(L0, b) || reaches(L1, b));
                    bf16x8 kb = {}, rb = {};
                    if (corner || (!SW && any)) kb = rows(st.K, b, s);
                    if (any) rb = SW ? rows(st.Q, b, s) : kb;
                    if (corner) kk[b - CR] = mma(kb, kl, kk[b - CR]);
                    if (MODE != KEEP && reaches(L0, b)) q0[b] = mma(rb, l0, q0[b]);
                    if (MODE != KEEP && reaches(L1, b)) q1[b] = mma(rb, l1, q1[b]);
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int y = 16 * b + 4 * lg;
                const f32x4 be = ld4f(&gp[2][y]), w = SW ? f32x4{scale, scale, scale, scale} : scale * be;
                if (b == CR || b == CR + 1) kk[b - CR] = decays(gp, 16 * CL + ln, y, be * kk[b - CR]);
                if (MODE != KEEP && reaches(L0, b)) q0[b] = decays(gp, 16 * L0 + ln, y, w * q0[b]);
                if (MODE != KEEP && reaches(L1, b)) q1[b] = decays(gp, 16 * L1 + ln, y, w * q1[b]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (SW ? 4 * lg + e < ln : 4 * lg + e > ln) q0[L0][e] = q1[L1][e] = 0.f;
            // sweep: rows 1 and 0 are in this order in the pairs
            put_side(st.Apair[SW ? 1 - PR : PR], lane, 0, -kk[0], eye);
            put_side(st.Apair[SW ? 1 - PR : PR], lane, 1, -kk[1], eye);
            const auto put_p = [&](int r, int b, f32x4 x) {
                const int op = SW ? (r < 2 ? 2 * r + (b >> 1) : r + 2) : (r < 2 ? r : 2 * r - 2 + (b >> 1));
#pragma unroll
                for (int i = 0; i < St::PP; ++i) {
                    const u32x2 h = pack4(x);
                    reinterpret_cast<u32x2 *>(&st.P[i][op][lane])[b & 1] = h;
                    if (i + 1 < St::PP) x = mma(eye.a, join(h, h), x);
                }
            };
            if constexpr (MODE != KEEP) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (reaches(L0, b)) put_p(L0, b, q0[b]);
                    if (reaches(L1, b)) put_p(L1, b, q1[b]);
                }
            }
        }
    }

    // every chunk of the chain; where(c): its first token and rows
    template <typename Tok>
    static __device__ __forceinline__ void run(const Args &a, Smem<DK, NC, MODE> &sm, int chunks, Tok where, int hk, int hv,
                                               int col, int lane, int ptid)
    {
        const int ln = lane % 16, lg = lane / 16;
        const Eye eye = make_eye(lane);
        Producer p;
        const auto request = [&](int c) {
            if (c < chunks) {
                int64_t tok;
                int n;
                where(c, tok, n);
                p.load(a, tok, n, hk, hv, col, ln, lg, ptid);
            }
        };
        request(0);
        for (int c = 0; c < chunks; ++c) {
            p.build(sm.st[c & 1], sm.V, sm.G[W], eye, a.scale, ln, lg, ptid, [&] { request(c + 1); });
            __syncthreads();
        }
    }
};

// ---------------------------------------------------------------------------
// consumers
// ---------------------------------------------------------------------------
// channels of the state's row tiles: rows 4 lg + e of tiles 2 s and 2 s + 1 are
// the channels 32 s + 8 lg + e and + 4, so a pair's rows in one lane are the
// eight channels of one 16-byte operand read
__device__ __forceinline__ int channel(int t, int lg, int e) { return 32 * (t >> 1) + 8 * lg + 4 * (t & 1) + e; }

// a block of rows against two of columns, in registers
struct PairRegs {
    bf16x8 h, m, l;
    __device__ __forceinline__ PairRegs(const bf16x8 (*t)[WAVE], int lane) : h(t[0][lane]), m(t[1][lane]), l(t[2][lane]) {}
    // one block: the other's columns are zero
    __device__ __forceinline__ PairRegs(const Block &t, int lane, bool second)
    {
        const u32x2 z = {0, 0};
        const u32x2 a = t.p[0][lane], b = t.p[1][lane], c = t.p[2][lane];
        h = second ? join(z, a) : join(a, z);
        m = second ? join(z, b) : join(b, z);
        l = second ? join(z, c) : join(c, z);
    }
};
__device__ __forceinline__ f32x4 mul_pair(const PairRegs &t, const Parts<3> &b, f32x4 c)
{
    c = mma(t.h, b.p[2], c);
    c = mma(t.l, b.p[0], c);
    c = mma(t.m, b.p[1], c);
    c = mma(t.m, b.p[0], c);
    c = mma(t.h, b.p[1], c);
    return mma(t.h, b.p[0], c);
}

template <typename TI, int DK, int NC, int MODE>
struct Consumer {
    static constexpr int RT = DK / 16, KS = DK / 32;
    // eight consumers: a third of the registers, and another consumer on the
    // same SIMD to run while one waits
    static constexpr bool LEAN = NC == 8;
    f32x4 S[RT];

    // K^T or Q^T operand: channels of row tile ct against tokens 32 s ..
    static __device__ __forceinline__ bf16x8 transposed(const bf16 *X, int ct, int s, int ln, int lg)
    {
        const int c = 32 * (ct >> 1) + 8 * (ln & 3) + 4 * (ct & 1), r = 32 * s + 4 * lg + (ln >> 2);
        const bf16 *p = X + Swz<DK>::at(r, c);           // row + 16: the same exchange of pieces
        return join(lds_tr(p), lds_tr(p + 16 * DK));
    }

    // row tiles t0 .. t1 of S += K^T (or Q^T) u over the tokens 32 s .. of the chunk
    template <int NS>
    __device__ __forceinline__ void update(const bf16 *M, const Parts<NS> &u, int s, int t0, int t1, int ln, int lg)
    {
#pragma unroll
        for (int t = 0; t < RT; ++t)
            if (t >= t0 && t < t1) S[t] = mma_parts<NS>(transposed(M, t, s, ln, lg), u, S[t]);
    }

    // Two blocks of 16 rows in fp32, from their three parts: a product with
    // the identity transposes a part exactly, and a lane stores four columns
    // of one row.  off: this lane's byte in the first block.
    static __device__ __forceinline__ void put_rows(const Parts<3> &r, const Eye &eye, rsrc_t out, int off, int row_bytes)
    {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4 x = -mma_by_parts(r, eye.a, zero), y = -mma_by_parts(r, eye.b, zero);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), out, off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), out, off + 16 * row_bytes, 0, 0);
    }

    // The state at a chunk border in fp32, in the order of the gradient
    // kernel's operands: tiles [16 channels][32 columns], each as two halves of
    // 1 KiB in lane order, lane (channel, lg) holding the columns 8 lg ..
    // 8 lg + 3 in the first and the next four in the second.  dst: the head's
    // tiles; cw: this wave's first column; row tiles 2 s and 2 s + 1.
    static __device__ __forceinline__ void put_state(const Parts<3> &p, int s, const Eye &eye, float *dst, int dv, int cw,
                                                     int ln, int lg)
    {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const int ks = dv / 32, lane = 8 * ((ln >> 2) & 1) + (ln & 3) + 16 * (((cw >> 4) & 1) * 2 + (lg >> 1));
        f32x4 *d = reinterpret_cast<f32x4 *>(dst) + (((2 * s + (ln >> 3)) * ks + cw / 32) * 2 + (lg & 1)) * WAVE + lane;
        __builtin_nontemporal_store(-mma_by_parts(p, eye.a, zero), d);
        __builtin_nontemporal_store(-mma_by_parts(p, eye.b, zero), d + 4);
    }

    // out: buffer of the chunk's rows of o (R); off: this lane's byte in block
    // 0; keep: where the entry state goes (KEEP)
    __device__ __forceinline__ void forward(const Stage<DK, NC, MODE> &st, const Values<NC> &values, const Eye &eye, int w, int ln, int lg,
                                            rsrc_t out, int row_bytes, int off, float *keep, int dv, int cw,
                                            bool more)
    {
        const int lane = ln + 16 * lg;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        // Operands are requested a phase ahead: the phases are dependent
        // chains of one wave, and the LDS latency would stand in each of
        // their steps (scheduling barriers keep the requests where they are).
        const auto pin = [] {
            if constexpr (!LEAN) __builtin_amdgcn_sched_barrier(0);
        };
        u32x2 vt[4];
        f32x4 eg[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            vt[t] = lds_tr(&values.x[16 * t + 4 * lg + (ln >> 2)][16 * w + 4 * (ln & 3)]);
            eg[t] = ld4f(&st.eG[16 * t + 4 * lg]);
        }
        const PairRegs T0(st.Tone[0], lane, false), T1(st.Tpair[0], lane);
        pin();
        f32x4 X[4] = {}, O[4] = {}, R[4];
        // three parts of S where R depends on it (with two the forward was 2%
        // faster and S_T off by up to 1e-6, dg by 1.9e-6), two where only o does
        Parts<3> p[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            p[s] = split_pair<3>(S[2 * s], S[2 * s + 1], eye);
            if constexpr (MODE == KEEP) put_state(p[s], s, eye, keep, dv, cw, ln, lg);
#pragma unroll
            for (int t = 0; t < 4; ++t) X[t] = mma_parts<3>(lds8(&st.K[Swz<DK>::at(16 * t + ln, 32 * s + 8 * lg)]), p[s], X[t]);
            if constexpr (MODE == FWD && LEAN) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    O[t] = mma_by_parts(Parts<2>{{p[s].p[0], p[s].p[1]}}, lds8(&st.Q[Swz<DK>::at(16 * t + ln, 32 * s + 8 * lg)]), O[t]);
            }
            if (s == 0 && more) __syncthreads();         // the producers' rows of the next chunk
        }
        const PairRegs A2(st.Apair[0], lane), A3(st.Apair[1], lane);
        const float gam = st.gamma;
        const f32x4 er0 = ld4f(&st.eR[4 * lg]), er1 = ld4f(&st.eR[16 + 4 * lg]);
        pin();
#pragma unroll
        for (int t = 0; t < 4; ++t) R[t] = widen(vt[t]) - eg[t] * X[t];
        // The substitution is one long dependent chain: products that do not
        // wait for it stand between its steps.  O is formed transposed (the
        // operands of a product trade places), so that a lane holds four
        // columns of one token and o goes out 8 bytes at a time.
        const auto qs = [&](int s) {
            if (MODE == FWD && s < KS && !LEAN)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    O[t] = mma_by_parts(Parts<2>{{p[s].p[0], p[s].p[1]}}, lds8(&st.Q[Swz<DK>::at(16 * t + ln, 32 * s + 8 * lg)]), O[t]);
        };
        const Parts<3> y01 = split_pair<3>(R[0], R[1], eye);
        qs(0);
        R[0] = mul_pair(T0, y01, zero);
        R[1] = mul_pair(T1, y01, zero);
        qs(1);
        const PairRegs T2(st.Tone[1], lane, false), T3(st.Tpair[1], lane);
        const f32x4 er2 = ld4f(&st.eR[32 + 4 * lg]), er3 = ld4f(&st.eR[48 + 4 * lg]);
        pin();
        const Parts<3> r01 = split_pair<3>(R[0], R[1], eye);
        qs(2);
        R[2] = mul_pair(A2, r01, R[2]);
        R[3] = mul_pair(A3, r01, R[3]);
        qs(3);
#pragma unroll
        for (int t = 0; t < RT; ++t) S[t] *= gam;
        const Parts<3> y23 = split_pair<3>(R[2], R[3], eye);
        const Parts<3> u0 = split_pair<3>(er0 * R[0], er1 * R[1], eye);
        update(st.K, u0, 0, 0, RT / 2, ln, lg);
        R[2] = mul_pair(T2, y23, zero);
        R[3] = mul_pair(T3, y23, zero);
        update(st.K, u0, 0, RT / 2, RT, ln, lg);
#pragma unroll
        for (int t = 0; t < 4; ++t) O[t] *= st.eGs[16 * t + ln];
        // operands 0, 1, 2a, 2b, 3a, 3b: rows 0, 1, 2, 2, 3, 3 against tokens
        // 0-31 (2b, 3b: 32-63)
        const auto pr = [&](int i, int t, bf16x8 rh, bf16x8 rm) {
            if constexpr (MODE == FWD) {
                const bf16x8 ph = st.P[0][i][lane], pm = st.P[1][i][lane];
                O[t] = mma(rh, pm, O[t]);
                O[t] = mma(rm, ph, O[t]);
                O[t] = mma(rh, ph, O[t]);
            }
        };
        pr(0, 0, r01.p[0], r01.p[1]);
        pr(1, 1, r01.p[0], r01.p[1]);
        pr(2, 2, r01.p[0], r01.p[1]);
        pr(4, 3, r01.p[0], r01.p[1]);
        const Parts<3> u1 = split_pair<3>(er2 * R[2], er3 * R[3], eye);
        const Parts<2> r23 = MODE == FWD ? split_pair<2>(R[2], R[3], eye) : Parts<2>{};
        pr(3, 2, r23.p[0], r23.p[1]);
        pr(5, 3, r23.p[0], r23.p[1]);
        if constexpr (MODE == FWD) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                __builtin_amdgcn_raw_buffer_store_b64(pack4(O[t]), out, off + 16 * t * row_bytes, 0, 0);
        } else {
            put_rows(r01, eye, out, off, row_bytes);
            put_rows(split_pair<3>(R[2], R[3], eye), eye, out, off + 32 * row_bytes, row_bytes);
        }
        update(st.K, u1, 1, 0, RT, ln, lg);
    }

    // out: buffer of the chunk's rows of Ub; offs: this lane's byte in block
    // 0 of it and of dv; keep: where the exit cotangent goes
    __device__ __forceinline__ void sweep(const Stage<DK, NC, MODE> &st, const Values<NC> &values, const Eye &eye, int w, int ln, int lg, rsrc_t out,
                                          int row_bytes, int off, rsrc_t dval, int vrow_bytes, int voff, float *keep, int dv,
                                          int cw, bool more)
    {
        const int lane = ln + 16 * lg;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        u32x2 d[4];
        f32x4 er[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            d[t] = lds_tr(&values.x[16 * t + 4 * lg + (ln >> 2)][16 * w + 4 * (ln & 3)]);
            er[t] = ld4f(&st.eR[16 * t + 4 * lg]);
        }
        const PairRegs T3(st.Tone[1], lane, true), T2(st.Tpair[1], lane);
        __builtin_amdgcn_sched_barrier(0);
        f32x4 F[4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Parts<3> p = split_pair<3>(S[2 * s], S[2 * s + 1], eye);
            put_state(p, s, eye, keep, dv, cw, ln, lg);
#pragma unroll
            for (int t = 0; t < 4; ++t) F[t] = mma_parts<3>(lds8(&st.K[Swz<DK>::at(16 * t + ln, 32 * s + 8 * lg)]), p, F[t]);
            if (s == 0 && more) __syncthreads();         // the producers' rows of the next chunk
        }
        const PairRegs A1(st.Apair[0], lane), A0(st.Apair[1], lane);
        const float gam = st.gamma;
        f32x4 eg[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) eg[t] = ld4f(&st.eGs[16 * t + 4 * lg]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < 4; ++t) F[t] *= er[t];
        const bf16x8 d01 = join(d[0], d[1]), d23 = join(d[2], d[3]);
        // operands 0a, 0b, 1a, 1b, 2, 3: rows 0, 0, 1, 1, 2, 3 against tokens
        // 32-63 (0a, 1a: 0-31)
        const auto pd = [&](int i, int t, bf16x8 x) {
            F[t] = mma(st.P[2][i][lane], x, F[t]);
            F[t] = mma(st.P[1][i][lane], x, F[t]);
            F[t] = mma(st.P[0][i][lane], x, F[t]);
        };
        pd(5, 3, d23);
        pd(4, 2, d23);
        const Parts<3> f23 = split_pair<3>(F[2], F[3], eye);
        pd(3, 1, d23);
        pd(1, 0, d23);
        F[3] = mul_pair(T3, f23, zero);
        F[2] = mul_pair(T2, f23, zero);
        pd(2, 1, d01);
        pd(0, 0, d01);
        const PairRegs T1(st.Tone[0], lane, true), T0(st.Tpair[0], lane);
        f32x4 eb[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) eb[t] = ld4f(&st.eGb[16 * t + 4 * lg]);
        __builtin_amdgcn_sched_barrier(0);
        const Parts<3> u23 = split_pair<3>(F[2], F[3], eye);
#pragma unroll
        for (int t = 0; t < RT; ++t) S[t] *= gam;
        const Parts<3> w01 = split_pair<3>(eg[0] * widen(d[0]), eg[1] * widen(d[1]), eye);
        F[1] = mul_pair(A1, u23, F[1]);
        F[0] = mul_pair(A0, u23, F[0]);
        const Parts<3> w23 = split_pair<3>(eg[2] * widen(d[2]), eg[3] * widen(d[3]), eye);
        update(st.Q, w01, 0, 0, RT, ln, lg);
        const Parts<3> f01 = split_pair<3>(F[0], F[1], eye);
        const Parts<3> y23 = split_pair<3>(-eb[2] * F[2], -eb[3] * F[3], eye);
        update(st.Q, w23, 1, 0, RT, ln, lg);
        F[1] = mul_pair(T1, f01, zero);
        F[0] = mul_pair(T0, f01, zero);
        update(st.K, y23, 1, 0, RT, ln, lg);
        const Parts<3> u01 = split_pair<3>(F[0], F[1], eye);
        const Parts<3> y01 = split_pair<3>(-eb[0] * F[0], -eb[1] * F[1], eye);
        // dv = beta Ub, from the transposed rows
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f32x4 u = -mma_by_parts(t < 2 ? u01 : u23, t & 1 ? eye.b : eye.a, zero);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, u), out, off + 16 * t * row_bytes, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b64(pack4(st.beta[16 * t + ln] * u), dval, voff + 16 * t * vrow_bytes, 0, 0);
        }
        update(st.K, y01, 0, 0, RT, ln, lg);
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
// that the second and later reads hit that XCD's L2.  Fewer than eight units
// leave XCDs without work, which costs where a unit has more workgroups than
// an XCD has compute units (32): 16384 tokens, 32 value heads of 128 x 128 on
// one key head take 1784 us, on two 877.  Units are dealt out with the longest
// sequences first (up to 128 of them): a long chain that starts last would run
// alone at the end.
constexpr int kSorted = 128;
__device__ __forceinline__ bool my_chain(const Args &a, int64_t b, int per_unit, int *lens, int tid, int nthreads, int &n, int &hk,
                                         int &j)
{
    const int64_t slot = b / 8;
    const int64_t u = (slot / per_unit) * 8 + b % 8;
    j = (int)(slot % per_unit);
    if (u >= (int64_t)a.seq.n_seqs * a.Hk) return false;
    n = (int)(u / a.Hk);
    hk = (int)(u % a.Hk);
    const int ns = a.seq.n_seqs;
    if (a.seq.cu_seqlens && ns > 1 && ns <= kSorted) {
        for (int i = tid; i < ns; i += nthreads) lens[i] = seq_of(a.seq, i).len;
        __syncthreads();
        if (tid < ns) {
            const int mine = lens[tid];
            int rank = 0;
            for (int i = 0; i < ns; ++i) rank += lens[i] > mine || (lens[i] == mine && i < tid);
            if (rank == n) lens[kSorted] = tid;
        }
        __syncthreads();
        n = __builtin_amdgcn_readfirstlane(lens[kSorted]);
        __syncthreads();                         // before the place is used for something else
    }
    return true;
}

// workgroup `block` of a pass over all chains
template <typename TI, int DK, int NC, int MODE>
__device__ __forceinline__ void chain_pass(const Args &a, Smem<DK, NC, MODE> &sm, int64_t block)
{
    constexpr int BV = 16 * NC;
    const int CB = a.dv / BV, grp = a.Hv / a.Hk;
    int n, hk, j;
    const int tid = threadIdx.x;
    if (!my_chain(a, block, grp * CB, reinterpret_cast<int *>(sm.G), tid, (NC + 4) * WAVE, n, hk, j)) return;
    const int hv = hk * grp + j / CB, col = (j % CB) * BV;
    const int lane = tid % WAVE, ln = lane % 16, lg = lane / 16;
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
    // step c of the chain is chunk c, or from the last one on in the sweep
    const auto where = [&](int c, int64_t &tok, int &nrow) {
        const int i = MODE == SWEEP ? chunks - 1 - c : c;
        tok = bos + (int64_t)i * C;
        nrow = len - i * C < C ? len - i * C : C;
    };
    if (wave >= NC) {
        const int w = wave - NC, ptid = tid - NC * WAVE;
#define GDR_RUN(W_) Producer<TI, DK, NC, MODE, W_>::run(a, sm, chunks, where, hk, hv, col, lane, ptid)
        if (w == 0) GDR_RUN(0);
        else if (w == 1) GDR_RUN(1);
        else if (w == 2) GDR_RUN(2);
        else GDR_RUN(3);
#undef GDR_RUN
        return;
    }
    const Eye eye = make_eye(lane);
    Consumer<TI, DK, NC, MODE> q;
    const int64_t st = ((int64_t)n * a.Hv + hv) * DK * a.dv + col + 16 * wave + ln;
    const float *init = MODE == SWEEP ? a.dS_T : a.S0;
    load_state<DK / 16>(q.S, init ? init + st : nullptr, a.dv, lg);
    // a lane's place in rows of o, R, Ub and dv: its token and four columns
    const int cw = col + 16 * wave, e0 = (ln * a.Hv + hv) * a.dv + cw + 4 * lg;
    constexpr int es = MODE == FWD ? 2 : 4;
    const int rb = a.Hv * a.dv * es;
    float *border = MODE == SWEEP ? a.Lc : a.Sc;
    if (chunks > 0) __syncthreads();                     // rows of chunk 0
    for (int c = 0; c < chunks; ++c) {
        __syncthreads();
        int64_t tok;
        int nrow;
        where(c, tok, nrow);
        const char *base = MODE == FWD ? static_cast<const char *>(a.o) : reinterpret_cast<const char *>(MODE == KEEP ? a.R : a.Ub);
        const rsrc_t out = make_rsrc(base + tok * rb, nrow * rb);
        const int64_t slot = bos / C + n + (MODE == SWEEP ? chunks - 1 - c : c);
        float *keep = border + (slot * a.Hv + hv) * DK * a.dv;
        if constexpr (MODE == SWEEP) {
            const rsrc_t dval = make_rsrc(static_cast<char *>(a.dval) + tok * (rb / 2), nrow * (rb / 2));
            q.sweep(sm.st[c & 1], sm.V, eye, wave, ln, lg, out, rb, e0 * 4, dval, rb / 2, e0 * 2, keep, a.dv, cw, c + 1 < chunks);
        } else
            q.forward(sm.st[c & 1], sm.V, eye, wave, ln, lg, out, rb, e0 * es, keep, a.dv, cw, c + 1 < chunks);
    }
    float *fin = MODE == FWD ? a.S_T : MODE == SWEEP ? a.dS0 : nullptr;
    if (fin) store_state<DK / 16>(q.S, fin + st, a.dv, lg);
}

template <int DK, int NC>
__global__ __launch_bounds__((NC + 4) * WAVE)
void gdr_chunk_fwd_kernel(Args a)
{
    __shared__ Smem<DK, NC, FWD> sm;
    static_assert(sizeof(sm) <= 160 * 1024, "LDS");
    chain_pass<bf16, DK, NC, FWD>(a, sm, blockIdx.x);
}

// The backward's two passes over the chains do not wait for each other: one
// launch has the sweep's workgroups (the longer ones) and then the keeping
// forward's, which share the compute units where either alone leaves some
// idle.
template <typename TI, int DK, int NC>
__global__ __launch_bounds__((NC + 4) * WAVE)
void gdr_chunk_bwd_kernel(Args a, int64_t half)
{
    using Sweep = Smem<DK, NC, SWEEP>;
    using Keep = Smem<DK, NC, KEEP>;
    static_assert(sizeof(Keep) <= sizeof(Sweep) && sizeof(Sweep) <= 160 * 1024, "LDS");
    __shared__ __align__(16) char raw[sizeof(Sweep)];
    if (blockIdx.x < half) chain_pass<TI, DK, NC, SWEEP>(a, *reinterpret_cast<Sweep *>(raw), blockIdx.x);
    else chain_pass<TI, DK, NC, KEEP>(a, *reinterpret_cast<Keep *>(raw), blockIdx.x - half);
}

// workgroups of one pass: units of a key head, padded to whole rounds of XCDs
template <int NC>
int64_t pass_blocks(const Args &a)
{
    const int64_t units = (int64_t)a.seq.n_seqs * a.Hk;
    return (units + 7) / 8 * 8 * (a.Hv / a.Hk) * (a.dv / (16 * NC));
}

template <int DK, int NC>
hipError_t launch_fwd_t(const Args &a)
{
    const int64_t blocks = pass_blocks<NC>(a);
    constexpr int NT = (NC + 4) * WAVE;
    if (blocks * NT >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    hipLaunchKernelGGL((gdr_chunk_fwd_kernel<DK, NC>), dim3((unsigned)blocks), dim3(NT), 0, a.stream, a);
    return hipGetLastError();
}

template <typename TI, int DK>
hipError_t launch_bwd_t(const Args &a)
{
    const int64_t half = pass_blocks<4>(a);
    constexpr int NT = 8 * WAVE;
    if (2 * half * NT >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    hipLaunchKernelGGL((gdr_chunk_bwd_kernel<TI, DK, 4>), dim3((unsigned)(2 * half)), dim3(NT), 0, a.stream, a, half);
    return hipGetLastError();
}

}  // namespace

// Eight consumers (one workgroup a chain of 128 columns) or four (two): with
// both halves of every chain running at once, four are faster (273 against
// 335 us, 128 chains of 64 chunks on 256 compute units); with more chains than
// half the compute units the halves would queue, and eight do the work of two
// workgroups in 1.2 times the time of one (129 chains: 448 against 329 us; 256:
// 534 against 429).  The count says nothing of the chains' lengths: one
// sequence of 16384 tokens beside eight of 100, 16 heads, takes 1248 us with
// eight and would take 918 with four.
constexpr int64_t kWide = 129;

hipError_t launch_chunk_fwd(const Args &a)
{
    if (a.dv == 128 && (int64_t)a.seq.n_seqs * a.Hv >= kWide)
        return a.dk == 128 ? launch_fwd_t<128, 8>(a) : launch_fwd_t<64, 8>(a);
    return a.dk == 128 ? launch_fwd_t<128, 4>(a) : launch_fwd_t<64, 4>(a);
}

hipError_t launch_chunk_keep_sweep(const Args &a)
{
    if (a.in == In::BF16) return a.dk == 128 ? launch_bwd_t<bf16, 128>(a) : launch_bwd_t<bf16, 64>(a);
    return a.dk == 128 ? launch_bwd_t<e4m3, 128>(a) : launch_bwd_t<e4m3, 64>(a);
}

}  // namespace gdr
