// Gated delta rule token by token in fp32: the forward, the forward that
// keeps states for the backward, and the reverse sweep.  Right for every
// type and head size.
//
// Columns of the state evolve independently, so a wave owns GC columns and
// all rows of S in registers: lane (c, r) = (lane % GC, lane / GC) holds rows
// 4 (NG m + r) + e of column c, NG = 64 / GC.  Two tokens are taken at once.
// With a = e^g, u = beta R, their column sums are all of the state before both:
//     R1 = v1 - a1 S^T k1;   R2 = v2 - a1 a2 S^T k2 - a2 u1 (k1 . k2)
//     o1 = scale (a1 S^T q1 + u1 (k1 . q1))
//     o2 = scale (a1 a2 S^T q2 + a2 u1 (k1 . q2) + u2 (k2 . q2))
//     S <- a1 a2 S + (a2 u1) k1 + u2 k2
// and in the sweep, from the later token to the earlier, y = scale dO:
//     Ub2 = L^T k2 + y2 (q2 . k2);   w = beta Ub
//     Ub1 = a2 (L^T k1 + y2 (q2 . k1) - w2 (k2 . k1)) + y1 (q1 . k1)
//     L <- a1 (a2 (L + q2 y2 - k2 w2) + q1 y1 - k1 w1)
// The sums over the lanes of a column go through the same moves between lanes,
// each value in its own quarter (half) of the wave: four sums cost little more
// than one.
//
// Bound by the chain of tokens: a pair is some 11 d_k / NG vector operations, a
// sum over lanes and their latencies, so with few chains a wave takes fewer
// columns and more lanes share one (GC 4 or 8 in place of 16), and as many
// waves again stage the tiles and form the keys' products (fp32, d_k = d_v =
// 128, 32 chains of 1024 tokens: token by token 0.26 ms, in pairs 0.20, with
// waves that stage 0.165: 160 ns a token; 2 x 1025 tokens, 8 heads of 64 x 128:
// 0.19, 0.148, 0.120 ms).  With 16 columns a wave there are waves enough, and
// all do both (512 chains: 1.17 ms, with waves that stage 1.61 ms).  A pair's
// operands are read from the LDS one pair ahead where that takes few registers
// (with 16 rows a lane it halves the waves: 128 chains 0.54 in place of 0.35
// ms), and a tile's from memory one tile ahead.
#include "gdr_device.h"

namespace gdr {
namespace {

constexpr int TT = 16;               // tokens staged at a time

enum { FWD = 0, KEEP = 1, SWEEP = 2 };

constexpr int64_t kFew = 8192, kSome = 32768;

template <int DK, int DV, int GC>
struct Shape {
    static constexpr int NG = WAVE / GC;
    static constexpr bool APART = GC <= 8;       // waves of their own fill the LDS
    static constexpr int NW = DV / GC < 4 ? DV / GC : 4;
    static constexpr int NT = NW * WAVE;         // threads that do either
    static constexpr int THREADS = APART ? 2 * NT : NT;
    static constexpr int BV = GC * NW;
    static constexpr int RM = DK / (4 * NG);     // four-row pieces a lane
    static_assert(RM >= 1, "row groups");
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// within each row of 16 lanes: sum over the lanes of equal lane % GC
template <int GC>
__device__ __forceinline__ float sum_row(float x)
{
    if constexpr (GC <= 4) x += dpp<0x124>(x);           // row_ror 4
    if constexpr (GC <= 8) x += dpp<0x128>(x);           // row_ror 8
    return x;
}
// sums over the lanes of equal lane % GC, each in every lane
template <int GC>
__device__ __forceinline__ void sum2(float &a, float &b)
{
    swap32(a, b);                                        // a below, b above
    float x, y;
    kda::row_pair(a + b, x, y);
    kda::half_pair(sum_row<GC>(x + y), a, b);
}
template <int GC>
__device__ __forceinline__ void sum4(float &a, float &b, float &c, float &d)
{
    swap32(a, c);
    swap32(b, d);
    float x = a + c, y = b + d;
    swap16(x, y);                                        // rows a, b, c, d
    kda::row_pair(sum_row<GC>(x + y), x, y);
    kda::half_pair(x, a, c);
    kda::half_pair(y, b, d);
}
// over N neighbouring lanes: the sum, in each; and the value of the lane N before
template <int N>
__device__ __forceinline__ float sum_near(float x)
{
    x += dpp<0xb1>(x);                                   // quad_perm 1 0 3 2
    x += dpp<0x4e>(x);                                   // quad_perm 2 3 0 1
    if constexpr (N >= 8) x += dpp<0x141>(x);            // row_half_mirror
    if constexpr (N >= 16) x += dpp<0x140>(x);           // row_mirror
    if constexpr (N >= 32) {
        float a, b;
        kda::row_pair(x, a, b);
        x = a + b;
    }
    return x;
}
template <int N>
__device__ __forceinline__ float earlier(float x)
{
    float a, b;
    if constexpr (N == 4) return dpp<0x114>(x);          // row_shr 4
    if constexpr (N == 8) return dpp<0x118>(x);          // row_shr 8
    if constexpr (N == 16) kda::row_pair(x, a, b);
    if constexpr (N == 32) kda::half_pair(x, a, b);
    return a;
}

// MODE FWD: writes o and S_T.  KEEP: the state before every token of index
// 0, C, 2C, ... of its sequence to Sc[slot], and R_t = v_t - S'^T k_t.
// SWEEP: from the last token to the first with the cotangent L of the state,
//     L += scale q_t dO_t^T;  Ub_t = L^T k_t;  L = exp(g_t) (L - k_t (beta_t Ub_t)^T),
// writing dv = beta Ub, Ub, L behind the last token of every chunk (Lc) and
// dS0.
template <int DK, int DV, int GC>
struct Tile {
    float k[TT][DK], q[TT][DK], v[TT][Shape<DK, DV, GC>::BV];
    // of a pair of tokens (written by different threads): e^g and beta of
    // each; k . q of each, k1 . k2, k1 . q2
    float gate[TT / 2][4], dots[TT / 2][4];
};

template <typename TI, int DK, int DV, int GC, int MODE>
__device__ __forceinline__ void token_pass(const Args &a, Tile<DK, DV, GC> *s_t, int64_t block)
{
    constexpr int C = kRecurrentChunk;
    using Sh = Shape<DK, DV, GC>;
    using TO = typename OutOf<TI>::type;
    constexpr int RM = Sh::RM, NG = Sh::NG, NT = Sh::NT, BV = Sh::BV;
    constexpr int CB = DV / BV;
    static_assert(sizeof(Tile<DK, DV, GC>) % 16 == 0, "16-byte reads");
    const bool fills = Sh::APART && threadIdx.x >= NT;
    const int tid = threadIdx.x % NT, lane = tid % WAVE, wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int c = lane % GC, r = lane / GC;
    const int64_t chain = block / CB;
    const int cb = (int)(block % CB);
    const int n = (int)(chain / a.Hv), hv = (int)(chain % a.Hv), hk = hv / (a.Hv / a.Hk);
    Seq sq = seq_of(a.seq, n);
    sq.bos = __builtin_amdgcn_readfirstlane(sq.bos);      // addresses of rows are scalar arithmetic
    sq.len = __builtin_amdgcn_readfirstlane(sq.len);
    const int col = cb * BV + GC * wave + c;
    const auto Q = src<TI>(a.q, a.qe), K = src<TI>(a.k, a.ke), V = src<TI>(a.v, a.ve);
    const auto G = src<TO>(a.dO, nullptr);
    const int64_t st = (chain * DK) * DV + col;
    const float *init = MODE == SWEEP ? a.dS_T : a.S0;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const auto row_of = [&](int m, int e) { return 4 * (NG * m + r) + e; };
    const int tiles = (sq.len + TT - 1) / TT;
    // a tile's rows: from memory to registers, from there to the LDS
    constexpr int NK = (TT * DK / 4 + NT - 1) / NT, NV = (TT * BV / 4 + NT - 1) / NT;
    f32x4 rk[NK], rq[NK], rv[NV];
    float ra = 0.f, rb = 0.f;
    const auto first = [&](int tile) { return (MODE == SWEEP ? tiles - 1 - tile : tile) * TT; };
    const auto request = [&](int tile) {
        const int t0 = first(tile), nt = sq.len - t0 < TT ? sq.len - t0 : TT;
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int i = tid + x * NT, t = i / (DK / 4), ch = 4 * (i % (DK / 4));
            rk[x] = rq[x] = zero;
            if (t < nt) {
                const int64_t row = (int64_t)(sq.bos + t0 + t) * a.Hk + hk;
                rk[x] = K.ld4(row, DK, ch);
                if (MODE != KEEP) rq[x] = Q.ld4(row, DK, ch);
            }
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = tid + x * NT, t = i / (BV / 4), y = 4 * (i % (BV / 4));
            rv[x] = zero;
            if (t < nt) {
                const int64_t row = (int64_t)(sq.bos + t0 + t) * a.Hv + hv;
                if constexpr (MODE == SWEEP) rv[x] = G.ld4(row, DV, cb * BV + y);
                else rv[x] = V.ld4(row, DV, cb * BV + y);
            }
        }
        if (tid < TT) {
            const bool in = tid < nt;
            const int64_t row = (int64_t)(sq.bos + t0 + (in ? tid : 0)) * a.Hv + hv;
            ra = in ? a.g[row] : 0.f;
            rb = in ? a.beta[row] : 0.f;
        }
    };
    const auto fill = [&](int tile) {
        Tile<DK, DV, GC> &s = s_t[tile & 1];
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int i = tid + x * NT, t = i / (DK / 4), ch = 4 * (i % (DK / 4));
            if (NK * NT == TT * DK / 4 || t < TT) {
                *reinterpret_cast<f32x4 *>(&s.k[t][ch]) = rk[x];
                if (MODE != KEEP) *reinterpret_cast<f32x4 *>(&s.q[t][ch]) = rq[x];
            }
            // DK / 4 neighbouring lanes a token, a pair's tokens side by side
            const auto dot = [](f32x4 y, f32x4 z) { return sum_near<DK / 4>(y[0] * z[0] + y[1] * z[1] + y[2] * z[2] + y[3] * z[3]); };
            f32x4 k1;
#pragma unroll
            for (int e = 0; e < 4; ++e) k1[e] = earlier<DK / 4>(rk[x][e]);
            const float kk = dot(k1, rk[x]), kq = MODE != KEEP ? dot(rk[x], rq[x]) : 0.f, kq2 = MODE != KEEP ? dot(k1, rq[x]) : 0.f;
            if (t < TT && ch == 0) {
                s.dots[t / 2][t & 1] = kq;
                if (t & 1) {
                    s.dots[t / 2][2] = kk;
                    s.dots[t / 2][3] = kq2;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = tid + x * NT, t = i / (BV / 4), y = 4 * (i % (BV / 4));
            if (t < TT) *reinterpret_cast<f32x4 *>(&s.v[t][y]) = rv[x];
        }
        if (tid < TT) {
            s.gate[tid / 2][2 * (tid & 1)] = decay(floor_g(ra));
            s.gate[tid / 2][2 * (tid & 1) + 1] = rb;
        }
    };
    // Tile t is filled before barrier t and read behind it; its half of the LDS
    // is filled again behind barrier t + 1, which readers reach when done.
    if (!Sh::APART || fills) {
        if (tiles > 0) request(0);
    }
    if (fills) {
        for (int tile = 0; tile < tiles; ++tile) {
            fill(tile);
            if (tile + 1 < tiles) request(tile + 1);
            __syncthreads();
        }
        return;
    }
    f32x4 S[RM];
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[m][e] = init ? init[st + (int64_t)row_of(m, e) * DV] : 0.f;
    for (int tile = 0; tile < tiles; ++tile) {
        const Tile<DK, DV, GC> &s = s_t[tile & 1];
        const int t0 = first(tile), nt = sq.len - t0 < TT ? sq.len - t0 : TT;
        if (!Sh::APART) fill(tile);
        __syncthreads();
        if (!Sh::APART && tile + 1 < tiles) request(tile + 1);
        // states at the chunks' borders, which are tiles' borders
        if (MODE == KEEP ? t0 % C == 0 : MODE == SWEEP && (tile == 0 || (t0 + TT) % C == 0)) {
            const int64_t slot = sq.bos / C + n + t0 / C;
            float *dst = (MODE == KEEP ? a.Sc : a.Lc) + ((slot * a.Hv + hv) * DK) * DV + col;
#pragma unroll
            for (int m = 0; m < RM; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[(int64_t)row_of(m, e) * DV] = S[m][e];
        }
        // Two lanes of a column store, one token each; the others' places, and
        // those of the rows behind the sequence (whole tiles are run: rows of
        // zeros with e^g = 1 change nothing), are past the buffers' ends and
        // dropped.
        const int64_t tok = (int64_t)(sq.bos + t0) * a.Hv * DV;
        const int rowe = a.Hv * DV, place = r < 2 ? r * rowe + hv * DV + col : 0x10000000;
        const rsrc_t out0 = make_rsrc(MODE == FWD ? (const void *)((TO *)a.o + tok) : (const void *)((MODE == KEEP ? a.R : a.Ub) + tok),
                                      nt * rowe * (MODE == FWD ? (int)sizeof(TO) : 4));
        const rsrc_t out1 = make_rsrc((TO *)a.dval + tok, MODE == SWEEP ? nt * rowe * (int)sizeof(TO) : 0);
        const auto put = [](rsrc_t r, int at, float x, auto type) {
            if constexpr (sizeof(type) == 2)
                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)x), r, 2 * at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, 4 * at, 0, 0);
        };
        struct Pair {
            f32x4 k1[RM], k2[RM], q1[RM], q2[RM], gate, dots;
            float x1, x2;
        };
        const auto read = [&](int i) {
            const int p = MODE == SWEEP ? TT / 2 - 1 - i : i, t = 2 * p;
            Pair y;
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                y.k1[m] = *reinterpret_cast<const f32x4 *>(&s.k[t][row_of(m, 0)]);
                y.k2[m] = *reinterpret_cast<const f32x4 *>(&s.k[t + 1][row_of(m, 0)]);
                if (MODE != KEEP) {
                    y.q1[m] = *reinterpret_cast<const f32x4 *>(&s.q[t][row_of(m, 0)]);
                    y.q2[m] = *reinterpret_cast<const f32x4 *>(&s.q[t + 1][row_of(m, 0)]);
                }
            }
            y.gate = *reinterpret_cast<const f32x4 *>(s.gate[p]);
            y.dots = *reinterpret_cast<const f32x4 *>(s.dots[p]);
            y.x1 = s.v[t][GC * wave + c];
            y.x2 = s.v[t + 1][GC * wave + c];
            return y;
        };
        const auto step = [&](const Pair &y, int i) {
            const int at = place + 2 * (MODE == SWEEP ? TT / 2 - 1 - i : i) * rowe;
            const float a1 = y.gate[0], b1 = y.gate[1], a2 = y.gate[2], b2 = y.gate[3], a12 = a1 * a2;
            const float kq1 = y.dots[0], kq2 = y.dots[1], kk = y.dots[2], kq = y.dots[3];
            const auto dot = [&](const f32x4 *x) {
                f32x4 z = S[0] * x[0];               // four partial sums: one would be a chain of dependent adds
#pragma unroll
                for (int m = 1; m < RM; ++m) z += S[m] * x[m];
                return (z[0] + z[1]) + (z[2] + z[3]);
            };
            float K1 = dot(y.k1), K2 = dot(y.k2);
            if constexpr (MODE == SWEEP) {
                sum2<GC>(K1, K2);
                const float y1 = a.scale * y.x1, y2 = a.scale * y.x2;
                const float U2 = K2 + y2 * kq2, w2 = b2 * U2;
                const float U1 = a2 * (K1 + y2 * kq - w2 * kk) + y1 * kq1, w1 = b1 * U1;
                const float p2 = a12 * y2, n2 = -a12 * w2, p1 = a1 * y1, n1 = -a1 * w1;
#pragma unroll
                for (int m = 0; m < RM; ++m) {
                    S[m] = a12 * S[m] + p2 * y.q2[m] + p1 * y.q1[m];
                    S[m] += n2 * y.k2[m];
                    S[m] += n1 * y.k1[m];
                }
                put(out0, at, r == 0 ? U1 : U2, 0.f);
                put(out1, at, r == 0 ? w1 : w2, TO());
            } else {
                float Q1 = 0.f, Q2 = 0.f;
                if constexpr (MODE == FWD) {
                    Q1 = dot(y.q1);
                    Q2 = dot(y.q2);
                    sum4<GC>(K1, K2, Q1, Q2);
                } else
                    sum2<GC>(K1, K2);
                const float R1 = y.x1 - a1 * K1, u1 = b1 * R1, w = a2 * u1;
                const float R2 = y.x2 - (a12 * K2 + w * kk), u2 = b2 * R2;
#pragma unroll
                for (int m = 0; m < RM; ++m) {
                    S[m] = a12 * S[m] + w * y.k1[m];
                    S[m] += u2 * y.k2[m];
                }
                if (MODE == FWD) put(out0, at, a.scale * (r == 0 ? a1 * Q1 + u1 * kq1 : a12 * Q2 + w * kq + u2 * kq2), TO());
                else put(out0, at, r == 0 ? R1 : R2, 0.f);
            }
        };
        if constexpr (RM <= 2) {
            // a pair ahead, two sets of registers in turn
            Pair x = read(0);
#pragma unroll 2
            for (int i = 0; i < TT / 2; i += 2) {
                const Pair y = read(i + 1);
                step(x, i);
                x = read((i + 2) % (TT / 2));
                step(y, i + 1);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < TT / 2; ++i) step(read(i), i);
        }
    }
    float *out = MODE == FWD ? a.S_T : MODE == SWEEP ? a.dS0 : nullptr;
    if (out) {
#pragma unroll
        for (int m = 0; m < RM; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[st + (int64_t)row_of(m, e) * DV] = S[m][e];
    }
}

// the forward, or the backward's two passes (which do not wait for each other)
// in one launch: the sweep's workgroups, then the keeping forward's
template <typename TI, int DK, int DV, int GC, bool BWD>
__global__ __launch_bounds__((Shape<DK, DV, GC>::THREADS))
void gdr_recurrent_kernel(Args a, int64_t half)
{
    __shared__ __align__(16) Tile<DK, DV, GC> tiles[2];
    if constexpr (BWD) {
        if (blockIdx.x < half) token_pass<TI, DK, DV, GC, SWEEP>(a, tiles, blockIdx.x);
        else token_pass<TI, DK, DV, GC, KEEP>(a, tiles, blockIdx.x - half);
    } else
        token_pass<TI, DK, DV, GC, FWD>(a, tiles, blockIdx.x);
}

template <typename TI, int DK, int DV, int GC>
hipError_t launch_gc(const Args &a, bool bwd)
{
    using Sh = Shape<DK, DV, GC>;
    const int64_t half = (int64_t)a.seq.n_seqs * a.Hv * (DV / Sh::BV), blocks = bwd ? 2 * half : half;
    if (blocks * Sh::THREADS >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    const dim3 grid((unsigned)blocks), block(Sh::THREADS);
    if (bwd)
        hipLaunchKernelGGL((gdr_recurrent_kernel<TI, DK, DV, GC, true>), grid, block, 0, a.stream, a, half);
    else if constexpr (!std::is_same<TI, e4m3>::value)
        hipLaunchKernelGGL((gdr_recurrent_kernel<TI, DK, DV, GC, false>), grid, block, 0, a.stream, a, half);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

template <typename TI, int DK, int DV>
hipError_t launch_t(const Args &a, bool bwd)
{
    // Sixteen columns a wave do the least work in all; eight (four) give twice
    // (four times) the waves, each with a shorter step.  Forward, fp32, d = 128,
    // 4 / 8 / 16 columns a wave: 32 chains of 1024 tokens 0.16 / 0.26 / 0.45 ms;
    // 64 chains 0.24 / 0.26 / 0.45 ms; 128 chains 0.44 / 0.34 / 0.46 ms; 512
    // chains 1.73 / 1.30 / 1.21 ms.  The backward's launch has two passes.
    const int64_t columns = (int64_t)a.seq.n_seqs * a.Hv * DV * (bwd ? 2 : 1);
    if constexpr (DK >= 64)
        if (columns <= kFew) return launch_gc<TI, DK, DV, 4>(a, bwd);
    if constexpr (DK >= 32)
        if (columns < kSome) return launch_gc<TI, DK, DV, 8>(a, bwd);
    return launch_gc<TI, DK, DV, 16>(a, bwd);
}

template <typename TI>
hipError_t dispatch(const Args &a, bool bwd)
{
#define GDR_CASE(DK_, DV_) if (a.dk == DK_ && a.dv == DV_) return launch_t<TI, DK_, DV_>(a, bwd);
#define GDR_ROW(DK_) GDR_CASE(DK_, 16) GDR_CASE(DK_, 32) GDR_CASE(DK_, 64) GDR_CASE(DK_, 128)
    GDR_ROW(16) GDR_ROW(32) GDR_ROW(64) GDR_ROW(128)
#undef GDR_ROW
#undef GDR_CASE
    return hipErrorInvalidValue;
}

hipError_t run(const Args &a, bool bwd)
{
    if (a.in == In::F32) return dispatch<float>(a, bwd);
    if (a.in == In::BF16) return dispatch<bf16>(a, bwd);
    return dispatch<e4m3>(a, bwd);
}

}  // namespace

hipError_t launch_recurrent_fwd(const Args &a) { return run(a, false); }
hipError_t launch_recurrent_keep_sweep(const Args &a) { return run(a, true); }

}  // namespace gdr
