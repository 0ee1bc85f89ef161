// Gated delta rule token by token in fp32: the forward, the forward that
// keeps states for the backward, and the reverse sweep.  Right for every
// type and head size.
//
// Columns of the state evolve independently, so a wave owns GC columns and
// all rows of S in registers: lane (c, r) = (lane % GC, lane / GC) holds rows
// 4 (NG m + r) + e of column c, NG = 64 / GC.  Per token the two column sums
// S'^T k and S'^T q are taken together (o = S'^T q + u (k . q)), each over a
// lane's own rows and then over the row groups by moves between lanes.
//
// Bound by the chain of tokens: a token is some 4 d_k / NG vector operations, a
// sum over lanes and their latencies, so with few chains a wave takes fewer
// columns and more lanes share one (GC 4 in place of 16).  A token's operands
// are read from the LDS one token ahead and a tile's from memory one tile
// ahead.
#include "gdr_device.h"

namespace gdr {
namespace {

constexpr int TT = 16;               // tokens staged at a time

// raw buffer resource: stores at or past `bytes` are dropped
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void *base, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

enum { FWD = 0, KEEP = 1, SWEEP = 2 };

constexpr int64_t kFew = 8192, kSome = 32768;

template <int DK, int DV, int GC>
struct Shape {
    static constexpr int NG = WAVE / GC;
    static constexpr int NW = DV / GC < 4 ? DV / GC : 4;
    static constexpr int NT = NW * WAVE;
    static constexpr int BV = GC * NW;
    static constexpr int RM = DK / (4 * NG);     // four-row pieces a lane
    static_assert(RM >= 1, "row groups");
};

// sum over the lanes of equal lane % GC
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <int GC>
__device__ __forceinline__ float sum_rows(float x)
{
    if constexpr (GC <= 4) x = dpp_add<0x124>(x);        // row_ror 4
    if constexpr (GC <= 8) x = dpp_add<0x128>(x);        // row_ror 8
    return sum_groups(x);
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
    float gate[TT][4];           // e^g, beta, k . q (written by different threads)
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
    const int tid = threadIdx.x, lane = tid % WAVE, wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
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
    f32x4 S[RM];
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[m][e] = init ? init[st + (int64_t)row_of(m, e) * DV] : 0.f;

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
    if (tiles > 0) request(0);
    for (int tile = 0; tile < tiles; ++tile) {
        Tile<DK, DV, GC> &s = s_t[tile & 1];
        const int t0 = first(tile), nt = sq.len - t0 < TT ? sq.len - t0 : TT;
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int i = tid + x * NT, t = i / (DK / 4), ch = 4 * (i % (DK / 4));
            if (NK * NT == TT * DK / 4 || t < TT) {
                *reinterpret_cast<f32x4 *>(&s.k[t][ch]) = rk[x];
                if (MODE != KEEP) *reinterpret_cast<f32x4 *>(&s.q[t][ch]) = rq[x];
            }
            if (MODE == FWD) {       // k . q of every token: DK / 4 neighbouring lanes a token
                float y = rk[x][0] * rq[x][0] + rk[x][1] * rq[x][1] + rk[x][2] * rq[x][2] + rk[x][3] * rq[x][3];
#pragma unroll
                for (int m = 1; m < DK / 4; m *= 2) y += __shfl_xor(y, m);
                if (t < TT && ch == 0) s.gate[t][2] = y;
            }
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int i = tid + x * NT, t = i / (BV / 4), y = 4 * (i % (BV / 4));
            if (t < TT) *reinterpret_cast<f32x4 *>(&s.v[t][y]) = rv[x];
        }
        if (tid < TT) {
            s.gate[tid][0] = kda::fast_exp2(floor_g(ra) * LOG2E);
            s.gate[tid][1] = rb;
        }
        // the other half of the LDS was last read before the barrier of the
        // tile before, so one barrier a tile is enough
        __syncthreads();
        if (tile + 1 < tiles) request(tile + 1);
        // states at the chunks' borders, which are tiles' borders
        if (MODE == KEEP ? t0 % C == 0 : MODE == SWEEP && (tile == 0 || (t0 + TT) % C == 0)) {
            const int64_t slot = sq.bos / C + n + t0 / C;
            float *dst = (MODE == KEEP ? a.Sc : a.Lc) + ((slot * a.Hv + hv) * DK) * DV + col;
#pragma unroll
            for (int m = 0; m < RM; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[(int64_t)row_of(m, e) * DV] = S[m][e];
        }
        // One lane of a column stores; the others' places, and those of the
        // rows behind the sequence (whole tiles are run: rows of zeros with
        // e^g = 1 change nothing), are past the buffers' ends and dropped.
        const int64_t tok = (int64_t)(sq.bos + t0) * a.Hv * DV;
        const int rowe = a.Hv * DV, place = r == 0 ? hv * DV + col : 0x10000000;
        const rsrc_t out0 = make_rsrc(MODE == FWD ? (const void *)((TO *)a.o + tok) : (const void *)((MODE == KEEP ? a.R : a.Ub) + tok),
                                      nt * rowe * (MODE == FWD ? (int)sizeof(TO) : 4));
        const rsrc_t out1 = make_rsrc((TO *)a.dval + tok, MODE == SWEEP ? nt * rowe * (int)sizeof(TO) : 0);
        const auto put = [](rsrc_t r, int at, float x, auto type) {
            if constexpr (sizeof(type) == 2)
                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (bf16)x), r, 2 * at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, 4 * at, 0, 0);
        };
        struct Tok {
            f32x4 k[RM], q[RM], gate;
            float x;
        };
        const auto read = [&](int i) {
            const int t = MODE == SWEEP ? TT - 1 - i : i;
            Tok y;
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                y.k[m] = *reinterpret_cast<const f32x4 *>(&s.k[t][row_of(m, 0)]);
                if (MODE != KEEP) y.q[m] = *reinterpret_cast<const f32x4 *>(&s.q[t][row_of(m, 0)]);
            }
            y.gate = *reinterpret_cast<const f32x4 *>(s.gate[t]);
            y.x = s.v[t][GC * wave + c];
            return y;
        };
        const auto step = [&](const Tok &y, int i) {
            const int at = place + (MODE == SWEEP ? TT - 1 - i : i) * rowe;
            const float al = y.gate[0], be = y.gate[1];
            // four partial sums each: one would be a chain of dependent adds
            f32x4 pk4 = zero, pq4 = zero;
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                if (MODE == SWEEP) S[m] += (a.scale * y.x) * y.q[m];
                else S[m] *= al;
                pk4 += S[m] * y.k[m];
                if (MODE == FWD) pq4 += S[m] * y.q[m];
            }
            const float pk = sum_rows<GC>((pk4[0] + pk4[1]) + (pk4[2] + pk4[3]));
            const float pq = MODE == FWD ? sum_rows<GC>((pq4[0] + pq4[1]) + (pq4[2] + pq4[3])) : 0.f;
            const float res = MODE == SWEEP ? pk : y.x - pk;
            const float u = MODE == SWEEP ? -be * pk : be * res;
#pragma unroll
            for (int m = 0; m < RM; ++m) {
                S[m] += y.k[m] * u;
                if (MODE == SWEEP) S[m] *= al;
            }
            if (MODE == FWD) put(out0, at, a.scale * (pq + u * y.gate[2]), TO());
            if (MODE != FWD) put(out0, at, res, 0.f);
            if (MODE == SWEEP) put(out1, at, -u, TO());
        };
        // a token ahead, two sets of registers in turn
        Tok x = read(0);
#pragma unroll 2
        for (int i = 0; i < TT; i += 2) {
            const Tok y = read(i + 1);
            step(x, i);
            x = read((i + 2) % TT);
            step(y, i + 1);
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
__global__ __launch_bounds__((Shape<DK, DV, GC>::NT))
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
    if (blocks * Sh::NT >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    const dim3 grid((unsigned)blocks), block(Sh::NT);
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
    // 4 / 8 / 16 columns a wave: 32 chains of 1024 tokens 0.28 / 0.34 / 0.48 ms;
    // 128 chains 0.47 / 0.42 / 0.49 ms; 512 chains 1.72 / 1.33 / 1.18 ms.
    const int64_t columns = (int64_t)a.seq.n_seqs * a.Hv * DV;
    if constexpr (DK >= 64)
        if (columns < kFew) return launch_gc<TI, DK, DV, 4>(a, bwd);
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
