// Gated delta rule, backward: the gradients of one chunk of 64 tokens on the
// matrix cores (bf16 or 8-bit inputs, d_k and d_v of 64 or 128), all chunks in
// parallel.  The formulas are those at the top of gdr_grad.hip.
//
// A workgroup takes a (chunk, key head) and its value heads one after
// another, so that shared heads' gradients are summed in registers, in one
// order; each of its d_k / 16 waves owns 16 key channels of dq and dk.
// Everything is formed transposed, result rows = key channels and columns =
// tokens: the state's operands come straight from memory in the order the
// sweeps left them, decays and masks are per-lane scalars, and dq, dk go out
// 8 bytes at a time.
//
// Operands of the products that dg depends on are held in three bf16 parts
// and multiplied without the parts' products below 2^-24 (with two parts dg
// was off by 4e-6 of its norm, with three by 2e-7 to 6e-7: sums in fp32 are no
// better); dP and dN, which only dq and dk see (rounded to bf16), in two.
//
// Bound by the latencies between its phases: a workgroup has a compute unit's
// LDS to itself, the matrix cores are busy for 29% of the time and the vector
// ALU for 41%, and 2.0 GB of states, cotangents and rows go at 3.2 TB/s.  4
// sequences of 4096 tokens, 32 value heads of 128 x 128 on 16 key heads: 0.63
// ms, of which per workgroup and value head the products over the value
// columns take 40%, the pairs 12%, the products with the chunk's rows 9%,
// staging 6%, the state's part 5%, and the workgroup's start 10%.  Two waves
// for each block of channels (16 waves of 128 registers, half the tokens each)
// spill and take 1.37 times as long; states requested a step ahead gain
// nothing, nor does a workgroup that goes on to other chunks.
#include "gdr_chunk.h"

namespace gdr {
namespace {

constexpr int C = 64;

// waves, and value columns staged at a time
template <int DK, int DV>
struct Shape {
    static constexpr int NW = DK / 16;
    static constexpr int SW = DK == 128 ? DV : 64;
};

template <int DK, int DV>
struct alignas(16) GradSmem {
    static constexpr int NW = Shape<DK, DV>::NW, SW = Shape<DK, DV>::SW;
    bf16 q[C * DK], k[C * DK];
    union {
        bf16 rows[7][C * SW];                    // dO; U, Yb in three parts each
        bf16 mat[4][C * C];                      // dP hi, dP lo, dN hi, dN lo   [i][j]
    };
    float G[2][C], a[NW][C], b[NW][C], e[NW][C], rev[C], ls[NW];
};

// four rows (consecutive, from row on) of one column a lane; see lds_tr
template <int D>
__device__ __forceinline__ u32x2 tr4(const bf16 *m, int row, int c, int ln)
{
    return lds_tr(m + Swz<D>::at(row + (ln >> 2), c + 4 * (ln & 3)));
}
// transposed operand: lane = column c + ln, slots = rows row + 8 lg ..
template <int D>
__device__ __forceinline__ bf16x8 tr8(const bf16 *m, int row, int c, int ln, int lg)
{
    return join(tr4<D>(m, row + 8 * lg, c, ln), tr4<D>(m, row + 8 * lg + 4, c, ln));
}
template <int D>
__device__ __forceinline__ bf16x8 row8(const bf16 *m, int row, int c) { return lds8(m + Swz<D>::at(row, c)); }

// sum over the 16 lanes of equal lane / 16, in every one of them
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float x)
{
    x = dpp_add<0xb1>(x);        // quad_perm 1 0 3 2
    x = dpp_add<0x4e>(x);        // quad_perm 2 3 0 1
    x = dpp_add<0x141>(x);       // row_half_mirror
    return dpp_add<0x140>(x);    // row_mirror
}

// the three parts of eight values
__device__ __forceinline__ Parts<3> split8(f32x4 x, f32x4 y)
{
    Parts<3> r;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const u32x2 hx = pack4(x), hy = pack4(y);
        r.p[i] = join(hx, hy);
        if (i < 2) {
            x -= widen(hx);
            y -= widen(hy);
        }
    }
    return r;
}
// a b + c, both in three parts
__device__ __forceinline__ f32x4 mma33(const Parts<3> &a, const Parts<3> &b, f32x4 c)
{
    c = mma(a.p[0], b.p[2], c);
    c = mma(a.p[2], b.p[0], c);
    c = mma(a.p[1], b.p[1], c);
    c = mma(a.p[0], b.p[1], c);
    c = mma(a.p[1], b.p[0], c);
    return mma(a.p[0], b.p[0], c);
}

template <typename TI, int DK, int DV>
__global__ __launch_bounds__((Shape<DK, DV>::NW * WAVE), 2)
void gdr_grad_chunk_kernel(Args a)
{
    __shared__ GradSmem<DK, DV> s;
    constexpr int NW = Shape<DK, DV>::NW, SW = Shape<DK, DV>::SW, NT = NW * WAVE;
    constexpr int KS = DK / 32, VS = DV / 32;
    const int tid = threadIdx.x, lane = tid % WAVE;
    int ln = lane % 16, lg = lane / 16;
    // Cuts what follows loose from the lane indices before it: addresses and
    // masks made of them are then formed where they are used, and not kept in
    // registers from before the loop over the heads.
    const auto fresh = [&] { asm volatile("" : "+v"(ln), "+v"(lg)); };
    const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int64_t slot = blockIdx.x / a.Hk;
    const int hk = blockIdx.x % a.Hk, grp = a.Hv / a.Hk;
    int n, c;
    if (!find_chunk(a.seq, slot, C, n, c)) return;
    const Seq sq = seq_of(a.seq, n);
    const int64_t tok = __builtin_amdgcn_readfirstlane(sq.bos + c * C);
    const int nt = __builtin_amdgcn_readfirstlane(sq.len - c * C < C ? sq.len - c * C : C);
    // The 16 x 16 tiles on and below the diagonal of the two C x C matrices,
    // dP (with Q K^T) and dN (with K K^T), in the order (0, 0), (1, 0), (1, 1),
    // ...  A tile of dN costs six products a step, one of dP three.  Eight
    // waves: 0 .. 4 take a tile of both and one more of dP, 5 .. 7 two of dN
    // (7: one); four waves: two or three tiles of both.
    constexpr int NS = NW == 8 ? 2 : 3;
    int row_block[NS], col_block[NS];
    bool in_p[NS], in_n[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int t = NW == 4 ? wave + 4 * i : wave < 5 ? wave + 5 * i : 2 * wave - 5 + i;
        row_block[i] = (t > 0) + (t > 2) + (t > 5);
        col_block[i] = t - row_block[i] * (row_block[i] + 1) / 2;
        in_p[i] = NW == 4 ? t < 10 : wave < 5;
        in_n[i] = NW == 4 ? t < 10 : wave < 5 ? i == 0 : t < 10;
    }
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const Eye eye = make_eye(lane);
    // rows of dO, R and Ub for one stage of value columns of one head, a
    // thread's part; requested a stage ahead
    constexpr int TPR = NT / C, CPT = SW / TPR;          // threads a row, columns a thread (a multiple of 8)
    const int row = tid / TPR, cc = CPT * (tid % TPR);
    u32x4 ro[CPT / 8];
    f32x4 rr[CPT / 4], ru[CPT / 4];
    float rbeta = 0.f, rgate = 0.f;
    const auto request = [&](int hv, int v0) {
        const Rows<bf16> O(a.dO, nullptr, tok, nt, a.Hv, DV);
        const int rb = a.Hv * DV * 4;
        const rsrc_t br = make_rsrc(reinterpret_cast<const char *>(a.R) + tok * rb, nt * rb);
        const rsrc_t bu = make_rsrc(reinterpret_cast<const char *>(a.Ub) + tok * rb, nt * rb);
        const rsrc_t bb = make_rsrc(a.beta + tok * a.Hv, nt * a.Hv * 4), bg = make_rsrc(a.g + tok * a.Hv, nt * a.Hv * 4);
        const int e = ((row * a.Hv + hv) * DV + v0 + cc) * 4;
#pragma unroll
        for (int i = 0; i < CPT / 8; ++i) ro[i] = O.raw(e / 2, 8 * i);
#pragma unroll
        for (int i = 0; i < CPT / 4; ++i) {
            rr[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(br, e + 16 * i, 0, 0));
            ru[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(bu, e + 16 * i, 0, 0));
        }
        rbeta = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bb, (row * a.Hv + hv) * 4, 0, 0));
        if (v0 == 0) rgate = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bg, (lane * a.Hv + hv) * 4, 0, 0));
    };
    request(hk * grp, 0);
    {
        const Rows<TI> Q(a.q, a.qe, tok, nt, a.Hk, DK), K(a.k, a.ke, tok, nt, a.Hk, DK);
#pragma unroll
        for (int i = 0; i < C * DK / 8; i += NT) {
            const int row = (i + tid) / (DK / 8), ch = 8 * ((i + tid) % (DK / 8));
            const auto at = Rows<TI>::at(row, a.Hk, hk, DK, ch);
            *reinterpret_cast<bf16x8 *>(&s.q[Swz<DK>::at(row, ch)]) = Rows<TI>::bf(Q.raw(at, 0));
            *reinterpret_cast<bf16x8 *>(&s.k[Swz<DK>::at(row, ch)]) = Rows<TI>::bf(K.raw(at, 0));
        }
    }
    f32x4 dq[4] = {}, dk[4] = {};                // channels 16 wave + 4 lg + e of token 16 t + ln
    for (int h = 0; h < grp; ++h) {
        const int hv = hk * grp + h;
        fresh();
        if (wave == 0) {
            const double G = scan64<double>((double)floor_g(rgate) * LOG2E64);
            const float gh = (float)G;
            s.G[0][lane] = gh;
            s.G[1][lane] = (float)(G - (double)gh);
        }
        // products over the value columns
        f32x4 mp[NS] = {}, mn[NS] = {}, x1[4] = {}, x2[4] = {}, x3[4] = {}, ls = zero;
        float db = 0.f;
        const int64_t st = (slot * a.Hv + hv) * (int64_t)(DK * DV / 4) + wave * VS * 2 * WAVE + lane;     // in f32x4
        const f32x4 *Sc = reinterpret_cast<const f32x4 *>(a.Sc) + st, *Lc = reinterpret_cast<const f32x4 *>(a.Lc) + st;
#pragma unroll 1
        for (int v0 = 0; v0 < DV; v0 += SW) {
            __syncthreads();                     // what lies here has been read
#pragma unroll
            for (int i = 0; i < CPT / 8; ++i) {
                const int at = Swz<SW>::at(row, cc + 8 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) db += rr[2 * i][j] * ru[2 * i][j] + rr[2 * i + 1][j] * ru[2 * i + 1][j];
                *reinterpret_cast<bf16x8 *>(&s.rows[0][at]) = Rows<bf16>::bf(ro[i]);
                const Parts<3> U = split8(rbeta * rr[2 * i], rbeta * rr[2 * i + 1]);
                const Parts<3> Y = split8(rbeta * ru[2 * i], rbeta * ru[2 * i + 1]);
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    *reinterpret_cast<bf16x8 *>(&s.rows[1 + j][at]) = U.p[j];
                    *reinterpret_cast<bf16x8 *>(&s.rows[4 + j][at]) = Y.p[j];
                }
            }
            __syncthreads();
#pragma unroll 1
            for (int ks = 0; ks < SW / 32; ++ks) {
                const int vc = 32 * ks + 8 * lg;
                const auto rows3 = [&](int first, int row) {
                    const int at = Swz<SW>::at(row, vc);
                    return Parts<3>{{lds8(&s.rows[first][at]), lds8(&s.rows[first + 1][at]), lds8(&s.rows[first + 2][at])}};
                };
                const int t0 = (v0 / 32 + ks) * 2 * WAVE;
                const Parts<3> S = split8(__builtin_nontemporal_load(Sc + t0), __builtin_nontemporal_load(Sc + t0 + WAVE));
                const Parts<3> L = split8(__builtin_nontemporal_load(Lc + t0), __builtin_nontemporal_load(Lc + t0 + WAVE));
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    if (!in_p[i] && !in_n[i]) continue;
                    const int own = 16 * row_block[i] + ln;
                    const Parts<3> U = rows3(1, 16 * col_block[i] + ln);
                    if (in_p[i]) mp[i] = mma_by_parts<3>(U, row8<SW>(s.rows[0], own, vc), mp[i]);
                    if (in_n[i]) mn[i] = mma33(U, rows3(4, own), mn[i]);
                }
                ls = mma33(S, L, ls);            // its diagonal is wanted
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    x1[t] = mma_by_parts<3>(S, row8<SW>(s.rows[0], 16 * t + ln, vc), x1[t]);
                    x2[t] = mma33(S, rows3(4, 16 * t + ln), x2[t]);
                    x3[t] = mma33(L, rows3(1, 16 * t + ln), x3[t]);
                    // keeps the reads of all blocks from being hoisted into registers at once
                    if (t == 1) __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (v0 + SW < DV) request(hv, v0 + SW);
            else if (h + 1 < grp) request(hv + 1, 0);
        }
#pragma unroll
        for (int m = 1; m < TPR; m *= 2) db += __shfl_xor(db, m);
        if (tid % TPR == 0 && row < nt) a.dbeta[(tok + row) * a.Hv + hv] = db;
        // what goes through the state: the decay's dots, then dq and dk
        fresh();
        const int ch0 = 16 * wave + 4 * lg;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int i = 16 * t + ln;
            const float eg = exp2_two(s.G[0][i], s.G[1][i]);
            const float er = kda::fast_exp2((s.G[0][C - 1] - s.G[0][i]) + (s.G[1][C - 1] - s.G[1][i]));
            const f32x4 qv = widen(*reinterpret_cast<const u32x2 *>(&s.q[Swz<DK>::at(i, ch0)]));
            const f32x4 kv = widen(*reinterpret_cast<const u32x2 *>(&s.k[Swz<DK>::at(i, ch0)]));
            const f32x4 d1 = (a.scale * eg) * x1[t], d2 = eg * x2[t], d3 = er * x3[t];
            float da = 0.f, dbb = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                da += qv[e] * d1[e] - kv[e] * d2[e];
                dbb += kv[e] * d3[e];
            }
            dq[t] += d1;
            dk[t] += d3 - d2;
            da = sum_groups(da);
            dbb = sum_groups(dbb);
            if (lg == 0) {
                s.a[wave][i] = da;
                s.b[wave][i] = dbb;
            }
        }
        {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ln == 4 * lg + e) x = ls[e];
            x = sum_groups(sum16(x));
            if (lane == 0) s.ls[wave] = x;
        }
        __syncthreads();                         // the staged rows are read
        // the chunk's own pairs: lane row i of the row block, rows j of the tile
        fresh();
        if (tid < 256) {                         // tiles above the diagonal that are read below: zeros
            const int y = tid / 2 % 32, x = y + (y & 16);
            *reinterpret_cast<bf16x8 *>(&s.mat[tid / 64][Swz<C>::at(x, (x & 32) + 16 + 8 * (tid % 2))]) = bf16x8{};
        }
        float es[4] = {};
        bf16x8 ones, tri;                        // [1 | 1], [j < t | j < t]
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            ones[x] = (bf16)1.f;
            tri[x] = 4 * lg + (x & 3) < ln ? (bf16)1.f : (bf16)0.f;
        }
#pragma unroll
        for (int x = 0; x < NS; ++x) {
            if (!in_p[x] && !in_n[x]) continue;
            const int rb = row_block[x], cb = col_block[x], i = 16 * rb + ln, j = 16 * cb + 4 * lg;
            const f32x4 gjh = *reinterpret_cast<const f32x4 *>(&s.G[0][j]), gjl = *reinterpret_cast<const f32x4 *>(&s.G[1][j]);
            const float gih = s.G[0][i], gil = s.G[1][i];
            f32x4 pq = zero, pk = zero, E = zero, d;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const bf16x8 kj = row8<DK>(s.k, 16 * cb + ln, 32 * ks + 8 * lg);
                if (in_p[x]) pq = mma(kj, row8<DK>(s.q, i, 32 * ks + 8 * lg), pq);
                if (in_n[x]) pk = mma(kj, row8<DK>(s.k, i, 32 * ks + 8 * lg), pk);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = j + e <= i ? kda::fast_exp2((gih - gjh[e]) + (gil - gjl[e])) : 0.f;
            const auto put = [&](int m, f32x4 v) {
                const u32x2 vh = pack4(v);
                const int at = Swz<C>::at(i, j);
                *reinterpret_cast<u32x2 *>(&s.mat[m][at]) = vh;
                *reinterpret_cast<u32x2 *>(&s.mat[m + 1][at]) = pack4(v - widen(vh));
            };
            if (in_p[x]) {
                f32x4 v = (a.scale * d) * mp[x];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = j + e <= i ? v[e] : 0.f;
                    E[e] = j + e < i ? v[e] * pq[e] : 0.f;
                }
                put(0, v);
            }
            if (in_n[x]) {
                f32x4 v = -d * mn[x];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = j + e < i ? v[e] : 0.f;
                    E[e] += j + e < i ? v[e] * pk[e] : 0.f;
                }
                put(2, v);
            }
            // sum over j < t <= i of E_ij: E [j < t] by products with zeros
            // and ones (rows i of the tile, a lane's column t), then the rows
            // i >= t
            u32x2 ep[3];
            split3(E, eye, ep);
            const bf16x8 hm = join(ep[0], ep[1]), lo = join(ep[2], u32x2{0, 0});
            const f32x4 wt = mma(hm, tri, mma(lo, tri, zero)), wo = mma(hm, ones, mma(lo, ones, zero));
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                if (tb < cb || tb > rb) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = tb == cb ? wt[e] : wo[e];
                    es[tb] += tb < rb || 4 * lg + e >= ln ? w : 0.f;
                }
            }
        }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const float x = sum_groups(es[tb]);
            if (lg == 0) s.e[wave][16 * tb + ln] = x;
        }
        // the last wave has the least to do here: the sums over the chunk that
        // do not need the pairs
        float dg = 0.f;
        if (wave == NW - 1) {
            const auto at = [&](const float (*x)[C], int r) {
                float y = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) y += x[w][r];
                return y;
            };
            s.rev[lane] = scan64<float>(at(s.a, C - 1 - lane));
            const float before = scan64<float>(lane ? at(s.b, lane - 1) : 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) l += s.ls[w];
            dg = s.rev[C - 1 - lane] + before + exp2_two(s.G[0][C - 1], s.G[1][C - 1]) * l;
        }
        __syncthreads();
        // products with the chunk's own rows
        fresh();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const bf16x8 kt = tr8<DK>(s.k, 32 * x, 16 * wave, ln, lg), qt = tr8<DK>(s.q, 32 * x, 16 * wave, ln, lg);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = Swz<C>::at(16 * t + ln, 32 * x + 8 * lg);
#pragma unroll
                for (int part = 1; part >= 0; --part) {
                    if (x <= t / 2) {
                        dq[t] = mma(kt, lds8(&s.mat[part][at]), dq[t]);
                        dk[t] = mma(kt, lds8(&s.mat[2 + part][at]), dk[t]);
                    }
                    if (x >= t / 2) {
                        dk[t] = mma(qt, tr8<C>(s.mat[part], 32 * x, 16 * t, ln, lg), dk[t]);
                        dk[t] = mma(kt, tr8<C>(s.mat[2 + part], 32 * x, 16 * t, ln, lg), dk[t]);
                    }
                }
            }
        }
        if (wave == NW - 1) {
#pragma unroll
            for (int w = 0; w < NW; ++w) dg += s.e[w][lane];
            if (lane < nt) a.dg[(tok + lane) * a.Hv + hv] = dg;
        }
    }
    const int rb = a.Hk * DK * 2;
    const rsrc_t oq = make_rsrc(static_cast<char *>(a.dq) + tok * rb, nt * rb), ok = make_rsrc(static_cast<char *>(a.dkey) + tok * rb, nt * rb);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int off = (16 * t + ln) * rb + (hk * DK + 16 * wave + 4 * lg) * 2;
        __builtin_amdgcn_raw_buffer_store_b64(pack4(dq[t]), oq, off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(pack4(dk[t]), ok, off, 0, 0);
    }
}

template <typename TI, int DK, int DV>
hipError_t launch_t(const Args &a)
{
    const int64_t blocks = bwd_slots(a.seq.n_seqs, a.seq.n_tokens, C) * a.Hk;
    constexpr int NT = Shape<DK, DV>::NW * WAVE;
    if (blocks * NT >= ((int64_t)1 << 32)) return hipErrorInvalidValue;   // grid size limit
    hipLaunchKernelGGL((gdr_grad_chunk_kernel<TI, DK, DV>), dim3((unsigned)blocks), dim3(NT), 0, a.stream, a);
    return hipGetLastError();
}

template <typename TI>
hipError_t dispatch(const Args &a)
{
    if (a.dk == 128) return a.dv == 128 ? launch_t<TI, 128, 128>(a) : launch_t<TI, 128, 64>(a);
    return a.dv == 128 ? launch_t<TI, 64, 128>(a) : launch_t<TI, 64, 64>(a);
}

}  // namespace

hipError_t launch_chunk_grad(const Args &a)
{
    return a.in == In::BF16 ? dispatch<bf16>(a) : dispatch<e4m3>(a);
}

}  // namespace gdr
