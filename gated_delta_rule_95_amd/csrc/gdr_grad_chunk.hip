// Gated delta rule, backward: the gradients of one chunk of 64 tokens on the
// matrix cores (bf16 or 8-bit inputs, d_k and d_v of 64 or 128), all chunks in
// parallel.  The formulas are those at the top of gdr_grad.hip.
//
// A workgroup takes a (chunk, key head) and its value heads one after
// another, so that shared heads' gradients are summed in registers, in one
// order; each of its d_k / 16 waves owns 16 key channels of dq and dk.  Everything is formed transposed, result rows = key channels and
// columns = tokens: the state's operands come straight from memory in the
// order the sweeps left them, decays and masks are per-lane scalars, and dq,
// dk go out 8 bytes at a time.
//
// Operands of the products that dg depends on are held in three bf16 parts
// and multiplied without the parts' products below 2^-24 (with two parts dg
// was off by 4e-6 of its norm, with three by 6e-7: sums in fp32 are little
// better); dP and dN, which only dq and dk see, in two.
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
    float G[2][C], a[NW][C], b[NW][C], e[8][C], rev[C], ls[NW];
};

__device__ __forceinline__ bool find_chunk(const SeqArgs &s, int64_t slot, int &n, int &c)
{
    // slots of sequence n start at edge(n) / C + n, which grows with n
    int lo = 0, hi = s.n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((int64_t)(seq_edge(s, mid) / C) + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    n = lo;
    c = (int)(slot - (seq_edge(s, lo) / C + lo));
    return c >= 0 && (int64_t)c * C < seq_of(s, lo).len;
}

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

template <typename T, int CTRL, int ROWS>
__device__ __forceinline__ T scan_step(T x);
template <typename T>
__device__ __forceinline__ T scan64(T x)
{
    x = scan_step<T, 0x111, 0xf>(x);
    x = scan_step<T, 0x112, 0xf>(x);
    x = scan_step<T, 0x114, 0xf>(x);
    x = scan_step<T, 0x118, 0xf>(x);
    x = scan_step<T, 0x142, 0xa>(x);
    return scan_step<T, 0x143, 0xc>(x);
}
template <typename T, int CTRL, int ROWS>
__device__ __forceinline__ T scan_step(T x)
{
    if constexpr (sizeof(T) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
        return x + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
    } else
        return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, ROWS, 0xf, false));
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
    if (!find_chunk(a.seq, slot, n, c)) return;
    const Seq sq = seq_of(a.seq, n);
    const int64_t tok = __builtin_amdgcn_readfirstlane(sq.bos + c * C);
    const int nt = __builtin_amdgcn_readfirstlane(sq.len - c * C < C ? sq.len - c * C : C);
    // Rows of the two C x C matrices: kind 0 is dP (with Q K^T), 1 is dN (with
    // K K^T); eight waves take one row block of one kind each, four waves one
    // of both.  Block rows are formed whole: the longest sets the time.
    constexpr int NKD = 8 / NW;
    const auto kind_of = [&](int i) { return NKD == 2 ? i : wave >> 2; };
    const auto block_of = [&](int i) { return kind_of(i) ? 3 - (wave & 3) : wave & 3; };
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
            const double G = scan64<double>((double)floor_g(rgate) * (double)LOG2E);
            const float gh = (float)G;
            s.G[0][lane] = gh;
            s.G[1][lane] = (float)(G - (double)gh);
        }
        // products over the value columns
        f32x4 mat[NKD][4] = {}, x1[4] = {}, x2[4] = {}, x3[4] = {}, ls = zero;
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
                const int t0=(v0/32+ks)*2*WAVE; const Parts<3> S = split8(__builtin_nontemporal_load(Sc + t0), __builtin_nontemporal_load(Sc + t0 + WAVE)), L = split8(__builtin_nontemporal_load(Lc + t0), __builtin_nontemporal_load(Lc + t0 + WAVE));
#pragma unroll
                for (int i = 0; i < NKD; ++i) {
                    const int own = 16 * block_of(i) + ln;
                    if (kind_of(i) == 0) {
                        const bf16x8 x = row8<SW>(s.rows[0], own, vc);
#pragma unroll
                        for (int b = 0; b < 4; ++b) mat[i][b] = mma_by_parts<3>(rows3(1, 16 * b + ln), x, mat[i][b]);
                    } else {
                        const Parts<3> x = rows3(4, own);
#pragma unroll
                        for (int b = 0; b < 4; ++b) mat[i][b] = mma33(rows3(1, 16 * b + ln), x, mat[i][b]);
                    }
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
            const float eg = kda::fast_exp2(s.G[0][i]);
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
#pragma unroll
        for (int kd = 0; kd < NKD; ++kd) {
            fresh();
            const int kind = kind_of(kd), rb = block_of(kd), i = 16 * rb + ln;
            const float gih = s.G[0][i], gil = s.G[1][i];
            f32x4 (&E)[4] = mat[kd];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                f32x4 pair = zero;
                const bf16 *x = kind == 0 ? s.q : s.k;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    pair = mma(row8<DK>(s.k, 16 * b + ln, 32 * ks + 8 * lg), row8<DK>(x, i, 32 * ks + 8 * lg), pair);
                const int j = 16 * b + 4 * lg;
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float d = kda::fast_exp2((gih - s.G[0][j + e]) + (gil - s.G[1][j + e]));
                    v[e] = (kind == 0 ? a.scale : -1.f) * d * mat[kd][b][e];
                    if (kind == 0 ? j + e > i : j + e >= i) v[e] = 0.f;
                    E[b][e] = j + e < i ? v[e] * pair[e] : 0.f;
                }
                const u32x2 vh = pack4(v), vl = pack4(v - widen(vh));
                const int at = Swz<C>::at(i, j);
                *reinterpret_cast<u32x2 *>(&s.mat[2 * kind][at]) = vh;
                *reinterpret_cast<u32x2 *>(&s.mat[2 * kind + 1][at]) = vl;
            }
            // sum over j < t <= i of E_ij: [j < t] E by products with zeros
            // and ones, then the rows i >= t
            const Parts<3> e01 = split_pair<3>(E[0], E[1], eye), e23 = split_pair<3>(E[2], E[3], eye);
            bf16x8 ones, tri0, tri1;             // all; [j < t | 0]; [1 | j < t]
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const bf16 lt = 4 * lg + (x & 3) < ln ? (bf16)1.f : (bf16)0.f;
                ones[x] = (bf16)1.f;
                tri0[x] = x < 4 ? lt : (bf16)0.f;
                tri1[x] = x < 4 ? (bf16)1.f : lt;
            }
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                f32x4 w = mma_parts<3>(tb == 0 ? tri0 : tb == 1 ? tri1 : ones, e01, zero);
                if (tb >= 2) w = mma_parts<3>(tb == 2 ? tri0 : tri1, e23, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * tb + 4 * lg + e;
                    const float x = sum16(i >= t ? w[e] : 0.f);
                    if (ln == 0) s.e[4 * kind + rb][t] = x;
                }
            }
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
        if (wave == 0) {
            const auto at = [&](const float (*x)[C], int r) {
                float y = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) y += x[w][r];
                return y;
            };
            s.rev[lane] = scan64<float>(at(s.a, C - 1 - lane));
            const float before = scan64<float>(lane ? at(s.b, lane - 1) : 0.f);
            float e = 0.f, l = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r) e += s.e[r][lane];
#pragma unroll
            for (int w = 0; w < NW; ++w) l += s.ls[w];
            if (lane < nt)
                a.dg[(tok + lane) * a.Hv + hv] = s.rev[C - 1 - lane] + before + e + kda::fast_exp2(s.G[0][C - 1]) * l;
        }
        if (h + 1 < grp) __syncthreads();        // the sums are read
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
