// Gated linear recurrence, forward.
//
// A tile is 128 tokens by 64 V channels, one workgroup: each of eight waves
// takes 16 tokens in registers (each lane V channels), forms their factors
// and inputs, and folds them into one map h -> A h + B.  The waves' maps meet
// in the LDS, the tile's goes to the tiles behind it (glr_index.h), the state
// that comes in is looked up from the tiles before it, and every wave runs
// its 16 tokens once more from the state that reaches it and stores them.
// Everything is read and written once, by one launch, however the batch is
// cut into sequences: a sequence's first token forgets what came before it,
// so borders cost nothing elsewhere.
//
// Bound by HBM where the factors are given (65536 tokens of 4096 channels,
// bf16: 2.15 GB in 349 us, 6.2 TB/s), by HBM and the vector ALU together where
// the gates are formed (20011 tokens, bf16: 0.66 GB in 134 us, 4.9 TB/s; 32 vector
// instructions an element, which take 54% of it).  One long sequence of few
// channels is bound by the chain, 128 looks at four tiles in a row: 65536 tokens of
// 64 channels take 125 us, of 512 128.  128 tokens: enough that the words of
// the chain (24 bytes a tile and channel) and a workgroup's latencies are a
// few percent, and two workgroups fit a compute unit, one loading while the
// other forms its gates.  (Where these take 138 us, 64 tokens by eight waves
// take 154 and by four 143; plain, 65536 tokens, 378, 440 and 434.)
#include "glr_tiles.h"

namespace glr {
namespace {

constexpr int NW = kScanWaves, K = kScanTokens, C = kScanTile, NT = NW * WAVE;

template <typename T, bool GATED, int V>
__global__ __launch_bounds__(NT, 4) void glr_scan_kernel(Args a, Chain chain)
{
    typedef Row<T, V> R;
    typedef Row<float, V> RF;
    __shared__ int s_tile, s_first[C], s_last[C];
    __shared__ Map s_map[NW][WAVE * V];
    __shared__ float s_in[WAVE * V];
    const int tid = threadIdx.x, lane = tid % WAVE, w = __builtin_amdgcn_readfirstlane(tid / WAVE), D = a.D;
    const gdr::SeqArgs sa = seq_args(a);
    const int total = total_tokens(sa);
    const int idx = blockIdx.x;
    if (idx >= chain.tiles * chain.blocks) {
        empty_states(sa, idx - chain.tiles * chain.blocks, D, a.h0, a.h_T, NT);
        return;
    }
    const int block = block_of(chain, idx);
    if (tid == 0) s_tile = take(chain, block);
    const Edges few = few_edges(sa, lane);
    if (tid < C) s_first[tid] = s_last[tid] = -1;
    __syncthreads();
    const int taken = __builtin_amdgcn_readfirstlane(s_tile);
    const int tile = taken, t0 = tile * C, c = block * WAVE * V + lane * V;
    const bool active = c < D;
    const int cc = active ? c : 0;
    uint64_t *const p = chain.words + (int64_t)tile * chain.pitch + block * (WAVE * V) + lane;
    const bool more = tile + 1 < chain.tiles;       // a tile behind this one
    if (t0 >= total) {
        if (more) put_nothing<V>(p, active);
        return;
    }
    const int count = total - t0 < C ? total - t0 : C;
    const int tw = t0 + w * K, mine = count - w * K < 0 ? 0 : count - w * K < K ? count - w * K : K;

    const unsigned ct = active ? c * (unsigned)sizeof(T) : kNowhere, cf = active ? c * 4u : kNowhere;
    const Rows<T, V> bx(a.x, tw, mine, D), br(a.r, tw, GATED ? mine : 0, D), bi(a.i, tw, GATED ? mine : 0, D);
    const Rows<float, V> bg(a.g, tw, GATED ? 0 : mine, D);

    typename R::raw rx[K], rr[K], ri[K];
    typename RF::raw rg[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        rx[k] = bx.ld(k, ct);
        if constexpr (GATED) {
            rr[k] = br.ld(k, ct);
            ri[k] = bi.ld(k, ct);
        } else
            rg[k] = bg.ld(k, cf);
    }
    float nr[V];
    if constexpr (GATED) {
        const typename RF::raw rate = ld<V>(a.rate + cc);
#pragma unroll
        for (int j = 0; j < V; ++j) nr[j] = -RF::get(rate, j);
    }
    if (w == 0) mark_borders(Lane{lane}, sa, [&](int) { return few; }, t0, C, s_first, s_last);
    __syncthreads();
    const uint64_t starts = __ballot(lane < K && s_first[w * K + lane % K] >= 0);
    const uint64_t ends = __ballot(lane < K && s_last[w * K + lane % K] >= 0);

    float al[K][V], u[K][V];
    const auto form = [&](auto near) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if constexpr (GATED) {
                    const Gates g = gates<decltype(near)::value>(R::get(rr[k], j), R::get(ri[k], j), nr[j]);
                    al[k][j] = g.a;
                    u[k][j] = g.b * R::get(rx[k], j);
                } else {
                    al[k][j] = decay(RF::get(rg[k], j));
                    u[k][j] = R::get(rx[k], j);
                }
            }
    };
    if (GATED && all_near<V>(nr)) form(std::true_type{});
    else form(std::false_type{});
    Map m[V];
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = Map{1.f, 0.f};
    const bool plain = starts == 0 && mine == K;
    if (plain) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = Map{m[j].A * al[k][j], __builtin_fmaf(al[k][j], m[j].B, u[k][j])};
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool start = starts >> k & 1;
            if (start && a.h0) {
                const int n = __builtin_amdgcn_readfirstlane(s_first[w * K + k]);
                const typename RF::raw h0 = ld<V>(a.h0 + (int64_t)n * D + cc);
#pragma unroll
                for (int j = 0; j < V; ++j) u[k][j] = __builtin_fmaf(al[k][j], RF::get(h0, j), u[k][j]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (k >= mine) {
                    al[k][j] = 1.f;
                    u[k][j] = 0.f;
                }
                m[j] = start ? Map{kForget, u[k][j]} : Map{m[j].A * al[k][j], __builtin_fmaf(al[k][j], m[j].B, u[k][j])};
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s_map[w][lane * V + j] = m[j];
    __syncthreads();

    if (w == 0) {
#pragma unroll
        for (int i = 1; i < NW; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) m[j] = after(s_map[i][lane * V + j], m[j]);
        const bool alone = tile == 0 || s_first[0] >= 0;        // nothing comes in
        float in[V];
        if (alone) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                in[j] = 0.f;
                if (more && active) put(p + j * kLanes, Map{kForget, m[j].B});
            }
        } else {
            if (more && active)
#pragma unroll
                for (int j = 0; j < V; ++j) put(p + j * kLanes, m[j]);
            look_back<8 / V, V>(p - chain.pitch, -(int64_t)chain.pitch, tile, active, in);
            if (more && active)
#pragma unroll
                for (int j = 0; j < V; ++j) put(p + j * kLanes, Map{kForget, m[j](in[j])});
        }
#pragma unroll
        for (int j = 0; j < V; ++j) s_in[lane * V + j] = in[j];
    }
    __syncthreads();

    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        h[j] = s_in[lane * V + j];
        for (int i = 0; i < w; ++i) h[j] = s_map[i][lane * V + j](h[j]);
    }
    if (!active || mine == 0) return;
    if (a.kept && w * K % kKept == 0) st<V>(a.kept + (int64_t)(tw / kKept) * D + c, h);
    const Rows<T, V> bh(a.h, tw, mine, D);
    if (plain && !ends) {
        if (!a.h) return;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = __builtin_fmaf(al[k][j], h[j], u[k][j]);
            bh.st(k, ct, h);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k >= mine) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = starts >> k & 1 ? u[k][j] : __builtin_fmaf(al[k][j], h[j], u[k][j]);
            if (a.h) bh.st(k, ct, h);
            if (a.h_T && (ends >> k & 1)) {
                const int n = __builtin_amdgcn_readfirstlane(s_last[w * K + k]);
                st<V>(a.h_T + (int64_t)n * D + c, h);
            }
        }
    }
}

// tickets and words, 16 bytes at a time (both are whole lines)
__global__ __launch_bounds__(256) void glr_clear_kernel(uint64_t *p, int64_t words)
{
    typedef uint64_t u2 __attribute__((ext_vector_type(2)));
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; 2 * i < words; i += (int64_t)gridDim.x * 256)
        reinterpret_cast<u2 *>(p)[i] = u2{kEmpty, kEmpty};
}

template <typename T, bool GATED>
void launch_v(const Args &a, const Chain &ch, int V, hipStream_t s)
{
    const dim3 grid((unsigned)ch.items);
    if constexpr (kPairs<T, GATED>)
        if (V == 2) {
            hipLaunchKernelGGL((glr_scan_kernel<T, GATED, 2>), grid, dim3(NT), 0, s, a, ch);
            return;
        }
    hipLaunchKernelGGL((glr_scan_kernel<T, GATED, 1>), grid, dim3(NT), 0, s, a, ch);
}

}  // namespace

hipError_t clear_chain(const Chain &c, hipStream_t s)
{
    if (!c.tickets) return hipSuccess;
    uint64_t *const p = reinterpret_cast<uint64_t *>(c.tickets);
    const int64_t words = c.words - p + (int64_t)c.tiles * c.pitch, blocks = (words + 511) / 512;
    hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s, p, words);
    return hipGetLastError();
}

hipError_t launch_fwd(const Args &a)
{
    const Plan p = plan_scan(a);
    if (p.chain.items == 0) return hipSuccess;
    const hipError_t e = clear_chain(p.chain, a.stream);
    if (e != hipSuccess) return e;
    if (a.bf16) a.gated ? launch_v<bf16, true>(a, p.chain, p.V, a.stream) : launch_v<bf16, false>(a, p.chain, p.V, a.stream);
    else a.gated ? launch_v<float, true>(a, p.chain, p.V, a.stream) : launch_v<float, false>(a, p.chain, p.V, a.stream);
    return hipGetLastError();
}

}  // namespace glr
