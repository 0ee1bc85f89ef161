// Host-only sanitizer driver (AddressSanitizer + UndefinedBehaviorSanitizer) of
// the C-ABI layers of the gated linear recurrence and of the state pools, and
// of the arithmetic that cuts a call into tiles and its workspace into parts.
//
// Links glr_api.cpp and pool_api.cpp (and kda_api.cpp, whose error state they
// share), compiled as plain host C++, against stub launchers that record their
// arguments instead of touching a GPU, up to the largest sizes the headers
// allow.  An undefined operation or out-of-bounds access aborts the run; the
// pytest wrapper checks for a clean exit.
#include <cstdio>
#include <cstring>
#include <vector>

#include "glr.h"
#include "glr_plan.h"
#include "kda_launch.h"
#include "pool.h"
#include "pool_launch.h"

namespace kda {
size_t prefill_workspace_bytes(const PrefillArgs &) { return 0; }
hipError_t launch_prefill(const PrefillArgs &) { return hipSuccess; }
hipError_t launch_decode(const DecodeArgs &) { return hipSuccess; }
size_t bwd_part_floats(int32_t d_k, int32_t d_v) { return (size_t)d_k * d_v; }
hipError_t launch_bwd(const BwdArgs &) { return hipSuccess; }
hipError_t launch_spec(const SpecArgs &) { return hipSuccess; }
}  // namespace kda

static hipError_t result = hipSuccess;
static int calls;

namespace glr {
static Args last;
static DecodeArgs last_decode;
hipError_t launch_fwd(const Args &a) { ++calls; last = a; return result; }
hipError_t launch_bwd(const Args &a) { ++calls; last = a; return result; }
hipError_t launch_decode(const DecodeArgs &a) { ++calls; last_decode = a; return result; }
}  // namespace glr

namespace pool {
static Pairs last;
static bool zeros;
static int taken, freed, planned;
hipError_t launch_copy(const pool_rows *from, const pool_rows *to, int32_t n_pools, const Pairs &p, hipStream_t)
{
    ++calls;
    last = p;
    zeros = !from;
    for (int i = 0; i < n_pools; ++i)
        if (!to[i].base || (from && from[i].row_bytes != to[i].row_bytes)) return hipErrorInvalidValue;
    return result;
}
hipError_t launch_take(const pool_rows *pools, int32_t n_pools, uint8_t *, int32_t, const int32_t *src, int32_t, int32_t *,
                       hipStream_t)
{
    ++taken;
    zeros = !src;
    for (int i = 0; i < n_pools; ++i)
        if (!pools[i].base) return hipErrorInvalidValue;
    return result;
}
hipError_t launch_free(uint8_t *, int32_t, const int32_t *, int32_t, hipStream_t) { ++freed; return result; }
hipError_t launch_plan(uint8_t *, int32_t, int32_t *, int64_t, int32_t *, const Moves &, hipStream_t) { ++planned; return result; }
}  // namespace pool

static int failures = 0;
#define EXPECT(cond)                                                              \
    do {                                                                          \
        if (!(cond)) {                                                            \
            std::fprintf(stderr, "%s:%d: expectation failed: %s (last error: %s)\n", \
                         __FILE__, __LINE__, #cond, kda_last_error());            \
            ++failures;                                                           \
        }                                                                         \
    } while (0)

// never dereferenced by the host layer: addresses far enough apart for the
// largest tensors (2^55 bytes)
static char *at(int i, size_t off = 0) { return reinterpret_cast<char *>(((uintptr_t)i << 56) + off); }
template <typename T> static T *p(int i, size_t off = 0) { return reinterpret_cast<T *>(at(i, off)); }

struct Call {
    int32_t n = 2, D = 100;
    int64_t N = 300;
    kda_dtype t = KDA_BF16;
    bool gated = true;
    const int32_t *cu = nullptr;
    float *kept = nullptr;
    size_t off = 0, ws_bytes = ~(size_t)0 >> 8;
    kda_status fwd() const
    {
        void *ws = at(20);
        return gated ? glr_fwd_scan_gated(at(1, off), at(2), at(3), p<float>(4), p<float>(5), cu, n, N, D, t, at(6), p<float>(7),
                                          kept, ws, ws_bytes, nullptr)
                     : glr_fwd_scan(at(1, off), p<float>(4), p<float>(5), cu, n, N, D, t, at(6), p<float>(7), kept, ws, ws_bytes,
                                    nullptr);
    }
    kda_status bwd() const
    {
        void *ws = at(20);
        return gated ? glr_bwd_scan_gated(at(1, off), at(2), at(3), p<float>(4), p<float>(5), cu, n, N, D, t, kept, at(8),
                                          p<float>(9), at(10), at(11), at(12), p<float>(13), p<float>(14), ws, ws_bytes, nullptr)
                     : glr_bwd_scan(at(1, off), p<float>(4), p<float>(5), cu, n, N, D, t, kept, at(8), p<float>(9), at(10),
                                    p<float>(13), p<float>(14), ws, ws_bytes, nullptr);
    }
};

// what a chain is handed lies in the workspace and can be launched
static void check_chain(const glr::Plan &q, const char *ws, size_t bytes, int64_t N, int32_t D, int tile, int threads)
{
    const glr::Chain &c = q.chain;
    EXPECT((int64_t)c.tiles * tile >= N && ((int64_t)c.tiles - 1) * tile < (N ? N : 1));
    EXPECT((int64_t)c.blocks * 64 * q.V >= D && ((int64_t)c.blocks - 1) * 64 * q.V < D);
    EXPECT((uint64_t)c.items * threads < (uint64_t)1 << 32 && c.items >= (int64_t)c.tiles * c.blocks);
    if (!c.tickets) {
        EXPECT(c.tiles <= 1);
        return;
    }
    EXPECT((char *)c.tickets >= ws && (char *)c.tickets + ((size_t)c.blocks - 1) * glr::kTicket + 4 <= (char *)c.words);
    EXPECT(c.pitch >= D && c.pitch == c.blocks * 64 * q.V);
    EXPECT((char *)(c.words + (size_t)c.tiles * c.pitch) <= ws + bytes);
}

int main()
{
    Call c;
    EXPECT(c.fwd() == KDA_OK && calls == 1 && glr::last.seqlen == 150 && glr::last.gated && glr::last.bf16);
    EXPECT(c.bwd() == KDA_OK && calls == 2);
    c.gated = false;
    c.t = KDA_F32;
    EXPECT(c.fwd() == KDA_OK && c.bwd() == KDA_OK && !glr::last.gated && !glr::last.bf16);
    for (int64_t N : {(int64_t)0, (int64_t)1, (int64_t)31, (int64_t)32, (int64_t)33, (int64_t)128, (int64_t)129, (int64_t)300,
                      (int64_t)100000, ((int64_t)1 << 31) - 256})
        for (int32_t D : {1, 2, 63, 64, 65, 128, 129, 1001, 4096, 8190, (1 << 24) - 1})
            for (int mode = 0; mode < 8; ++mode) {
                Call x;
                x.N = N; x.D = D; x.gated = mode & 1; x.t = mode & 2 ? KDA_BF16 : KDA_F32; x.off = mode & 4 ? 4 : 0; x.n = 1;
                static const int32_t some = 0;
                x.cu = mode & 4 ? &some : nullptr;
                const bool fits = (N + 63) / 64 * ((D + 63) / 64) < (1 << 22) && N * D < (int64_t)1 << 40;
                x.ws_bytes = glr_fwd_workspace_bytes(N, D);
                const int before = calls;
                EXPECT((x.fwd() == KDA_OK) == fits);
                if (!fits) {
                    EXPECT(calls == before && x.ws_bytes == 0 && glr_bwd_workspace_bytes(N, D) == 0 && glr_kept_bytes(N, D) == 0);
                    continue;
                }
                EXPECT(x.ws_bytes % 256 == 0);
                check_chain(glr::plan_scan(glr::last), at(20), x.ws_bytes, N, D, 128, 512);
                if (x.ws_bytes) {
                    x.ws_bytes -= 1;
                    EXPECT(x.fwd() == KDA_ERR_INVALID_ARG);
                }
                x.ws_bytes = glr_bwd_workspace_bytes(N, D);
                EXPECT(x.bwd() == KDA_OK && x.ws_bytes % 256 == 0);
                const glr::Args &a = glr::last;
                const glr::GradParts w(a);
                const char *ws = at(20);
                const glr::Plan q = glr::plan_grad(a, w.chain);
                check_chain(q, (char *)w.chain, ws + x.ws_bytes - (char *)w.chain, N, D, glr::grad_tile(a.gated, q.V),
                            64 * glr::grad_waves(a.gated, q.V));
                EXPECT((char *)w.kept == ws && glr_kept_bytes(N, D) <= (size_t)((char *)w.part - ws));
                EXPECT((size_t)q.chain.tiles * D * 4 <= (size_t)((char *)w.chain - (char *)w.part));
                // the forward that forms the kept states again
                glr::Args f = a;
                f.ws = w.chain;
                check_chain(glr::plan_scan(f), (char *)w.chain, ws + x.ws_bytes - (char *)w.chain, N, D, 128, 512);
                if (x.ws_bytes) {
                    x.ws_bytes -= 1;
                    EXPECT(x.bwd() == KDA_ERR_INVALID_ARG);
                }
            }
    // many sequences of nothing
    c = Call();
    c.N = 0; c.n = (1 << 27) - 1; c.D = 1;
    EXPECT(c.fwd() == KDA_OK && (uint64_t)glr::plan_scan(glr::last).chain.items * 512 < (uint64_t)1 << 32);
    c.n = 1 << 27;
    EXPECT(c.fwd() == KDA_ERR_INVALID_ARG && c.bwd() == KDA_ERR_INVALID_ARG);
    c.n = -0x7fffffff - 1;
    EXPECT(c.fwd() == KDA_ERR_INVALID_ARG && c.bwd() == KDA_ERR_INVALID_ARG);
    c.n = 0;
    EXPECT(c.fwd() == KDA_OK && c.bwd() == KDA_OK && glr::plan_grad(glr::last, nullptr).chain.items == 0);
    result = hipErrorInvalidValue;
    c = Call();
    EXPECT(c.fwd() == KDA_ERR_HIP && c.bwd() == KDA_ERR_HIP && std::strstr(kda_last_error(), "glr_bwd_scan_gated"));
    result = hipSuccess;

    // decode
    const auto dec = [](int32_t N, int32_t slots, int32_t D, const int32_t *s) {
        return glr_decode_step_gated(at(1), at(2), at(3), p<float>(4), p<float>(5), s, slots, N, D, KDA_BF16, at(6), nullptr);
    };
    EXPECT(dec(4, 4, 100, nullptr) == KDA_OK && glr::last_decode.gated);
    EXPECT(dec(5, 4, 100, nullptr) == KDA_ERR_INVALID_ARG && dec(5, 4, 100, p<int32_t>(7)) == KDA_OK);
    EXPECT(dec(0x7fffffff, 4, 1, p<int32_t>(7)) == KDA_ERR_INVALID_ARG && dec(4, 0x7fffffff, 513, p<int32_t>(7)) == KDA_ERR_INVALID_ARG);
    EXPECT(dec(4, 0x7fffffff, 511, p<int32_t>(7)) == KDA_OK && dec(0, 0, 1, nullptr) == KDA_OK);

    // pools
    std::vector<pool_rows> a(40), b(40);
    const size_t far = (size_t)1 << 48;
    for (int i = 0; i < 40; ++i) {
        a[i] = pool_rows{at(30, i * far), (size_t)i + 1};
        b[i] = pool_rows{at(31, i * far), (size_t)i + 1};
    }
    uint8_t *used = p<uint8_t>(1);
    int32_t *src = p<int32_t>(2), *dst = p<int32_t>(3);
    EXPECT(pool_copy(a.data(), b.data(), 40, 100, 50, src, dst, 7, nullptr) == KDA_OK && !pool::zeros && pool::last.n == 7 &&
           pool::last.from_slots == 100 && pool::last.to_slots == 50);
    EXPECT(pool_copy(a.data(), a.data(), 40, 100, 100, src, dst, 7, nullptr) == KDA_OK);
    EXPECT(pool_alloc(a.data(), 40, used, 100, 7, dst, nullptr) == KDA_OK && pool::zeros && pool::taken == 1);
    EXPECT(pool_fork(a.data(), 40, used, 100, src, 7, dst, nullptr) == KDA_OK && !pool::zeros && pool::taken == 2);
    EXPECT(pool_free(used, 100, src, 7, nullptr) == KDA_OK && pool::freed == 1);
    b[3].row_bytes = 5;
    EXPECT(pool_copy(a.data(), b.data(), 40, 100, 50, src, dst, 7, nullptr) == KDA_ERR_INVALID_ARG);
    b[3] = a[2];
    EXPECT(pool_copy(a.data(), b.data(), 40, 100, 50, src, dst, 7, nullptr) == KDA_ERR_INVALID_ARG);
    // the largest rows and counts
    pool_rows big{at(30), (size_t)1 << 22};
    EXPECT(pool_fork(&big, 1, used, (1 << 24) - 1, src, 1 << 24, dst, nullptr) == KDA_OK);
    EXPECT(pool_fork(&big, 1, used, 1 << 24, src, 1, dst, nullptr) == KDA_ERR_INVALID_ARG);
    big.row_bytes = (size_t)1 << 40;
    EXPECT(pool_fork(&big, 1, used, 63, src, 1, dst, nullptr) == KDA_OK);
    EXPECT(pool_fork(&big, 1, used, 64, src, 1, dst, nullptr) == KDA_ERR_INVALID_ARG);
    big.row_bytes = ~(size_t)0;
    EXPECT(pool_fork(&big, 1, used, 2, src, 1, dst, nullptr) == KDA_ERR_INVALID_ARG);
    // a compaction's workspace
    for (int32_t n : {0, 1, 2, 3, 127, 128, 129, 1000, 1 << 24}) {
        const size_t need = pool_compact_workspace_bytes(n);
        const pool::Moves m(at(5), n);
        EXPECT(need % 256 == 0 && (char *)m.count == at(5) && (char *)(m.count + 1) <= (char *)m.src);
        EXPECT((char *)(m.src + n / 2) <= (char *)m.dst && (char *)(m.dst + n / 2) <= at(5) + need);
        EXPECT(pool_compact(nullptr, 0, used, n, p<int32_t>(4), 9, p<int32_t>(6), at(5), need, nullptr) == KDA_OK);
        EXPECT(pool_compact(nullptr, 0, used, n, p<int32_t>(4), 9, p<int32_t>(6), at(5), need - 1, nullptr) == KDA_ERR_INVALID_ARG);
    }
    const int before = calls;
    EXPECT(pool_compact(a.data(), 2, used, 1, nullptr, 0, p<int32_t>(6), at(5), 4096, nullptr) == KDA_OK && calls == before);
    EXPECT(pool_compact(a.data(), 2, used, 2, nullptr, 0, p<int32_t>(6), at(5), 4096, nullptr) == KDA_OK && calls == before + 1 &&
           pool::last.count && pool::last.n == 1);

    if (failures) return 1;
    std::printf("sanitized linear recurrence and pool host checks passed\n");
    return 0;
}
