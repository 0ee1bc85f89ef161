// Host-only sanitizer driver (AddressSanitizer + UndefinedBehaviorSanitizer) of
// the gated delta rule's C-ABI layer.
//
// Links gdr_api.cpp (and kda_api.cpp, whose error state it shares), compiled
// as plain host C++, against stub kernel launchers that record their arguments
// instead of touching a GPU, and walks the validation, overlap and size
// arithmetic of every entry point, up to the largest sizes the header allows.
// An undefined operation or out-of-bounds access aborts the run; the pytest
// wrapper checks for a clean exit.
#include <cstdio>
#include <cstring>
#include <vector>

#include "gdr.h"
#include "gdr_launch.h"
#include "kda_launch.h"

namespace kda {
size_t prefill_workspace_bytes(const PrefillArgs &) { return 0; }
hipError_t launch_prefill(const PrefillArgs &) { return hipSuccess; }
hipError_t launch_decode(const DecodeArgs &) { return hipSuccess; }
size_t bwd_part_floats(int32_t d_k, int32_t d_v) { return (size_t)d_k * d_v; }
hipError_t launch_bwd(const BwdArgs &) { return hipSuccess; }
hipError_t launch_spec(const SpecArgs &) { return hipSuccess; }
}  // namespace kda

namespace gdr {
static int chunk_calls, recurrent_calls, grad_calls, decode_calls, copy_calls;
static Args last;
static DecodeArgs last_decode;
static Kept8 last_kept;
static hipError_t result = hipSuccess;
static hipError_t note(int &calls, const Args &a)
{
    ++calls;
    last = a;
    return result;
}
hipError_t launch_recurrent_fwd(const Args &a) { return note(recurrent_calls, a); }
hipError_t launch_recurrent_keep_sweep(const Args &a) { return note(recurrent_calls, a); }
hipError_t launch_grad32(const Args &a) { return note(grad_calls, a); }
hipError_t launch_chunk_fwd(const Args &a) { return note(chunk_calls, a); }
hipError_t launch_chunk_keep_sweep(const Args &a) { return note(chunk_calls, a); }
hipError_t launch_chunk_grad(const Args &a) { return note(grad_calls, a); }
hipError_t launch_decode(const DecodeArgs &a)
{
    ++decode_calls;
    last_decode = a;
    return result;
}
hipError_t launch_save8(Kept8 a, hipStream_t)
{
    ++copy_calls;
    last_kept = a;
    return result;
}
hipError_t launch_load8(Kept8 a, hipStream_t)
{
    ++copy_calls;
    last_kept = a;
    return result;
}
static int calls() { return chunk_calls + recurrent_calls + grad_calls + decode_calls + copy_calls; }
}  // namespace gdr

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
    int32_t n = 2, Hk = 2, Hv = 4, dk = 128, dv = 64;
    int64_t N = 300;
    kda_dtype t = KDA_BF16;
    const int32_t *cu = nullptr;
    const void *q = at(1), *k = at(2), *v = at(3), *dO = at(4);
    const float *g = p<float>(5), *beta = p<float>(6), *S0 = p<float>(7), *dS_T = p<float>(8);
    void *o = at(9), *dq = at(10), *dkey = at(11), *dval = at(12);
    float *S_T = p<float>(13), *dg = p<float>(14), *db = p<float>(15), *dS0 = p<float>(16);
    void *ws = at(17);
    size_t ws_bytes = ~(size_t)0 >> 8;
    kda_status fwd() const
    {
        return gdr_fwd_chunked(q, k, v, g, beta, S0, cu, n, N, Hk, Hv, dk, dv, 1.f, t, o, S_T, nullptr);
    }
    kda_status bwd() const
    {
        return gdr_bwd_chunked(q, k, v, g, beta, S0, cu, n, N, Hk, Hv, dk, dv, 1.f, t, dO, dS_T, dq, dkey, dval, dg, db,
                               dS0, ws, ws_bytes, nullptr);
    }
    kda_status bwd8() const
    {
        return gdr_bwd_chunked_saved8((const uint8_t *)q, p<uint8_t>(20), (const uint8_t *)k, p<uint8_t>(21),
                                      (const uint8_t *)v, p<uint8_t>(22), g, beta, S0, cu, n, N, Hk, Hv, dk, dv, 1.f, dO,
                                      dS_T, dq, dkey, dval, dg, db, dS0, ws, ws_bytes, nullptr);
    }
    size_t need() const { return gdr_bwd_workspace_bytes(n, N, Hk, Hv, dk, dv, t); }
};

int main()
{
    Call c;
    // both forms, all three passes
    EXPECT(c.fwd() == KDA_OK && gdr::chunk_calls == 1 && gdr::last.seq.seqlen == 150);
    EXPECT(c.bwd() == KDA_OK && gdr::chunk_calls == 2 && gdr::grad_calls == 1 && gdr::last.in == gdr::In::BF16);
    EXPECT(c.bwd8() == KDA_OK && gdr::grad_calls == 2 && gdr::last.in == gdr::In::E4M3);
    c.t = KDA_F32;
    EXPECT(c.fwd() == KDA_OK && c.bwd() == KDA_OK && gdr::recurrent_calls == 2 && gdr::grad_calls == 3);
    // the workspace's parts lie behind one another, within what is asked for
    for (int32_t dk : {16, 32, 64, 128})
        for (int32_t dv : {16, 32, 64, 128})
            for (kda_dtype t : {KDA_BF16, KDA_F32})
                for (int64_t N : {0, 1, 63, 64, 300, 100000}) {
                    Call x;
                    x.dk = dk; x.dv = dv; x.t = t; x.N = N; x.n = 1; x.ws_bytes = x.need();
                    EXPECT(x.need() % 256 == 0 && x.need() > 0);
                    EXPECT(x.bwd() == KDA_OK);
                    const gdr::Args &a = gdr::last;
                    const char *w = static_cast<const char *>(x.ws);
                    const int C = gdr::bwd_chunk(dk, dv, t == KDA_BF16);
                    const size_t st = (size_t)gdr::bwd_slots(1, N, C) * x.Hv * dk * dv * 4, rw = (size_t)N * x.Hv * dv * 4;
                    const char *ends[] = {(const char *)a.Sc + st, (const char *)a.Lc + st, (const char *)a.R + rw,
                                          (const char *)a.Ub + rw};
                    EXPECT((const char *)a.Sc == w && ends[0] <= (const char *)a.Lc && ends[1] <= (const char *)a.R &&
                           ends[2] <= (const char *)a.Ub && ends[3] <= w + x.ws_bytes);
                    if (N > 0) {
                        x.ws_bytes -= 1;
                        EXPECT(x.bwd() == KDA_ERR_INVALID_ARG);
                    }
                }
    // nothing reaches a launcher from here on, unless said
    const int before = gdr::calls();
    const auto bad = [&](auto change, kda_status want = KDA_ERR_INVALID_ARG) {
        Call x;
        change(x);
        EXPECT(x.bwd() == want);
        EXPECT(std::strlen(kda_last_error()) > 0);
    };
    bad([](Call &x) { x.q = nullptr; });
    bad([](Call &x) { x.g = nullptr; });
    bad([](Call &x) { x.dq = nullptr; });
    bad([](Call &x) { x.ws = nullptr; });
    bad([](Call &x) { x.ws = at(17, 128); });
    bad([](Call &x) { x.v = at(3, 8); });
    bad([](Call &x) { x.dg = p<float>(14, 2); });
    bad([](Call &x) { x.cu = p<int32_t>(18, 1); });
    bad([](Call &x) { x.dS0 = p<float>(16, 4); });
    bad([](Call &x) { x.dkey = x.dq; });
    bad([](Call &x) { x.dq = at(1, 300 * 2 * 128 * 2 - 16); });
    bad([](Call &x) { x.dval = (void *)x.dO; });
    bad([](Call &x) { x.ws = at(7); });
    bad([](Call &x) { x.dk = 48; }, KDA_ERR_UNSUPPORTED);
    bad([](Call &x) { x.dv = 256; }, KDA_ERR_UNSUPPORTED);
    bad([](Call &x) { x.Hk = 0; });
    bad([](Call &x) { x.Hv = 3; });
    bad([](Call &x) { x.Hv = -4; });
    bad([](Call &x) { x.Hk = x.Hv = 0x7fffffff; });
    bad([](Call &x) { x.Hk = 1; x.Hv = 1 << 15; });
    bad([](Call &x) { x.n = -1; });
    bad([](Call &x) { x.n = 0; });
    bad([](Call &x) { x.n = 7; });
    bad([](Call &x) { x.N = -1; });
    bad([](Call &x) { x.N = (int64_t)1 << 31; });
    bad([](Call &x) { x.N = INT64_MAX; });
    bad([](Call &x) { x.N = INT64_MIN; });
    bad([](Call &x) { x.n = 0x7fffffff; x.cu = p<int32_t>(18); });
    bad([](Call &x) { x.N = ((int64_t)1 << 31) - 64; x.n = 1; x.Hk = 1; });      // 2^25 chunks
    bad([](Call &x) { x.dv = 128; x.Hk = x.Hv = 1; x.n = (1 << 21) - 1; x.N = x.n; });
    EXPECT(gdr::calls() == before);
    // what may lie beside each other or be absent
    {
        Call x;
        x.S0 = x.dS_T = nullptr;
        x.dS0 = nullptr;
        x.dq = at(1, 300 * 2 * 128 * 2);
        EXPECT(x.bwd() == KDA_OK);
        x.S_T = nullptr;
        EXPECT(x.fwd() == KDA_OK);
        x.N = 0;
        x.q = x.k = x.v = x.dO = nullptr;
        x.g = x.beta = nullptr;
        x.o = x.dq = x.dkey = x.dval = nullptr;
        x.dg = x.db = nullptr;
        EXPECT(x.fwd() == KDA_OK && x.bwd() == KDA_OK);
        x.n = 0;
        EXPECT(x.fwd() == KDA_OK && x.bwd() == KDA_OK);
    }
    // the largest sizes
    for (kda_dtype t : {KDA_BF16, KDA_F32}) {
        Call x;
        x.t = t; x.dk = x.dv = 128; x.Hk = 1; x.Hv = (1 << 15) - 1; x.n = 1; x.N = ((int64_t)1 << 31) - 64;
        EXPECT(x.fwd() == KDA_OK && gdr::last.seq.n_tokens == 0x7fffffc0);
        x.N = (int64_t)1 << 27;
        EXPECT(x.need() > (size_t)1 << 50);
        EXPECT(x.bwd() == KDA_OK);
        EXPECT(x.bwd8() == KDA_OK);
        x.dk = x.dv = 16; x.Hk = x.Hv = 1; x.n = (1 << 21) - 1; x.N = x.n;
        EXPECT(x.fwd() == KDA_OK && x.bwd() == KDA_OK);
        x.n = 1 << 21; x.N = x.n;
        EXPECT(x.fwd() == KDA_ERR_INVALID_ARG && x.bwd() == KDA_ERR_INVALID_ARG);
    }
    EXPECT(gdr_bwd_workspace_bytes(0, 10, 1, 1, 64, 64, KDA_BF16) == 0);
    EXPECT(gdr_bwd_workspace_bytes(1, -1, 1, 1, 64, 64, KDA_BF16) == 0);
    EXPECT(gdr_bwd_workspace_bytes(1, 10, 1, 1, 64, 64, (kda_dtype)7) == 0);
    // a launcher's error comes back as one, with the call's name
    gdr::result = hipErrorInvalidValue;
    EXPECT(Call().fwd() == KDA_ERR_HIP && std::strstr(kda_last_error(), "gdr_fwd_chunked"));
    EXPECT(Call().bwd() == KDA_ERR_HIP && std::strstr(kda_last_error(), "gdr_bwd_chunked"));
    gdr::result = hipSuccess;

    // decode
    const auto dec = [](int32_t n_slots, int32_t N, const int32_t *slots, float *S, int32_t Hk = 2, int32_t Hv = 4) {
        return gdr_decode_step(at(1), at(2), at(3), p<float>(5), p<float>(6), S, slots, n_slots, N, Hk, Hv, 128, 128, 1.f,
                               KDA_BF16, at(9), nullptr);
    };
    EXPECT(dec(8, 5, p<int32_t>(18), p<float>(7)) == KDA_OK && gdr::last_decode.n_slots == 8);
    EXPECT(dec(5, 5, nullptr, p<float>(7)) == KDA_OK);
    EXPECT(dec(4, 5, nullptr, p<float>(7)) == KDA_ERR_INVALID_ARG);
    EXPECT(dec(-1, 5, p<int32_t>(18), p<float>(7)) == KDA_ERR_INVALID_ARG);
    EXPECT(dec(0, 5, p<int32_t>(18), nullptr) == KDA_OK);
    EXPECT(dec(1, 5, p<int32_t>(18), nullptr) == KDA_ERR_INVALID_ARG);
    EXPECT(dec(8, -5, p<int32_t>(18), p<float>(7)) == KDA_ERR_INVALID_ARG);
    EXPECT(dec(8, 0, nullptr, nullptr) == KDA_OK);
    EXPECT(dec(8, 5, p<int32_t>(7), p<float>(7)) == KDA_ERR_INVALID_ARG);
    EXPECT(dec(1 << 24, 5, p<int32_t>(18), p<float>(7), 1, (1 << 15) - 1) == KDA_OK);
    EXPECT(dec(0x7fffffff, 0x7fffffff, p<int32_t>(18), p<float>(7)) == KDA_ERR_INVALID_ARG);

    // 8 bits
    const auto keep = [](int64_t N, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, uint8_t *ve, bool load = false) {
        uint8_t *x[] = {p<uint8_t>(20), p<uint8_t>(21), p<uint8_t>(22), p<uint8_t>(23), p<uint8_t>(24)};
        return load ? gdr_load8(x[0], x[1], x[2], x[3], x[4], ve, N, Hk, Hv, dk, dv, at(1), at(2), at(3), nullptr)
                    : gdr_save8(at(1), at(2), at(3), N, Hk, Hv, dk, dv, x[0], x[1], x[2], x[3], x[4], ve, nullptr);
    };
    EXPECT(keep(100, 2, 4, 16, 128, p<uint8_t>(25)) == KDA_OK && gdr::last_kept.n8[0] == 400 && gdr::last_kept.lanes[0] == 2 &&
           gdr::last_kept.lanes[2] == 4);
    EXPECT(keep(100, 2, 4, 16, 128, p<uint8_t>(25), true) == KDA_OK);
    EXPECT(keep(((int64_t)1 << 31) - 64, 1, (1 << 15) - 1, 128, 128, p<uint8_t>(25)) == KDA_OK &&
           gdr::last_kept.n8[2] == (((int64_t)1 << 31) - 64) * ((1 << 15) - 1) * 16);
    EXPECT(keep((int64_t)1 << 31, 1, 1, 128, 128, p<uint8_t>(25)) == KDA_ERR_INVALID_ARG);
    EXPECT(keep(100, 2, 4, 16, 128, p<uint8_t>(24, 100)) == KDA_ERR_INVALID_ARG);          // overlaps v8
    EXPECT(keep(100, 2, 4, 16, 128, p<uint8_t>(24, 100), true) == KDA_OK);                 // both only read
    EXPECT(keep(100, 2, 4, 16, 128, p<uint8_t>(3, 1), true) == KDA_ERR_INVALID_ARG);
    EXPECT(keep(100, 2, 4, 16, 128, nullptr) == KDA_ERR_INVALID_ARG);
    EXPECT(keep(0, 2, 4, 16, 128, nullptr) == KDA_OK);
    EXPECT(keep(100, 2, 4, 24, 128, p<uint8_t>(25)) == KDA_ERR_UNSUPPORTED);

    if (failures) return 1;
    std::printf("sanitized gated delta rule host checks passed\n");
    return 0;
}
