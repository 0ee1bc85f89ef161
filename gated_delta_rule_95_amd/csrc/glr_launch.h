// Internal launch interface of the gated linear recurrence (glr_*) between
// the C-ABI layer (glr_api.cpp) and the kernel translation units.  Arguments
// arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "glr.h"

namespace glr {

// tokens between two kept states
constexpr int kKept = 32;

struct Args {
    const void *x, *r, *i;               // r, i: gated
    const float *g, *rate;               // plain; gated
    const float *h0;
    const int32_t *cu_seqlens;           // nullptr: equal lengths seqlen
    int32_t n_seqs, n_tokens, seqlen, D;
    bool gated, bf16;
    void *h;                             // forward (nullptr: not written)
    float *h_T, *kept;
    // backward; kept is read
    const void *dh;
    const float *dh_T;
    void *dx, *dr, *di;
    float *dg, *drate, *dh0;
    void *ws;
    hipStream_t stream;
};

struct DecodeArgs {
    const void *x, *r, *i;
    const float *g, *rate;
    float *S;
    const int32_t *slots;
    int32_t n_slots, N, D;
    bool gated, bf16;
    void *h;
    hipStream_t stream;
};

hipError_t launch_fwd(const Args &a);
hipError_t launch_bwd(const Args &a);
hipError_t launch_decode(const DecodeArgs &a);

}  // namespace glr
