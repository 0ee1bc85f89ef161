// Internal launch interface of the gated delta rule (gdr_*) between the
// C-ABI layer (gdr_api.cpp) and the kernel translation units.  Arguments
// arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr.h"

namespace gdr {

// q, k, v as stored: bf16, fp32, or e4m3 bytes with their exponent bytes
enum class In { F32, BF16, E4M3 };

struct SeqArgs {
    const int32_t *cu_seqlens;   // nullptr: equal lengths seqlen
    int32_t n_seqs;
    int32_t n_tokens;
    int32_t seqlen;
};

struct Args {
    const void *q, *k, *v;
    const uint8_t *qe, *ke, *ve;         // exponents (In::E4M3)
    const float *g, *beta, *S0;
    SeqArgs seq;
    int32_t Hk, Hv, dk, dv;
    float scale;
    In in;
    void *o;                             // forward
    float *S_T;
    // backward: cotangents, gradients and the workspace's parts
    const void *dO;
    const float *dS_T;
    void *dq, *dkey, *dval;
    float *dg, *dbeta, *dS0;
    float *Sc, *Lc;                      // [slots, Hv, dk * dv] chunk-entry states, exit cotangents (in the
                                         // form's own order, 4 bytes an element)
    float *R, *Ub;                       // [n_tokens, Hv, dv]
    hipStream_t stream;
};

struct DecodeArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float *S;
    const int32_t *slots;
    int32_t n_slots, N, Hk, Hv, dk, dv;
    float scale;
    bool bf16;
    void *o;
    hipStream_t stream;
};

// tokens between two kept states of the backward, token by token
constexpr int kRecurrentChunk = 32;
// ... and in either form
int bwd_chunk(int dk, int dv, bool bf16);
// chunk slots cu_seqlens[n] / C + n + c of a batch: an upper bound on every slot + 1
__host__ __device__ inline int64_t bwd_slots(int32_t n_seqs, int64_t n_tokens, int C)
{
    return n_tokens / C + n_seqs + 1;
}

// the kernels behind launch_fwd and launch_bwd (gdr_api.cpp), by form: token
// by token in fp32, or chunks of 64 on the matrix cores
hipError_t launch_recurrent_fwd(const Args &a);
hipError_t launch_recurrent_keep_sweep(const Args &a);
hipError_t launch_grad32(const Args &a);
hipError_t launch_chunk_fwd(const Args &a);
hipError_t launch_chunk_keep_sweep(const Args &a);
hipError_t launch_chunk_grad(const Args &a);
hipError_t launch_decode(const DecodeArgs &a);

// q, k, v (bf16) and their 8-bit form
struct Kept8 {
    const void *x[3];
    uint8_t *x8[3], *xe[3];
    int64_t n8[3];                       // groups of eight elements
    int lanes[3];                        // groups a block
    int first[4];                        // first workgroups (filled in at launch)
};
hipError_t launch_save8(Kept8 a, hipStream_t s);
hipError_t launch_load8(Kept8 a, hipStream_t s);

}  // namespace gdr
