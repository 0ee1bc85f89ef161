// Device-side helpers of the gated linear recurrence kernels (gfx950 only).
#pragma once

#include "gdr_device.h"
#include "glr_launch.h"

namespace glr {

using kda::bf16;
using kda::LOG2E;
using kda::WAVE;

// e^g, plain
__device__ __forceinline__ float decay(float g) { return gdr::decay(gdr::floor_g(g)); }

// s(z) = 1 / (1 + e^-z), and 1 - s(z) = e^-z s(z) with its own digits.  Below
// -87 (where s is 1.6e-38) z counts as -87, which keeps e^-z finite; a NaN stays.
struct Logistic {
    float s, rest;
};
__device__ __forceinline__ Logistic logistic(float z)
{
    z = z < -87.f ? -87.f : z;
    const float e = kda::fast_exp2(z * -LOG2E), s = __builtin_amdgcn_rcpf(1.f + e);
    return Logistic{s, e * s};
}

// e^g and e^g - 1 for g <= 0: with k the nearest whole number to g log2 e and
// r = g - k ln 2 (ln 2 in two floats), e^r - 1 to the seventh power of r (the
// eighth is below 6e-9) and e^g - 1 = 2^k (e^r - 1) + (2^k - 1), so that the
// difference keeps its digits however near e^g is to 1.  k is read off the low
// bits of a float in [2^23, 2^24), which leaves a NaN a NaN.  Below -87 (where
// e^g is 1.6e-38) g counts as -87.
struct Expm1 {
    float e, m1;
};
__device__ __forceinline__ Expm1 exp_m1(float g)
{
    g = g < -87.f ? -87.f : g;
    const float big = 12582912.f, kb = __builtin_fmaf(g, LOG2E, big), k = kb - big;
    float r = __builtin_fmaf(-k, 0.693147182464599609375f, g);
    r = __builtin_fmaf(-k, -1.904654299957767878541e-9f, r);
    float p = 1.f / 5040;
    p = __builtin_fmaf(p, r, 1.f / 720);
    p = __builtin_fmaf(p, r, 1.f / 120);
    p = __builtin_fmaf(p, r, 1.f / 24);
    p = __builtin_fmaf(p, r, 1.f / 6);
    p = __builtin_fmaf(p, r, 0.5f);
    p = __builtin_fmaf(p, r * r, r);
    const float two = __uint_as_float((__float_as_uint(kb) << 23) + (127u << 23));
    return Expm1{__builtin_fmaf(two, p, two), __builtin_fmaf(two, p, two - 1.f)};
}

// One token's factor a and input u of a channel, gated.  m = sqrt(1 - a^2) =
// sqrt(-(a - 1)(a + 1)).
struct Gates {
    float a, b;          // u = b x, b = m s(i)
};
__device__ __forceinline__ Gates gates(float r, float i, float neg_rate)
{
    const Expm1 x = exp_m1(neg_rate * logistic(r).s);
    return Gates{x.e, __builtin_amdgcn_sqrtf(-x.m1 * (x.m1 + 2.f)) * logistic(i).s};
}

// ... and what the gradients want of them besides: with w = a h_{t-1},
// d h_t / d r = (w - c x) q,  d h_t / d rate = -(w - c x) s(r), from
// d m / d g = -a^2 / m, where the slope at m = 0 counts as 0.
struct GateGrads {
    float a, b, rest_i, s_r, q, c;
};
__device__ __forceinline__ GateGrads gate_grads(float r, float i, float neg_rate)
{
    const Logistic sr = logistic(r), si = logistic(i);
    const Expm1 x = exp_m1(neg_rate * sr.s);
    const float m2 = -x.m1 * (x.m1 + 2.f);
    // (below the smallest normal number the hardware's root takes m2 for 0)
    const float inv = m2 < 1.17549435e-38f ? 0.f : __builtin_amdgcn_rsqf(m2);
    return GateGrads{x.e, m2 * inv * si.s, si.rest, sr.s, neg_rate * sr.s * sr.rest, si.s * x.e * x.e * inv};
}

__device__ __forceinline__ gdr::SeqArgs seq_args(const Args &a)
{
    return gdr::SeqArgs{a.cu_seqlens, a.n_seqs, a.n_tokens, a.seqlen};
}

}  // namespace glr
