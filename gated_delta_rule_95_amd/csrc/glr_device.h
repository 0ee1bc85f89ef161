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

// s(z) = 1 / (1 + e^-z); where e^-z overflows, s is 0
__device__ __forceinline__ float logistic(float z)
{
    return __builtin_amdgcn_rcpf(1.f + kda::fast_exp2(z * -LOG2E));
}
// ... and 1 - s(z) = e^-z s(z) with its own digits (where s is 0, any number)
struct Logistic {
    float s, rest;
};
__device__ __forceinline__ Logistic logistic_both(float z)
{
    const float e = kda::fast_exp2(z * -LOG2E), s = __builtin_amdgcn_rcpf(1.f + e);
    return Logistic{s, __builtin_fminf(e, 3.4028235e38f) * s};
}

// e^g and e^g - 1 for g <= 0, the difference with its own digits however near
// e^g is to 1: (e^x - 1) / x as a polynomial of the fifth degree, which is the
// best in the maximum norm on its range (off by 2.3e-8 of itself at most; in
// fp32 x times it is off by 1.3e-7, two roundings).
// NEAR: for g >= -kNear only, the polynomial at g itself.
// Else: with k the nearest whole number to g log2 e, at x = g - k ln 2 (ln 2
// in two floats), and e^g - 1 = 2^k (e^x - 1) + (2^k - 1).  k is read off the
// low bits of a float in [2^23, 2^24), which leaves a NaN a NaN.  Below -87
// (where e^g is 1.6e-38) g counts as -87.
constexpr float kNear = 0.69f;
struct Expm1 {
    float e, m1;
};
template <bool NEAR> __device__ __forceinline__ Expm1 exp_m1(float g)
{
    if constexpr (NEAR) {
        float p = 0.0010301340371370316f;
        p = __builtin_fmaf(p, g, 0.008062456734478474f);
        p = __builtin_fmaf(p, g, 0.04156935214996338f);
        p = __builtin_fmaf(p, g, 0.16665059328079224f);
        p = __builtin_fmaf(p, g, 0.4999990165233612f);
        p = __builtin_fmaf(p, g, 1.f);
        p *= g;
        return Expm1{1.f + p, p};
    } else {
        g = g < -87.f ? -87.f : g;
        const float big = 12582912.f, kb = __builtin_fmaf(g, LOG2E, big), k = kb - big;
        float x = __builtin_fmaf(-k, 0.693147182464599609375f, g);
        x = __builtin_fmaf(-k, -1.904654299957767878541e-9f, x);
        float p = 0.0013888872927054763f;
        p = __builtin_fmaf(p, x, 0.00836909469217062f);
        p = __builtin_fmaf(p, x, 0.041667137295007706f);
        p = __builtin_fmaf(p, x, 0.16666506230831146f);
        p = __builtin_fmaf(p, x, 0.4999999701976776f);
        p = __builtin_fmaf(p, x, 1.f);
        p *= x;
        const float two = __uint_as_float((__float_as_uint(kb) << 23) + (127u << 23));
        return Expm1{__builtin_fmaf(two, p, two), __builtin_fmaf(two, p, two - 1.f)};
    }
}

// One token's factor a and input u of a channel, gated.  m = sqrt(1 - a^2) =
// sqrt(-(a - 1)(a + 1)).
struct Gates {
    float a, b;          // u = b x, b = m s(i)
};
template <bool NEAR> __device__ __forceinline__ Gates gates(float r, float i, float neg_rate)
{
    const Expm1 x = exp_m1<NEAR>(neg_rate * logistic(r));
    return Gates{x.e, __builtin_amdgcn_sqrtf(-x.m1 * (x.m1 + 2.f)) * logistic(i)};
}

// ... and what the gradients want of them besides: with w = a h_{t-1},
// d h_t / d r = (w - c x) q,  d h_t / d rate = -(w - c x) s(r), from
// d m / d g = -a^2 / m, where the slope at m = 0 counts as 0.
struct GateGrads {
    float a, b, rest_i, s_r, q, c;
};
template <bool NEAR> __device__ __forceinline__ GateGrads gate_grads(float r, float i, float neg_rate)
{
    const Logistic sr = logistic_both(r), si = logistic_both(i);
    const float g = neg_rate * sr.s;
    const Expm1 x = exp_m1<NEAR>(g);
    const float m2 = -x.m1 * (x.m1 + 2.f);
    // (below the smallest normal number the hardware's root takes m2 for 0)
    const float inv = m2 < 1.17549435e-38f ? 0.f : __builtin_amdgcn_rsqf(m2);
    return GateGrads{x.e, m2 * inv * si.s, si.rest, sr.s, g * sr.rest, si.s * x.e * x.e * inv};
}

__device__ __forceinline__ gdr::SeqArgs seq_args(const Args &a)
{
    return gdr::SeqArgs{a.cu_seqlens, a.n_seqs, a.n_tokens, a.seqlen};
}

}  // namespace glr
