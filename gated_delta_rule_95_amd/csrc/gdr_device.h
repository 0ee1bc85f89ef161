// Device-side helpers shared by the gated delta rule kernels (gfx950 only).
#pragma once

#include "gdr_launch.h"
#include "kda_device.h"

namespace gdr {

using kda::bf16;
using kda::bf16x4;
using kda::bf16x8;
using kda::f32x2;
using kda::f32x4;
using kda::WAVE;
using kda::LOG2E;

// a byte of e4m3 beside the exponent bytes of its blocks
struct e4m3 {
    uint8_t x;
};

// q, k or v as stored.  ld4: four consecutive channels of a head row, in fp32.
template <typename T> struct Src {
    const T *p;
    __device__ __forceinline__ f32x4 ld4(int64_t row, int d, int c) const
    {
        return kda::Elem<T>::ld4(p + row * d + c);
    }
};
template <> struct Src<e4m3> {
    const uint8_t *p, *e;
    __device__ __forceinline__ f32x4 ld4(int64_t row, int d, int c) const
    {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p + row * d + c);
        const int blk = d < 32 ? d : 32;
        // exponent bytes are in [17, 246]: the factor is a normal power of
        // two and the product exact
        const float f = __uint_as_float((uint32_t)e[row * (d / blk) + c / blk] << 23);
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        return f32x4{a[0] * f, a[1] * f, b[0] * f, b[1] * f};
    }
};
template <typename T> __device__ __host__ inline Src<T> src(const void *p, const uint8_t *)
{
    return Src<T>{static_cast<const T *>(p)};
}
template <> __device__ __host__ inline Src<e4m3> src<e4m3>(const void *p, const uint8_t *e)
{
    return Src<e4m3>{static_cast<const uint8_t *>(p), e};
}
// storage type of o, dO and the gradients of q, k, v
template <typename T> struct OutOf { typedef T type; };
template <> struct OutOf<e4m3> { typedef bf16 type; };

// first token and length of sequence n; a table that breaks its contract
// gives lengths >= 0 inside [0, n_tokens]
struct Seq {
    int bos, len;
};
__device__ __forceinline__ Seq seq_of(const SeqArgs &s, int n)
{
    const int b = seq_edge(s, n), e = seq_edge(s, n + 1);
    return Seq{b, e > b ? e - b : 0};
}

// the sequence and chunk of a slot: slots of sequence n start at
// edge(n) / C + n, which grows with n
__device__ __forceinline__ bool find_chunk(const SeqArgs &s, int64_t slot, int C, int &n, int &c)
{
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

// Raw buffer resources: reads at or past `bytes` give 0, stores there are dropped.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void *base, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// log-decay with its floor (a NaN stays): exp of the floor is 0, and sums of
// 64 such values keep far more than single precision in their differences
__device__ __forceinline__ float floor_g(float g) { return g < -1e4f ? -1e4f : g; }

// e^g for the decay of one token.  With k the nearest whole number to
// g log2 e, r = g - k ln 2 (ln 2 in two floats; |r| <= 0.35) and e^r to the
// seventh power of r (the eighth is below 6e-9): the last sum rounds once, so
// the factor is off by little more than half a step, to either side as often.
// The hardware's 2^x of a product g log2 e is off by |g| 2^-24 at fast decays
// (3e-6 at g = -80) and by -7e-9 in the mean at slow ones, which a state
// multiplied by one such factor a token adds up (fp32, g > -1e-4, 700 tokens:
// o off by 1.65e-6).
__device__ __forceinline__ float decay(float g)
{
    // the bounds only keep NaN and overflow out of the conversion below
    const float k = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(g * LOG2E), -2e4f), 2e4f);
    float r = __builtin_fmaf(-k, 0.693147182464599609375f, g);
    r = __builtin_fmaf(-k, -1.904654299957767878541e-9f, r);
    float p = 1.f / 5040;
    p = __builtin_fmaf(p, r, 1.f / 720);
    p = __builtin_fmaf(p, r, 1.f / 120);
    p = __builtin_fmaf(p, r, 1.f / 24);
    p = __builtin_fmaf(p, r, 1.f / 6);
    p = __builtin_fmaf(p, r, 0.5f);
    p = __builtin_fmaf(p, r, 1.f);
    return __builtin_ldexpf(__builtin_fmaf(p, r, 1.f), (int)k);
}

// 2^(h + l), l what is left of the exponent behind the float h: alone, h would
// leave the factor off by |h| 2^-25
constexpr double LOG2E64 = 1.4426950408889634;
__device__ __forceinline__ float exp2_two(float h, float l)
{
    const float e = kda::fast_exp2(h);
    return __builtin_fmaf(e, 0.6931472f * l, e);
}
__device__ __forceinline__ float exp2_64(double x)
{
    const float h = (float)x;
    return exp2_two(h, (float)(x - (double)h));
}

// the upper 32 lanes of a change places with the lower 32 of b
__device__ __forceinline__ void swap32(float &a, float &b)
{
    uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(x), "+v"(y));
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
// the same with odd rows of 16 lanes of a and even ones of b
__device__ __forceinline__ void swap16(float &a, float &b)
{
    uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\ts_nop 1" : "+v"(x), "+v"(y));
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
// inclusive sum over the 64 lanes, on register moves between lanes
template <int CTRL, int ROWS, typename T>
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
template <typename T>
__device__ __forceinline__ T scan64(T x)
{
    x = scan_step<0x111, 0xf>(x);       // row_shr 1, 2, 4, 8
    x = scan_step<0x112, 0xf>(x);
    x = scan_step<0x114, 0xf>(x);
    x = scan_step<0x118, 0xf>(x);
    x = scan_step<0x142, 0xa>(x);       // lane 15 of each even row to the row behind it
    return scan_step<0x143, 0xc>(x);    // lane 31 to the upper half
}

// sum over the lanes of equal lane % 16
__device__ __forceinline__ float sum_groups(float x)
{
    float a, b;
    kda::row_pair(x, a, b);
    x = a + b;
    kda::half_pair(x, a, b);
    return a + b;
}

}  // namespace gdr
