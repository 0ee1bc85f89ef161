// Building blocks of the gated delta rule's chunk kernels (gfx950): matrix
// core products with operands held as several bf16 parts, transposing LDS
// reads, and bounded loads of q, k, v rows in either storage form.
//
// Precision.  An fp32 operand is held as up to three bf16 parts h + m + l,
// each the rounding of what the parts before it leave: together 24 bits, so
// a product of an exact bf16 operand with three parts, or of two such
// operands without the parts products below 2^-24, is an fp32 product.
//
// Operand layouts of v_mfma_f32_16x16x32_bf16 (lane = ln + 16 lg): A holds
// row ln, slots 8 lg .. 8 lg + 7; B column ln, the same slots; the result
// column ln, rows 4 lg .. 4 lg + 3.  A result tile pair (x0, x1) of 32 rows is
// therefore a B operand as it stands, if slot (lg, i) means row 4 lg + i of x0
// for i < 4 and row 4 lg + i - 4 of x1 behind it; the A operand beside it is
// read or written in that order.
#pragma once

#include "gdr_device.h"

namespace gdr {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ u32x2 pack4(f32x4 x) { return u32x2{pack2(x[0], x[1]), pack2(x[2], x[3])}; }
__device__ __forceinline__ bf16x8 join(u32x2 a, u32x2 b)
{
    return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// The negative identity on the slots 0..3 (a) or 4..7 (b) of a lane's own
// rows: mma(eye.a, [h | .], x) = x - h of the same lane, exactly, on the
// matrix core instead of the vector ALU.
struct Eye {
    bf16x8 a, b;
};
__device__ __forceinline__ Eye make_eye(int lane)
{
    const int m = lane & 15, g = lane >> 4;
    Eye e;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        e.a[i] = (i < 4 && m == 4 * g + i) ? (bf16)-1.0f : (bf16)0.0f;
        e.b[i] = (i >= 4 && m == 4 * g + i - 4) ? (bf16)-1.0f : (bf16)0.0f;
    }
    return e;
}

// parts of a 32-row tile pair as B operands
template <int NS> struct Parts {
    bf16x8 p[NS];
};
template <int NS>
__device__ __forceinline__ Parts<NS> split_pair(f32x4 x0, f32x4 x1, const Eye &eye)
{
    Parts<NS> r;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        r.p[i] = join(pack4(x0), pack4(x1));
        if (i + 1 < NS) {
            x0 = mma(eye.a, r.p[i], x0);
            x1 = mma(eye.b, r.p[i], x1);
        }
    }
    return r;
}
// acc + a * (parts of b), smallest first
template <int NS>
__device__ __forceinline__ f32x4 mma_parts(bf16x8 a, const Parts<NS> &b, f32x4 c)
{
#pragma unroll
    for (int i = NS - 1; i >= 0; --i) c = mma(a, b.p[i], c);
    return c;
}

// acc + (parts of a) * b: the transposed product, result column = b's row
template <int NS>
__device__ __forceinline__ f32x4 mma_by_parts(const Parts<NS> &a, bf16x8 b, f32x4 c)
{
#pragma unroll
    for (int i = NS - 1; i >= 0; --i) c = mma(a.p[i], b, c);
    return c;
}

// the three parts of a lane's four values of one tile
__device__ __forceinline__ void split3(f32x4 x, const Eye &eye, u32x2 (&p)[3])
{
    p[0] = pack4(x);
    x = mma(eye.a, join(p[0], p[0]), x);
    p[1] = pack4(x);
    x = mma(eye.a, join(p[1], p[1]), x);
    p[2] = pack4(x);
}

__device__ __forceinline__ bf16x8 lds8(const void *p) { return *static_cast<const bf16x8 *>(p); }

// Rows of 2 D bytes with their 16-byte pieces exchanged by row, so that 16
// lanes reading one piece of 16 rows touch every bank once.
template <int D>
struct Swz {
    static constexpr int NP = D / 8;             // pieces a row
    static __device__ __forceinline__ int at(int row, int c)
    {
        const int x = NP >= 16 ? row & 15 : (row >> 1) & 7;
        return row * D + (((c >> 3) ^ x) << 3) + (c & 7);
    }
};

// Transposing LDS read: lane (ln, lg) gets four rows of one column, given the
// address of row (ln / 4) of its group's four rows, columns 4 (ln % 4) ..
__device__ __forceinline__ u32x2 lds_tr(const bf16 *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_t;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)p));
}
__device__ __forceinline__ f32x4 widen(u32x2 w)
{
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u),
                 __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u)};
}

// Rows of q, k or v: n rows from token tok on (n <= 0: none), zeros behind
// them.  at() is a lane's place (row, channel of head h), raw() requests the
// eight channels c (a constant) behind it, bf() gives them in bf16.
template <typename T> struct Rows;
template <> struct Rows<bf16> {
    typedef u32x4 raw_t;
    typedef int at_t;
    rsrc_t r;
    __device__ __forceinline__ Rows(const void *p, const uint8_t *, int64_t tok, int n, int H, int d)
    {
        const int row_bytes = H * d * 2;
        r = make_rsrc(static_cast<const char *>(p) + tok * row_bytes, (n > 0 ? n : 0) * row_bytes);
    }
    static __device__ __forceinline__ at_t at(int row, int H, int h, int d, int c) { return ((row * H + h) * d + c) * 2; }
    __device__ __forceinline__ raw_t raw(at_t at, int c) const
    {
        return __builtin_amdgcn_raw_buffer_load_b128(r, at + 2 * c, 0, 0);
    }
    static __device__ __forceinline__ bf16x8 bf(raw_t w) { return __builtin_bit_cast(bf16x8, w); }
};
template <> struct Rows<e4m3> {
    struct raw_t {
        u32x2 w;
        uint32_t e;
    };
    struct at_t {
        int x, e;
    };
    rsrc_t r, re;
    __device__ __forceinline__ Rows(const void *p, const uint8_t *e, int64_t tok, int n, int H, int d)
    {
        const int row_bytes = H * d;
        n = n > 0 ? n : 0;
        r = make_rsrc(static_cast<const char *>(p) + tok * row_bytes, n * row_bytes);
        re = make_rsrc(e + tok * (row_bytes / 32), n * (row_bytes / 32));
    }
    static __device__ __forceinline__ at_t at(int row, int H, int h, int d, int c)
    {
        const int x = (row * H + h) * d + c;
        return at_t{x, x / 32};              // exact for raw()'s c: it never crosses a block from c % 32
    }
    __device__ __forceinline__ raw_t raw(at_t at, int c) const
    {
        raw_t x;
        x.w = __builtin_amdgcn_raw_buffer_load_b64(r, at.x + c, 0, 0);
        x.e = __builtin_amdgcn_raw_buffer_load_b8(re, at.e + c / 32, 0, 0);
        return x;
    }
    static __device__ __forceinline__ bf16x8 bf(raw_t x)
    {
        const float f = __uint_as_float(x.e << 23);
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)x.w[i], false);
            const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)x.w[i], true);
            o[2 * i] = pack2(a[0] * f, a[1] * f);
            o[2 * i + 1] = pack2(b[0] * f, b[1] * f);
        }
        return __builtin_bit_cast(bf16x8, o);
    }
};

}  // namespace gdr
