// q, k, v in 8 bits: e4m3 elements with one power-of-two exponent for each
// block of min(32, d) channels, and back.
//
// The exponent is the smallest e with max|x| <= 448 2^e over the block's
// finite elements, from the bits of the maximum: with max = m 2^p, m in
// [1, 2), e = p - 8 where m <= 1.75, else p - 7.  x 2^-e is then exact in
// fp32 and the one rounding is the conversion's (to nearest even).  Every
// e4m3 value times a power of two in range is a bf16 value, so what the
// backward reads is exact in its matrix operands.
// A copy in its cost: 2 + 1 + 1/32 bytes an element each way.  One thread
// takes eight elements (16 bytes of bf16); a block is four neighbouring
// lanes (two at d = 16).  16384 tokens of 16 + 16 + 32 heads of 128: 407 MB each
// way, both ways in 139 us, 5.8 TB/s.
#include "gdr_device.h"

namespace gdr {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(256)
void gdr_save8_kernel(Kept8 a)
{
    // q, k and v in one launch: a workgroup's part is that of its index
    const int t = blockIdx.x < a.first[1] ? 0 : blockIdx.x < a.first[2] ? 1 : 2;
    const u32x4 *__restrict__ x = static_cast<const u32x4 *>(a.x[t]);
    const int64_t n8 = a.n8[t], stride = (a.first[t + 1] - a.first[t]) * 256ll;
    const int lanes = a.lanes[t];
    u32x2 *__restrict__ x8 = reinterpret_cast<u32x2 *>(a.x8[t]);
    uint8_t *__restrict__ xe = a.xe[t];
    // every lane of a block is in or out together: blocks do not straddle n8
    for (int64_t i = (blockIdx.x - a.first[t]) * 256ll + threadIdx.x; i < n8; i += stride) {
        const u32x4 w = __builtin_nontemporal_load(x + i);
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
        uint32_t top = 0;                       // bits of the largest finite magnitude
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = __float_as_uint(f[j]) & 0x7fffffffu;
            if (m < 0x7f800000u && m > top) top = m;
        }
        for (int m = 1; m < lanes; m *= 2) {
            const uint32_t y = (uint32_t)__shfl_xor((int)top, m);
            top = y > top ? y : top;
        }
        // biased exponent p + 127; e + 127 kept in [17, 246]
        int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = e < 17 ? 17 : e > 246 ? 246 : e;
        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // past the largest exponent values stop at 448; NaN and
            // infinities become NaN
            const float z = f[j] * inv;
            const bool fin = (__float_as_uint(f[j]) & 0x7fffffffu) < 0x7f800000u;
            y[j] = fin ? fminf(fmaxf(z, -448.f), 448.f) : __uint_as_float(0x7fc00000u);
        }
        u32x2 b;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j], y[4 * j + 1], 0, false);
            b[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j + 2], y[4 * j + 3], p, true);
        }
        x8[i] = b;
        if (threadIdx.x % lanes == 0) xe[i / lanes] = (uint8_t)e;
    }
}

__global__ __launch_bounds__(256)
void gdr_load8_kernel(Kept8 a)
{
    const int t = blockIdx.x < a.first[1] ? 0 : blockIdx.x < a.first[2] ? 1 : 2;
    u32x4 *__restrict__ x = static_cast<u32x4 *>(const_cast<void *>(a.x[t]));
    const int64_t n8 = a.n8[t], stride = (a.first[t + 1] - a.first[t]) * 256ll;
    const int lanes = a.lanes[t];
    const u32x2 *__restrict__ x8 = reinterpret_cast<const u32x2 *>(a.x8[t]);
    const uint8_t *__restrict__ xe = a.xe[t];
    for (int64_t i = (blockIdx.x - a.first[t]) * 256ll + threadIdx.x; i < n8; i += stride) {
        const u32x2 b = __builtin_nontemporal_load(x8 + i);
        const float f = __uint_as_float((uint32_t)xe[i / lanes] << 23);
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto p = __builtin_amdgcn_cvt_pk_f32_fp8((int)b[j], false);
            const auto r = __builtin_amdgcn_cvt_pk_f32_fp8((int)b[j], true);
            // exact: the upper halves of these floats are the bf16 values
            const float p0 = p[0] * f, p1 = p[1] * f, r0 = r[0] * f, r1 = r[1] * f;
            w[2 * j] = (__float_as_uint(p0) >> 16) | (__float_as_uint(p1) & 0xffff0000u);
            w[2 * j + 1] = (__float_as_uint(r0) >> 16) | (__float_as_uint(r1) & 0xffff0000u);
        }
        __builtin_nontemporal_store(w, x + i);
    }
}

// fills in the workgroups' ranges; the number of them, or 0
int plan(Kept8 &a)
{
    int at = 0;
    for (int t = 0; t < 3; ++t) {
        a.first[t] = at;
        const int64_t b = (a.n8[t] + 255) / 256;
        at += (int)(b < 65536 ? b : 65536);
    }
    a.first[3] = at;
    return at;
}

}  // namespace

hipError_t launch_save8(Kept8 a, hipStream_t s)
{
    const int blocks = plan(a);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(gdr_save8_kernel, dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_load8(Kept8 a, hipStream_t s)
{
    const int blocks = plan(a);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(gdr_load8_kernel, dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace gdr
