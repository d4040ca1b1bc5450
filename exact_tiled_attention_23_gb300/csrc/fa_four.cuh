// fa_four.cuh -- the numbers of a 4-bit cache.
//
// A row is padded to 64, 128 or 256 elements and held in groups of 16: element d is
// u s, where u has 4 bits (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6; an even d is the lower half of its byte) and the group's scale s has 8
// (5 exponent bits, 3 mantissa bits: the upper bits of an IEEE half, whose sign is
// never set).  s is largest / 6, rounded to nearest, and u is x / s, rounded to
// nearest; halfway goes to the even mantissa, and past 6 to 6.
//
// u s has at most 6 significant bits and lies between 2^-18 and 6 * 10240 = 61440, so
// that it is exact as an IEEE half and as a bf16 number.
#pragma once

#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

// The largest scale, 10240: what it stands for with u = 6 is below fp16's largest.
constexpr uint32_t kLargestScale = 226;

// x / s to nearest, from y = 1 / s to nearest: P. Markstein's correction of a quotient
// by its remainder (1990).  (s is not so small or large that a step leaves the normal
// range, and a quotient that small is 0 in 4 bits.)
__device__ __forceinline__ float quotient(float x, float s, float y)
{
    const float q = x * y;
    return fmaf(fmaf(-q, s, x), y, q);
}

// Two of them; s as (-s, -s), y as (y, y).
__device__ __forceinline__ uint64_t quotient2(uint64_t x, uint64_t minus_s, uint64_t y)
{
    const uint64_t q = ptx::mul2(x, y);
    return ptx::fma2(ptx::fma2(q, minus_s, x), y, q);
}

// The scale for a group whose largest magnitude is `largest` (infinities: the
// largest scale; a NaN among the values is not counted).
__device__ __forceinline__ uint32_t scale_code(float largest)
{
    const float t = quotient(largest, 6.f, 1.f / 6.f);        // (NaN: the largest scale)
    if (t < 6.103515625e-5f) return (uint32_t)__float2int_rn(t * 131072.f);     // below 2^-14: multiples of 2^-17
    const uint32_t bits = __float_as_uint(t);
    const uint32_t up = (bits + 0x7ffffu + ((bits >> 20) & 1u)) >> 20;          // 3 mantissa bits, to nearest
    return min(up - ((127u - 15u) << 3), kLargestScale);
}

__device__ __forceinline__ float scale_value(uint32_t code)
{
    return __half2float(__ushort_as_half((unsigned short)(code << 7)));
}

// 16 values in 4 bits each, and their scale.
__device__ __forceinline__ uint2 to_four(const float (&x)[16], uint32_t &code)
{
    float largest = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
    for (int i = 2; i < 16; i += 2) largest = ptx::max3(largest, fabsf(x[i]), fabsf(x[i + 1]));
    code = scale_code(largest);
    if (code == 0) return make_uint2(0u, 0u);
    // (exact quotients: x / s halfway between two numbers stays halfway)
    const float s = scale_value(code), y = __frcp_rn(s);
    const uint64_t minus_s2 = ptx::pack2(-s, -s), y2 = ptx::pack2(y, y);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            ptx::unpack2(quotient2(ptx::pack2(x[8 * h + i], x[8 * h + i + 1]), minus_s2, y2), q[i], q[i + 1]);
        w[h] = ptx::pack_e2m1x8(q);
    }
    return make_uint2(w[0], w[1]);
}

// 8 elements of 4 bits times `scale` (a pair of equal halves), as 16-bit pairs of
// neighbours.
__device__ __forceinline__ void from_four(uint32_t w, __half2 scale, __half2 (&x)[4])
{
    uint32_t r[4];
    ptx::unpack_e2m1x8(w, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __hmul2(*reinterpret_cast<const __half2 *>(&r[i]), scale);
}

// The same values in the 16-bit type of the queries.
template <bool kF16>
__device__ __forceinline__ uint4 rows_from_four(uint32_t w, uint32_t code)
{
    const uint32_t pair = (code << 7) * 0x10001u;
    __half2 x[4];
    from_four(w, *reinterpret_cast<const __half2 *>(&pair), x);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kF16) {
            r[i] = *reinterpret_cast<const uint32_t *>(&x[i]);
        } else {
            const float2 f = __half22float2(x[i]);
            r[i] = ptx::pack_bf16x2(f.x, f.y);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The power of two that takes a row of bf16 queries whose largest magnitude is
// `largest` to halves (2^14 .. 2^15 at most), and its inverse.
struct RowScale {
    float up, down;
};

__device__ __forceinline__ RowScale row_scale(float largest)
{
    int up = 127 + 14 - (int)(__float_as_uint(largest) >> 23);
    up = largest == 0.f ? 0 : max(-112, min(up, 100));
    return RowScale{__uint_as_float((uint32_t)(127 + up) << 23), __uint_as_float((uint32_t)(127 - up) << 23)};
}

}  // namespace fa
