// Device-side helpers of the e4m3 block-scaled operators (gfx950).
//
// A group of values with the largest magnitude a has the scale s = 2^e, the smallest power of
// two >= 2^-127 with a <= 448 s, kept as its e8m0 byte e + 127; the code of x is the nearest
// e4m3 value (ties to even) of x / s, which is exact before that one rounding.  Powers of two
// are what the matrix unit's scaled instruction takes: it applies both operands' scales itself.
#pragma once

#include "common.hpp"

namespace llmint8 {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kFp8Block = 128;  // values of a group along each axis

__host__ __device__ constexpr int64_t fp8_pitch(int64_t n) { return round_up(n, 128); }
__host__ __device__ constexpr int64_t fp8_scale_pitch_of(int64_t n) { return round_up(ceil_div(n, 128), 4); }

// The scale's byte from the largest magnitude: 448 = 1.75 * 2^8, so the exponent of a is
// raised by one where its mantissa is above 1.75, and lowered by 8.
__device__ __forceinline__ uint32_t e8m0_of(float a) {
    const int b = (int)((__builtin_bit_cast(uint32_t, a) + 0x1fffffu) >> 23) - 8;
    return b > 0 ? (uint32_t)b : 0u;
}
// 1 / s (a byte is at most 248: the exponent stays in range), and s itself
__device__ __forceinline__ float e8m0_inverse(uint32_t b) { return __builtin_bit_cast(float, (254u - b) << 23); }
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __builtin_bit_cast(float, b ? b << 23 : 0x00400000u);
}

// Four codes, the first in the low byte.  |v| <= 448 or not finite (which gives NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
    return (uint32_t)p;
}

// Eight 16-bit values (one 16-byte piece): their magnitudes as patterns, whose unsigned order
// is the order of the magnitudes (an infinity above the numbers, a NaN above that).
__device__ __forceinline__ uint32_t max_pattern(const u32x4& v, uint32_t m) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t a = v[d] & 0x7fff7fffu;
        const uint32_t lo = a & 0xffffu, hi = a >> 16;
        m = m > lo ? m : lo;
        m = m > hi ? m : hi;
    }
    return m;
}

template <int DT>
__device__ __forceinline__ u32x2 e4m3x8(const u32x4& v, float inv) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(to_f32<DT>((uint16_t)(v[k >> 1] >> (16 * (k & 1)))), inv);
    u32x2 q;
    q[0] = e4m3x4(f[0], f[1], f[2], f[3]);
    q[1] = e4m3x4(f[4], f[5], f[6], f[7]);
    return q;
}

}  // namespace llmint8
