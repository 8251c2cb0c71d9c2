// Device-side helpers of the 4-bit floating point operators (gfx950).
//
// A group of 32 values with the largest magnitude a has the scale s = 2^e, the smallest power of
// two >= 2^-127 with a <= 7 s, kept as its e8m0 byte e + 127; the code of x is the nearest e2m1
// value (0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to even, magnitudes above 6 to 6) of x / s, which is exact
// before that one rounding.  7, and not 6 (the largest code): what lies between rounds to 6 at half
// the step of the next scale.  On normal values a group of 32 is off by 11.2 % of its norm with 7,
// 11.5 % with 6 or 8; on values of a t distribution with 4 degrees 12.9, 13.9 and 13.1 %.
// A group with a value that is not finite has the byte 255 (NaN), and stands for NaN as a whole.
#pragma once

#include "fp8_common.hpp"

namespace llmint8 {

// Codes: two to a byte, the first in the low half, a row over n values padded to a multiple of 256
// (a line of 128 bytes).
__host__ __device__ constexpr int64_t fp4_pitch(int64_t n) { return ceil_div(n, 256) * 128; }

// Scales: tiles of 32 rows x 256 values, 256 bytes each, as the matrix instruction takes them: a
// dword per lane (row mod 16, and group mod 4 in the lane's upper bits), of which the instruction
// picks a byte: rows 16 apart, and the two halves of 128 values.
__host__ __device__ constexpr int64_t fp4_scale_pitch_of(int64_t n) { return ceil_div(n, 256) * 256; }  // of 32 rows
__host__ __device__ constexpr int64_t fp4_scale_at(int64_t r, int64_t g, int64_t pitch) {
    return (r >> 5) * pitch + (g >> 3) * 256 + (g & 3) * 64 + (r & 15) * 4 + ((g >> 2) & 1) * 2 + ((r >> 4) & 1);
}
__host__ __device__ constexpr int64_t fp4_scale_bytes(int64_t rows, int64_t n) { return ceil_div(rows, 32) * fp4_scale_pitch_of(n); }

// The scale's byte from the largest magnitude as a 16-bit pattern: 7 = 1.75 * 2^2, so the exponent is
// raised by one where its mantissa is above 1.75, and lowered by 2.
template <int DT>
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t pattern) {
    const int b = (int)((__builtin_bit_cast(uint32_t, to_f32<DT>((uint16_t)pattern)) + 0x1fffffu) >> 23) - 2;
    return pattern >= (DT == F16 ? 0x7c00u : 0x7f80u) ? 255u : (b > 0 ? (uint32_t)b : 0u);
}

// The value of the scale at which a group is coded.  With byte 255 (a finite number needs at most 253) that is
// 2^127, where a zero still has the code zero, so that what pads a row stays zero: at NaN itself the
// instruction codes a zero as something else.
__device__ __forceinline__ float fp4_code_scale(uint32_t e) { return e8m0_value(e < 254u ? e : 254u); }

// Codes of two 16-bit values (a pattern pair) at the scale's value s, into byte B of `old`: the
// instruction divides by the power of two, rounds once and saturates.
template <int DT, int B>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t old, uint32_t v, float s) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    if constexpr (DT == F16) return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(v2h, v), s, B);
    else return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(v2bf, v), s, B);
}
template <int DT>
__device__ __forceinline__ uint32_t e2m1x8(const u32x4& v, float s) {
    return e2m1x2<DT, 3>(e2m1x2<DT, 2>(e2m1x2<DT, 1>(e2m1x2<DT, 0>(0u, v[0], s), v[1], s), v[2], s), v[3], s);
}

// The largest of the four lanes of a quad, in all of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0xb1, 0xf, 0xf, false);  // lanes 1 0 3 2
    m = m > o ? m : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x4e, 0xf, 0xf, false);  // lanes 2 3 0 1
    return m > o ? m : o;
}

}  // namespace llmint8
