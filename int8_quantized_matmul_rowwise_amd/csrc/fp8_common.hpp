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

__host__ __device__ constexpr int64_t fp8_pitch(int64_t n) { return round_up(n, 128); }
__host__ __device__ constexpr int64_t fp8_scale_pitch_of(int64_t n) { return round_up(ceil_div(n, 128), 4); }

// The scales of coded activations, one per row and group, as the product kernels take them: for
// each group, for each 64 rows, a dword per row mod 16 that holds the bytes of the four rows
// 16 apart -- the matrix instruction picks a byte of its scale operand, so one dword per lane
// scales four pieces of 16 rows.  What the bytes of rows past the last hold has no effect.
__host__ __device__ constexpr int64_t fp8_row_scale_at(int64_t r, int64_t g, int64_t rows) {
    return (g * ceil_div(rows, 64) + (r >> 6)) * 64 + (r & 15) * 4 + ((r >> 4) & 3);
}
__host__ __device__ constexpr int64_t fp8_row_scale_bytes(int64_t rows, int64_t sum) {
    return ceil_div(sum, 128) * round_up(rows, 64);
}

// The scale's byte from the largest magnitude: 448 = 1.75 * 2^8, so the exponent of a is
// raised by one where its mantissa is above 1.75, and lowered by 8.
__device__ __forceinline__ uint32_t e8m0_of(float a) {
    const int b = (int)((__builtin_bit_cast(uint32_t, a) + 0x1fffffu) >> 23) - 8;
    return b > 0 ? (uint32_t)b : 0u;
}
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __builtin_bit_cast(float, b ? b << 23 : 0x00400000u);
}

// Magnitudes are compared as 16-bit patterns, two to a dword: their unsigned order is the order of
// the magnitudes (an infinity above the numbers, a NaN above that).
__device__ __forceinline__ uint32_t max_patterns(uint32_t a, uint32_t b) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ u32x4 magnitudes(const u32x4& v) { return v & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t max_pattern(const u32x4& m) {  // of eight magnitudes, one pattern
    const uint32_t a = max_patterns(max_patterns(m[0], m[1]), max_patterns(m[2], m[3]));
    return (a & 0xffffu) > a >> 16 ? a & 0xffffu : a >> 16;
}
// The largest of the 16 lanes of a row, in all of them: rotations as operands of the maximum.
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
#define LLMINT8_ROR(N)                                                                          \
    do {                                                                                        \
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x120 + N, 0xf, 0xf, false); \
        m = m > o ? m : o;                                                                      \
    } while (0)
    LLMINT8_ROR(8);
    LLMINT8_ROR(4);
    LLMINT8_ROR(2);
    LLMINT8_ROR(1);
#undef LLMINT8_ROR
    return m;
}
// The larger patterns of lanes 16 apart, then 32 apart: of the four rows of a wave, in all of them.
__device__ __forceinline__ uint32_t max_patterns_rows(uint32_t m) {
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max_patterns(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max_patterns(b[0], b[1]);
}

// Codes of two 16-bit values (a pattern pair) at the scale's value s, into half HI of `old`: the
// instruction divides by the power of two and rounds once (not finite: NaN).
template <int DT, bool HI>
__device__ __forceinline__ uint32_t e4m3x2(uint32_t old, uint32_t v, float s) {
    typedef short v2s __attribute__((ext_vector_type(2)));
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    v2s o = __builtin_bit_cast(v2s, old);
    if constexpr (DT == F16) o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(o, __builtin_bit_cast(v2h, v), s, HI);
    else o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(v2bf, v), s, HI);
    return __builtin_bit_cast(uint32_t, o);
}

template <int DT>
__device__ __forceinline__ u32x2 e4m3x8(const u32x4& v, float s) {
    u32x2 q;
    q[0] = e4m3x2<DT, true>(e4m3x2<DT, false>(0u, v[0], s), v[1], s);
    q[1] = e4m3x2<DT, true>(e4m3x2<DT, false>(0u, v[2], s), v[3], s);
    return q;
}

// After a loop of matrix instructions, before their results are read: the wait states the reader
// needs, which the compiler (ROCm 7.2) has been seen to leave out across a branch.
__device__ __forceinline__ void mfma_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)bytes, 0x00020000);
}

// ---- sums split over workgroups
constexpr int kCoherent = 16;  // cache policy: coherent across the XCDs, past their L2s

// A workgroup's share of a sum is in memory (stores of every wave issued): true for the one that
// finds all `parts` in, which leaves the counter at zero.  flag: a word of LDS.
__device__ __forceinline__ bool last_part(int32_t* counter, int parts, int* flag) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const int done = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
        *flag = done == parts;
        if (done == parts) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    // (one answer for the wave: a branch on a lane's value would make the compiler take all that the
    // code before it places -- resources, offsets -- for lanes' values, and loop over them)
    const bool last = __builtin_amdgcn_readfirstlane(*flag) != 0;
    __syncthreads();  // before the word is used again
    return last;
}
__device__ __forceinline__ v4f load_part(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t at) {
    return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, off, at, kCoherent));
}
__device__ __forceinline__ void store_part(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t at, const v4f& v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, off, at, kCoherent);
}

}  // namespace llmint8
