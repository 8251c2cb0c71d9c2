// e2m1 codes with power-of-two scales of 16-bit matrices, and back (the format: mxfp4_common.hpp).
//
// mxfp4_rows_kernel: groups along the rows (activations, weights kept one row per output).  A
//   workgroup takes a tile of 32 rows x 256 values: 32 lanes a row, 8 values each, four passes of 8
//   rows; a quad of lanes holds a group.  The tile's scales meet in LDS and leave as whole dwords.
// mxfp4_columns_kernel: groups along the columns (a K x N weight): a workgroup takes 256 rows x 128
//   columns; a thread reads one group of 4 columns (32 rows, 8 bytes each), so that a group's maximum
//   and codes are its own, and turns them by pairs of rows.  The codes of a column, 16 bytes a
//   thread, meet in LDS (piece g of column c at piece g ^ (c / 4 % 8)) and leave as lines of 128 bytes.
// mxfp4_values_kernel: the values of codes, 8 to a thread.
// All three are bound by memory: 2 + 0.53 bytes a value.  Rows of 8192 x 28672 126 us, back 121 us (4.7 and
// 4.9 TB/s; a 2 GiB copy 4.96); columns of 2064 x 7424 9.6 us, back 9.4 (4.0 and 4.1 TB/s, a launch's start
// included); rows of 16 x 8192 3.0 us, the latency of a load, a join and a store.
// Rows: tiles of 32 rows, since the format keeps the scales of 32 rows together, so that a workgroup writes
// whole lines of codes and of scales, and four loads a thread under way before the first is used.  Columns: a
// group's 32 rows in one thread, since a maximum over lanes of different rows would take five exchanges a
// group, and the turn of 16-bit values through LDS four times the bytes of the turn of codes.
#include "launch.hpp"
#include "mxfp4_common.hpp"

namespace llmint8 {

namespace {

template <int DT>
__global__ __launch_bounds__(256) void mxfp4_rows_kernel(const uint16_t* __restrict__ X, int64_t R, int64_t C, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ s, int32_t* __restrict__ zero, int64_t n_zero) {
    __shared__ __attribute__((aligned(16))) uint8_t scales[256];
    const uint32_t tiles = (uint32_t)ceil_div(C, 256), id = blockIdx.x;
    for (int64_t i = (int64_t)id * 256 + threadIdx.x; i < n_zero; i += (int64_t)gridDim.x * 256) zero[i] = 0;
    const int64_t tr = id / tiles, tc = id % tiles;
    const int sub = threadIdx.x >> 5, sl = threadIdx.x & 31;
    const int64_t c = tc * 256 + 8 * sl, pitch = fp4_pitch(C);
    // rows past R and columns past C read zero
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(X + tr * 32 * C, (R - tr * 32 < 32 ? R - tr * 32 : 32) * C * 2);
    const uint32_t row_bytes = (uint32_t)C * 2, at = c < C ? sub * row_bytes + (uint32_t)c * 2 : 0x80000000u;  // C is a multiple of 8
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, c < C ? at + 8 * i * row_bytes : at, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = tr * 32 + 8 * i + sub;
        const uint32_t e = fp4_scale_byte<DT>(quad_max(max_pattern(magnitudes(v[i]))));
        if (r < R) *(uint32_t*)(q + r * pitch + (c >> 1)) = e2m1x8<DT>(v[i], fp4_code_scale(e));
        if ((sl & 3) == 0) scales[fp4_scale_at(8 * i + sub, sl >> 2, 256)] = (uint8_t)e;  // (rows past the last: zeros)
    }
    __syncthreads();
    if (threadIdx.x < 64) ((uint32_t*)s)[(int64_t)id * 64 + threadIdx.x] = ((const uint32_t*)scales)[threadIdx.x];
}

template <int DT>
__global__ __launch_bounds__(256) void mxfp4_columns_kernel(const uint16_t* __restrict__ A, int64_t R, int64_t C, uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ s) {
    __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
    __shared__ __attribute__((aligned(16))) uint8_t scales[1024];
    const int tid = threadIdx.x, cc = tid & 31, g = tid >> 5;  // columns 4 cc .. + 3, group g of the tile
    const int64_t c0 = (int64_t)blockIdx.x * 128, r0 = (int64_t)blockIdx.y * 256;
    // rows past R and columns past C read zero
    const int64_t rows = R - r0 < 256 ? R - r0 : 256;
    const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(A + r0 * C, rows * C * 2);
    const uint32_t row_bytes = (uint32_t)C * 2;
    const bool in = c0 + 4 * cc < C;  // C is a multiple of 4
    const uint32_t at = in ? 32 * g * row_bytes + (uint32_t)(c0 + 4 * cc) * 2 : 0x80000000u;
    u32x2 v[32];
#pragma unroll
    for (int u = 0; u < 32; ++u)
        v[u] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(ra, in ? at + u * row_bytes : at, 0, 0));
    uint32_t m[2] = {0u, 0u};  // of the four columns, two to a dword
#pragma unroll
    for (int u = 0; u < 32; ++u)
#pragma unroll
        for (int d = 0; d < 2; ++d) m[d] = max_patterns(m[d], v[u][d] & 0x7fff7fffu);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t e = fp4_scale_byte<DT>((m[j >> 1] >> (16 * (j & 1))) & 0xffffu);
        const float sv = fp4_code_scale(e);
        const int col = 4 * cc + j;
        scales[fp4_scale_at(col, g, 256)] = (uint8_t)e;
        u32x4 code;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            u32x4 pair;  // rows 8 w .. + 7 of the column; v_perm: bytes 0-3 of the second operand, 4-7 of the first
#pragma unroll
            for (int u = 0; u < 4; ++u)
                pair[u] = __builtin_amdgcn_perm(v[8 * w + 2 * u + 1][j >> 1], v[8 * w + 2 * u][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
            code[w] = e2m1x8<DT>(pair, sv);
        }
        *(u32x4*)(tile + col * 128 + ((g ^ (cc & 7)) << 4)) = code;
    }
    __syncthreads();
    const int64_t pitch = fp4_pitch(R), sp = fp4_scale_pitch_of(R);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = 32 * i + (tid >> 3), piece = tid & 7;
        const u32x4 t = *(const u32x4*)(tile + col * 128 + ((piece ^ ((col >> 2) & 7)) << 4));
        if (c0 + col < C) *(u32x4*)(q + (c0 + col) * pitch + (r0 >> 1) + 16 * piece) = t;
    }
    const int64_t first = (c0 >> 5) + (tid >> 6);  // of the four scale tiles
    if (first * 32 < C) *(uint32_t*)(s + first * sp + (int64_t)blockIdx.y * 256 + 4 * (tid & 63)) = *(const uint32_t*)(scales + 4 * tid);
}

// A thread's 8 values: codes and scale apart (a code's value is exact in fp32, the product with the
// scale too, but for a NaN of the scale), one rounding to the output's type.
template <int DT>
__global__ __launch_bounds__(256) void mxfp4_values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t rows,
                                                           int64_t n, uint16_t* __restrict__ A) {
    const int64_t pieces = n >> 3, pitch = fp4_pitch(n), sp = fp4_scale_pitch_of(n), total = rows * pieces;  // n is a multiple of 8
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / pieces, c = i - r * pieces;
        const uint32_t code = *(const uint32_t*)(q + r * pitch + 4 * c);
        const uint32_t e = s[fp4_scale_at(r, c >> 2, sp)];
        const float sv = e == 255u ? __builtin_nanf("") : e8m0_value(e);
        typedef float v2f __attribute__((ext_vector_type(2)));
        v2f f[4];
        f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
        f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1);
        f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2);
        f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3);
        u32x4 out;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            out[j] = (uint32_t)from_f32<DT>(f[j][0] * sv) | ((uint32_t)from_f32<DT>(f[j][1] * sv) << 16);
        *(u32x4*)(A + r * n + 8 * c) = out;
    }
}

}  // namespace

hipError_t launch_mxfp4_rows(int dt, const void* X, int64_t R, int64_t C, uint8_t* q, uint8_t* s, int32_t* zero, int64_t n_zero,
                             hipStream_t stream) {
    if (R == 0 || C == 0) return hipSuccess;
    const unsigned grid = (unsigned)(ceil_div(R, 32) * ceil_div(C, 256));
    if (dt == F16) mxfp4_rows_kernel<F16><<<grid, 256, 0, stream>>>((const uint16_t*)X, R, C, q, s, zero, n_zero);
    else mxfp4_rows_kernel<BF16><<<grid, 256, 0, stream>>>((const uint16_t*)X, R, C, q, s, zero, n_zero);
    return hipGetLastError();
}

hipError_t launch_mxfp4_columns(int dt, const void* A, int64_t R, int64_t C, uint8_t* q, uint8_t* s, hipStream_t stream) {
    if (R == 0 || C == 0) return hipSuccess;
    const dim3 grid((unsigned)ceil_div(C, 128), (unsigned)ceil_div(R, 256));
    if (dt == F16) mxfp4_columns_kernel<F16><<<grid, 256, 0, stream>>>((const uint16_t*)A, R, C, q, s);
    else mxfp4_columns_kernel<BF16><<<grid, 256, 0, stream>>>((const uint16_t*)A, R, C, q, s);
    return hipGetLastError();
}

hipError_t launch_mxfp4_values(int dt, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t n, void* A, hipStream_t stream) {
    if (rows == 0 || n == 0) return hipSuccess;
    const int64_t need = ceil_div(rows * (n >> 3), 256);
    const unsigned grid = (unsigned)(need < 65536 ? need : 65536);
    if (dt == F16) mxfp4_values_kernel<F16><<<grid, 256, 0, stream>>>(q, s, rows, n, (uint16_t*)A);
    else mxfp4_values_kernel<BF16><<<grid, 256, 0, stream>>>(q, s, rows, n, (uint16_t*)A);
    return hipGetLastError();
}

}  // namespace llmint8
