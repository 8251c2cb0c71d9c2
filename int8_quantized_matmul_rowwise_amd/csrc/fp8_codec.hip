// e4m3 codes and power-of-two scales of 16-bit matrices (the format: fp8_common.hpp).
//
// fp8_rows_kernel: one scale per row and group of 128 columns (activations before a product).
//   16 lanes take a group, 16 bytes each; HBM-bound, 2 + 1 bytes per value.
// fp8_tile_kernel: one workgroup per 128 x 128 tile, read once into registers (each thread 8
//   rows x 8 columns), from which it makes, as the caller asks,
//     BLOCK  one scale for the tile (weights): codes transposed and, if wanted, in order;
//     COLS   one scale per column of the tile, codes transposed (operands of the weight
//            gradient, whose sum runs over the rows), and with ROWS also
//     ROWS   one scale per row of the tile, codes in order, from the same read.
//   The transposed codes pass through LDS, where piece p (8 rows) of a column sits at piece
//   p ^ (column / 8 % 16): the 8-byte writes of the 16 lanes of a row and the 16-byte reads of
//   a column then spread over all banks.
// Code rows are padded with zeros to a multiple of 128, a weight's scale rows to one of 4.
// HBM-bound: 28672 x 8192 weights, both orders, 184 us = 5.1 TB/s; 2048 x 16384 (ROWS and COLS) and
// 2048 x 4096 (COLS) in one launch 36 us = 4.2 TB/s (two launches 43 us; 67 us with maxima passed
// between lanes through LDS one value at a time and registers for two waves a SIMD: now two
// patterns to a dword, lane operands, at most 80 registers).
#include "fp8_common.hpp"
#include "launch.hpp"

namespace llmint8 {

namespace {

template <int DT>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const uint16_t* __restrict__ X, int64_t M, int64_t K,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                                                       int32_t* __restrict__ zero, int64_t n_zero) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_zero; i += (int64_t)gridDim.x * 256) zero[i] = 0;
    const int64_t kp = fp8_pitch(K), ng = ceil_div(K, 128);
    const int64_t total = M * ng;
    const int sl = threadIdx.x & 15;
    for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; b < total; b += (int64_t)gridDim.x * 16) {
        const int64_t row = b / ng, g = b - row * ng;
        const int64_t k = g * 128 + 8 * sl;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (k < K) v = *(const u32x4*)(X + row * K + k);  // K is a multiple of 8
        const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)row_max(max_pattern(magnitudes(v)))));
        *(u32x2*)(q + row * kp + k) = e4m3x8<DT>(v, e8m0_value(e));
        if (sl == 0) s[fp8_row_scale_at(row, g, M)] = (uint8_t)e;
    }
}

struct TileParams {
    const uint16_t* A;  // R x C, row-major
    int64_t R, C;
    uint8_t* q;   // codes in order: R x pitch(C), or NULL
    uint8_t* s;   // their scales: BLOCK ceil(R/128) x sp(C), ROWS fp8_row_scale_at
    uint8_t* qt;  // codes transposed: C x pitch(R)
    uint8_t* st;  // their scales: BLOCK ceil(C/128) x sp(R), COLS fp8_row_scale_at
};

// One tile.  MODE 0: BLOCK, transposed codes; 1: BLOCK, both; 2: COLS, with ROWS where q is given
struct TileShared {
    __attribute__((aligned(16))) uint8_t tile[128 * 128];
    u32x4 red[4][16];
    __attribute__((aligned(16))) uint8_t col_e[128], row_e[128];  // the scales' bytes
};

template <int DT, int MODE>
__device__ __forceinline__ void code_tile(const TileParams& p, int64_t tc, int64_t tr, TileShared& sh) {
    constexpr bool BLOCK = MODE < 2;
    uint8_t *const tile = sh.tile, *const col_e = sh.col_e, *const row_e = sh.row_e;
    auto& red = sh.red;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int cc = tid & 15, rr = tid >> 4;  // columns 8 cc .. + 7, rows 8 rr .. + 7 of the tile
    const int64_t c0 = tc * 128, r0 = tr * 128;
    const int64_t cpitch = fp8_pitch(p.C), rpitch = fp8_pitch(p.R);
    const int64_t csp = fp8_scale_pitch_of(p.C), rsp = fp8_scale_pitch_of(p.R);
    const bool last_c = c0 + 128 >= p.C, last_r = r0 + 128 >= p.R;
    const int64_t c = c0 + 8 * cc;
    // rows past R and columns past C read zero
    const int64_t rows = p.R - r0 < 128 ? p.R - r0 : 128;
    const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(p.A + r0 * p.C, rows * p.C * 2);
    const uint32_t row_bytes = (uint32_t)p.C * 2, at = c < p.C ? 8 * rr * row_bytes + (uint32_t)c * 2 : 0x80000000u;
    u32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, at + u * row_bytes, 0, 0));
    // ---- codes in order
    if (MODE == 2 && p.q) {  // ROWS
        uint32_t es[2] = {0u, 0u};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)row_max(max_pattern(magnitudes(v[u])))));
            es[u >> 2] |= e << (8 * (u & 3));
            const int64_t r = r0 + 8 * rr + u;
            if (r < p.R) *(u32x2*)(p.q + r * cpitch + c) = e4m3x8<DT>(v[u], e8m0_value(e));
        }
        if (cc == 0) *(u32x2*)(row_e + 8 * rr) = u32x2{es[0], es[1]};
    }
    // ---- the scales of the transposed codes: largest patterns of the tile or of its columns
    float sv[8];
    u32x4 m = magnitudes(v[0]);  // of this thread's 8 columns over its 8 rows
#pragma unroll
    for (int u = 1; u < 8; ++u)
#pragma unroll
        for (int d = 0; d < 4; ++d) m[d] = max_patterns(m[d], v[u][d] & 0x7fff7fffu);
    if constexpr (BLOCK) {
        const uint32_t t = max_patterns_rows(row_max(max_pattern(m)));
        if (lane == 0) red[w][0][0] = t;
        __syncthreads();
        uint32_t a = red[0][0][0];
#pragma unroll
        for (int i = 1; i < 4; ++i) a = a > red[i][0][0] ? a : red[i][0][0];
        const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)a));
#pragma unroll
        for (int j = 0; j < 8; ++j) sv[j] = e8m0_value(e);
        if (tid == 0) {
            p.st[tc * rsp + tr] = (uint8_t)e;
            if (last_r)
                for (int64_t i = tr + 1; i < rsp; ++i) p.st[tc * rsp + i] = 0;
            if constexpr (MODE == 1) {
                p.s[tr * csp + tc] = (uint8_t)e;
                if (last_c)
                    for (int64_t i = tc + 1; i < csp; ++i) p.s[tr * csp + i] = 0;
            }
        }
    } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) m[d] = max_patterns_rows(m[d]);
        if (lane < 16) red[w][cc] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) m[d] = max_patterns(m[d], red[i][cc][d]);
        uint32_t es[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)(m[j >> 1] >> (16 * (j & 1)))));
            es[j >> 2] |= e << (8 * (j & 3));
            sv[j] = e8m0_value(e);
        }
        if (rr == 0) *(u32x2*)(col_e + 8 * cc) = u32x2{es[0], es[1]};
    }
    if constexpr (MODE == 1) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t r = r0 + 8 * rr + u;
            if (r < p.R) *(u32x2*)(p.q + r * cpitch + c) = e4m3x8<DT>(v[u], sv[0]);
        }
    }
    // ---- codes transposed: 8 rows of a column are 8 bytes of its output row
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        u32x4 col;  // the column's 8 rows
#pragma unroll
        for (int u = 0; u < 4; ++u)  // v_perm: bytes 0-3 of the second operand, 4-7 of the first
            col[u] = __builtin_amdgcn_perm(v[2 * u + 1][j >> 1], v[2 * u][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
        *(u32x2*)(tile + (8 * cc + j) * 128 + ((rr ^ cc) << 3)) = e4m3x8<DT>(col, sv[j]);
    }
    __syncthreads();
    if constexpr (!BLOCK) {
        // 64 scales are 16 dwords of four 16 apart (those past the last are padding)
        const int at = 64 * ((tid >> 4) & 1) + cc;
        if (tid < 32 && c0 + at - cc < p.C)
            *(uint32_t*)(p.st + fp8_row_scale_at(c0 + at, tr, p.C)) =
                col_e[at] | (uint32_t)col_e[at + 16] << 8 | (uint32_t)col_e[at + 32] << 16 | (uint32_t)col_e[at + 48] << 24;
        if (p.q) {
            if (tid >= 64 && tid < 96 && r0 + at - cc < p.R)
                *(uint32_t*)(p.s + fp8_row_scale_at(r0 + at, tc, p.R)) =
                    row_e[at] | (uint32_t)row_e[at + 16] << 8 | (uint32_t)row_e[at + 32] << 16 | (uint32_t)row_e[at + 48] << 24;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = 32 * i + (tid >> 3), piece = tid & 7;  // 16 bytes = row pieces 2 piece, 2 piece + 1
        const int x = (col >> 3) & 15;
        u32x4 t = *(const u32x4*)(tile + col * 128 + ((((2 * piece) ^ x) >> 1) << 4));
        if (x & 1) t = u32x4{t[2], t[3], t[0], t[1]};
        if (c0 + col < p.C) *(u32x4*)(p.qt + (c0 + col) * rpitch + r0 + 16 * piece) = t;
    }
}

template <int DT, int MODE>
__global__ __launch_bounds__(256, 6) void fp8_tile_kernel(TileParams p) {
    __shared__ TileShared sh;
    code_tile<DT, MODE>(p, blockIdx.x, blockIdx.y, sh);
}

// Both operands of the weight gradient in one launch: the tiles of `a`, then those of `b`.  Zeroes
// the counters of the products that follow.
template <int DT>
__global__ __launch_bounds__(256, 6) void fp8_cols_kernel(TileParams a, TileParams b, int tiles_a, int32_t* zero, int64_t n_zero) {
    __shared__ TileShared sh;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_zero; i += (int64_t)gridDim.x * 256) zero[i] = 0;
    const bool first = (int)blockIdx.x < tiles_a;
    const TileParams p{first ? a.A : b.A,  first ? a.R : b.R,   first ? a.C : b.C,  first ? a.q : b.q,
                       first ? a.s : b.s, first ? a.qt : b.qt, first ? a.st : b.st};
    const int t = first ? blockIdx.x : blockIdx.x - tiles_a, across = (int)ceil_div(p.C, 128), down = __builtin_amdgcn_readfirstlane(t / across);
    code_tile<DT, 2>(p, t - down * across, down, sh);
}

template <int MODE>
hipError_t tile_launch(int dt, const TileParams& p, hipStream_t stream) {
    const dim3 g((unsigned)ceil_div(p.C, 128), (unsigned)ceil_div(p.R, 128));
    if (dt == F16) fp8_tile_kernel<F16, MODE><<<g, 256, 0, stream>>>(p);
    else fp8_tile_kernel<BF16, MODE><<<g, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_weight(int dt, const void* W, int64_t K, int64_t N, uint8_t* Wq, uint8_t* s_w, uint8_t* WqT,
                             uint8_t* s_wT, hipStream_t stream) {
    if (K == 0 || N == 0) return hipSuccess;
    const TileParams p{(const uint16_t*)W, K, N, WqT, s_wT, Wq, s_w};
    return WqT ? tile_launch<1>(dt, p, stream) : tile_launch<0>(dt, p, stream);
}

hipError_t launch_fp8_rows(int dt, const void* X, int64_t M, int64_t K, uint8_t* q, uint8_t* s, int32_t* zero,
                           int64_t n_zero, hipStream_t stream) {
    if (M == 0 || K == 0) return hipSuccess;
    const int64_t need = ceil_div(M * ceil_div(K, 128), 16);
    const unsigned grid = (unsigned)(need < 16384 ? need : 16384);
    if (dt == F16) fp8_rows_kernel<F16><<<grid, 256, 0, stream>>>((const uint16_t*)X, M, K, q, s, zero, n_zero);
    else fp8_rows_kernel<BF16><<<grid, 256, 0, stream>>>((const uint16_t*)X, M, K, q, s, zero, n_zero);
    return hipGetLastError();
}

hipError_t launch_fp8_cols(int dt, const void* A, const void* B, int64_t R, int64_t CA, int64_t CB, uint8_t* at, uint8_t* s_at,
                           uint8_t* a, uint8_t* s_a, uint8_t* bt, uint8_t* s_bt, int32_t* zero, int64_t n_zero,
                           hipStream_t stream) {
    if (R == 0 || CA == 0 || CB == 0) return hipSuccess;
    const TileParams pa{(const uint16_t*)A, R, CA, a, s_a, at, s_at}, pb{(const uint16_t*)B, R, CB, nullptr, nullptr, bt, s_bt};
    const int64_t rows = ceil_div(R, 128), ta = rows * ceil_div(CA, 128), tb = rows * ceil_div(CB, 128);
    const unsigned grid = (unsigned)(ta + tb);
    if (dt == F16) fp8_cols_kernel<F16><<<grid, 256, 0, stream>>>(pa, pb, (int)ta, zero, n_zero);
    else fp8_cols_kernel<BF16><<<grid, 256, 0, stream>>>(pa, pb, (int)ta, zero, n_zero);
    return hipGetLastError();
}

}  // namespace llmint8
