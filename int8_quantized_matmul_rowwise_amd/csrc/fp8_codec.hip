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
        uint32_t m = max_pattern(v, 0u);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
            const uint32_t o = (uint32_t)__shfl_xor((int)m, off, kWave);
            m = m > o ? m : o;
        }
        const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)m));
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
    int32_t* zero;
    int64_t n_zero;
};

// MODE 0: BLOCK, transposed codes; 1: BLOCK, both; 2: COLS; 3: COLS and ROWS
template <int DT, int MODE>
__global__ __launch_bounds__(256) void fp8_tile_kernel(TileParams p) {
    constexpr bool BLOCK = MODE < 2;
    __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
    __shared__ uint32_t red[4][128];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int cc = tid & 15, rr = tid >> 4;  // columns 8 cc .. + 7, rows 8 rr .. + 7 of the tile
    const int64_t tc = blockIdx.x, tr = blockIdx.y;
    if constexpr (!BLOCK) {
        const int64_t id = (tr * gridDim.x + tc) * 256 + tid;
        for (int64_t i = id; i < p.n_zero; i += (int64_t)gridDim.x * gridDim.y * 256) p.zero[i] = 0;
    }
    const int64_t c0 = tc * 128, r0 = tr * 128;
    const int64_t cpitch = fp8_pitch(p.C), rpitch = fp8_pitch(p.R);
    const int64_t csp = fp8_scale_pitch_of(p.C), rsp = fp8_scale_pitch_of(p.R);
    const bool last_c = c0 + 128 >= p.C, last_r = r0 + 128 >= p.R;
    const int64_t c = c0 + 8 * cc;
    u32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t r = r0 + 8 * rr + u;
        v[u] = u32x4{0u, 0u, 0u, 0u};
        if (r < p.R && c < p.C) v[u] = *(const u32x4*)(p.A + r * p.C + c);  // C is a multiple of 8
    }
    // ---- codes in order
    if constexpr (MODE == 3) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            uint32_t m = max_pattern(v[u], 0u);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)m, off, kWave);
                m = m > o ? m : o;
            }
            const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)m));
            const int64_t r = r0 + 8 * rr + u;
            if (r < p.R) {
                *(u32x2*)(p.q + r * cpitch + c) = e4m3x8<DT>(v[u], e8m0_value(e));
                if (cc == 0) p.s[fp8_row_scale_at(r, tc, p.R)] = (uint8_t)e;
            }
        }
    }
    // ---- the scales of the transposed codes: largest patterns of the tile or of its columns
    float sv[8];
    if constexpr (BLOCK) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) m = max_pattern(v[u], m);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const uint32_t o = (uint32_t)__shfl_xor((int)m, off, kWave);
            m = m > o ? m : o;
        }
        if (lane == 0) red[w][0] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) m = m > red[i][0] ? m : red[i][0];
        const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)m));
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
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t a = (v[u][j >> 1] >> (16 * (j & 1))) & 0x7fffu;
                m[j] = m[j] > a ? m[j] : a;
            }
#pragma unroll
            for (int off = 32; off >= 16; off >>= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)m[j], off, kWave);
                m[j] = m[j] > o ? m[j] : o;
            }
            if (lane < 16) red[w][8 * cc + j] = m[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t o = red[i][8 * cc + j];
                m[j] = m[j] > o ? m[j] : o;
            }
            const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)m[j]));
            sv[j] = e8m0_value(e);
            if (rr == 0 && c + j < p.C) p.st[fp8_row_scale_at(c + j, tr, p.C)] = (uint8_t)e;
        }
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = 32 * i + (tid >> 3), piece = tid & 7;  // 16 bytes = row pieces 2 piece, 2 piece + 1
        const int x = (col >> 3) & 15;
        u32x4 t = *(const u32x4*)(tile + col * 128 + ((((2 * piece) ^ x) >> 1) << 4));
        if (x & 1) t = u32x4{t[2], t[3], t[0], t[1]};
        if (c0 + col < p.C) *(u32x4*)(p.qt + (c0 + col) * rpitch + r0 + 16 * piece) = t;
    }
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
    const TileParams p{(const uint16_t*)W, K, N, WqT, s_wT, Wq, s_w, nullptr, 0};
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

hipError_t launch_fp8_cols(int dt, const void* A, int64_t R, int64_t C, uint8_t* qt, uint8_t* st, uint8_t* q, uint8_t* s,
                           int32_t* zero, int64_t n_zero, hipStream_t stream) {
    if (R == 0 || C == 0) return hipSuccess;
    const TileParams p{(const uint16_t*)A, R, C, q, s, qt, st, zero, n_zero};
    return q ? tile_launch<3>(dt, p, stream) : tile_launch<2>(dt, p, stream);
}

}  // namespace llmint8
