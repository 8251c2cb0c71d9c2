// Root-mean-square norm with the residual's addition, its output in 16 bits and as codes, and its
// gradient:
//   h = RN_T(x + residual),  r = 1 / sqrt(mean(h^2) + eps),  y = RN_T(h r w),
//   d = dy w,  dx = RN_T(r (d - h r^2 mean(d h)) + dh),  dw = RN_T(sum over rows of dy h r).
// Sums in fp32.  The codes are those of y after its rounding, so that they are the ones which the
// products make of y themselves.
//
// Both are bound by memory: a row is read once into registers (8 columns a piece and thread, a
// workgroup a row, up to 32768 columns and in the gradient 16384), summed over lanes, then waves, and
// written.  With few rows a row's own latency is what is left: a load, two meetings, a store.
// Norm: 1 x 4096 to 16 bits without a residual 1.8 us, 16 x 8192 to e2m1 codes 4.0; 4096 x 8192 with a residual to
// e2m1 43.8 us (5.4 TB/s), to e4m3 45.5 (5.2), to 16 bits 47.4 (5.7); 2048 x 4096 to e4m3 11.3.
// Gradient, with dw: 2048 x 4096 with dh 21 us, 8192 x 8192 with dh 106 (5.1 TB/s), 4096 x 16384 with dh 109 (4.9),
// 333 x 1040 7.6 (two launches).  dw needs a sum over rows: each
// workgroup keeps its own in registers over its rows, at most 512 rows of partial sums leave, and a second
// launch joins them in their order (3.8 to 5 us); no atomics, so results do not change from run to run.
#include "../../include/llmint8.h"
#include "launch.hpp"
#include "mxfp4_common.hpp"

namespace llmint8 {

namespace {

constexpr int64_t kMaxGrid = 1 << 20;   // workgroups of a launch: 2^32 threads are too many

// The sum over the 64 lanes, in all of them, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#define LLMINT8_ROR(N) v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, false))
    LLMINT8_ROR(8);
    LLMINT8_ROR(4);
    LLMINT8_ROR(2);
    LLMINT8_ROR(1);
#undef LLMINT8_ROR
    const auto swapped = [](uint32_t x, bool far) {  // (a bit cast of a vector's element itself would take the first one)
        const auto p = far ? __builtin_amdgcn_permlane32_swap(x, x, false, false) : __builtin_amdgcn_permlane16_swap(x, x, false, false);
        const uint32_t a = p[0], b = p[1];
        return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    };
    v = swapped(__builtin_bit_cast(uint32_t, v), false);
    return swapped(__builtin_bit_cast(uint32_t, v), true);
}

// N sums over T threads (whole waves), in all of them; red: words that the call before last may have
// used.  Every wave of the workgroup calls it.
template <int N, int T>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*red)[T / 64]) {
    constexpr int W = T / 64;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (W > 1) {
        const int lane = threadIdx.x & 63, w = (threadIdx.x % T) >> 6;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[i][w] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = red[i][0];
#pragma unroll
            for (int j = 1; j < W; ++j) v[i] += red[i][j];
        }
    }
}

template <int DT>
__device__ __forceinline__ float low(uint32_t v) { return to_f32<DT>((uint16_t)v); }
template <int DT>
__device__ __forceinline__ float high(uint32_t v) { return to_f32<DT>((uint16_t)(v >> 16)); }
template <int DT>
__device__ __forceinline__ uint32_t pack(float a, float b) { return (uint32_t)from_f32<DT>(a) | ((uint32_t)from_f32<DT>(b) << 16); }

template <int DT>
__device__ __forceinline__ u32x4 add(const u32x4& a, const u32x4& b) {
    u32x4 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = pack<DT>(low<DT>(a[d]) + low<DT>(b[d]), high<DT>(a[d]) + high<DT>(b[d]));
    return o;
}
template <int DT>
__device__ __forceinline__ float squares(const u32x4& h, float s) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float a = low<DT>(h[d]), b = high<DT>(h[d]);
        s = __builtin_fmaf(a, a, s);
        s = __builtin_fmaf(b, b, s);
    }
    return s;
}
// h w r: the product of two 16-bit values is exact in fp32, so y has one rounding before its own.
template <int DT>
__device__ __forceinline__ u32x4 scaled(const u32x4& h, const u32x4& w, float r) {
    u32x4 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = pack<DT>(low<DT>(h[d]) * low<DT>(w[d]) * r, high<DT>(h[d]) * high<DT>(w[d]) * r);
    return o;
}

// 1 / sqrt(sum / n + eps), rounded once to fp32: the hardware's estimate in 64 bits and one step of
// Newton's on it (codes of y flip where y is next to a border, so r is not left with three roundings).
__device__ __forceinline__ float inverse_root(float sum, double inv_n, float eps) {
    const double v = __builtin_fma((double)sum, inv_n, (double)eps);
    const double y = __builtin_amdgcn_rsq(v);
    const double z = y * __builtin_fma(-0.5 * v * y, y, 1.5);
    return sum < __builtin_inff() ? (float)z : (sum == sum ? 0.0f : __builtin_nanf(""));
}

// Whether rows past the last fill the last tile of scales, and the workgroups that take rows.
template <int FORMAT>
__host__ __device__ __forceinline__ bool has_padding(const NormArgs& p) {
    return FORMAT != LLMINT8_CODES_NONE && p.M % (FORMAT == LLMINT8_CODES_MXFP4 ? 32 : 64) != 0;
}
template <int FORMAT>
__device__ __forceinline__ int64_t norm_groups(const NormArgs& p, int64_t grid) { return grid - (has_padding<FORMAT>(p) ? 1 : 0); }

// The workgroup's place in its XCD's run of rows: neighbours share the lines of the codes' scales.
__device__ __forceinline__ int64_t in_runs(int64_t id, int64_t n) {
    const int64_t xcd = id & 7, per = n >> 3, rem = n & 7;
    return xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
}

// Eight neighbouring values y from column c of row `row` on, as codes and scales.
template <int DT, int FORMAT>
__device__ __forceinline__ void store_codes(const NormArgs& p, int64_t row, int64_t c, const u32x4& y) {
    if constexpr (FORMAT == LLMINT8_CODES_FP8_BLOCK) {
        const int64_t pitch = fp8_pitch(p.K);
        const uint32_t e = e8m0_of(to_f32<DT>((uint16_t)row_max(max_pattern(magnitudes(y)))));
        if (c >= pitch) return;
        *(u32x2*)(p.q + row * pitch + c) = e4m3x8<DT>(y, e8m0_value(e));
        if ((threadIdx.x & 15) == 0) p.s[fp8_row_scale_at(row, c >> 7, p.M)] = (uint8_t)e;
    } else if constexpr (FORMAT == LLMINT8_CODES_MXFP4) {
        const int64_t pitch = fp4_pitch(p.K);
        const uint32_t e = fp4_scale_byte<DT>(quad_max(max_pattern(magnitudes(y))));
        if (c >= 2 * pitch) return;
        *(uint32_t*)(p.q + row * pitch + (c >> 1)) = e2m1x8<DT>(y, fp4_code_scale(e));
        if ((threadIdx.x & 3) == 0) p.s[fp4_scale_at(row, c >> 5, fp4_scale_pitch_of(p.K))] = (uint8_t)e;
    }
}

// The scales of the rows that fill the last tile of scales: zeros, written by a workgroup of their own
// (the last one, where there are such rows), which adds nothing to the time of a row.
template <int FORMAT>
__device__ __forceinline__ void clear_scales(const NormArgs& p) {
    constexpr bool four = FORMAT == LLMINT8_CODES_MXFP4;
    const int64_t end = round_up(p.M, four ? 32 : 64);
    const int groups = (int)(four ? fp4_scale_pitch_of(p.K) / 32 : ceil_div(p.K, 128));
    for (int g = threadIdx.x; g < groups; g += blockDim.x)
        for (int64_t row = p.M; row < end; ++row) p.s[four ? fp4_scale_at(row, g, fp4_scale_pitch_of(p.K)) : fp8_row_scale_at(row, g, p.M)] = 0;
}

// A workgroup a row, V pieces of 8 columns a thread.  (p.H may be p.X or p.R: each element is read
// before it is written, by the same thread.)
template <int DT, int V, int FORMAT, int T>
__global__ __launch_bounds__(T, 4) void rmsnorm_kernel(NormArgs p) {
    __shared__ float red[2][1][T / 64];
    const int tid = threadIdx.x;
    const int64_t groups = norm_groups<FORMAT>(p, gridDim.x);
    if (FORMAT != LLMINT8_CODES_NONE && blockIdx.x >= groups) return clear_scales<FORMAT>(p);
    int turn = 0;
    for (int64_t row = in_runs(blockIdx.x, groups); row < p.M; row += groups, turn ^= 1) {
        u32x4 h[V], w[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = ((int64_t)v * T + tid) * 8;
            h[v] = w[v] = u32x4{0u, 0u, 0u, 0u};
            if (c < p.K) {  // K is a multiple of 8
                h[v] = *(const u32x4*)(p.X + row * p.K + c);
                w[v] = *(const u32x4*)(p.W + c);
            }
        }
        if (p.R) {
            u32x4 b[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = ((int64_t)v * T + tid) * 8;
                b[v] = u32x4{0u, 0u, 0u, 0u};
                if (c < p.K) b[v] = *(const u32x4*)(p.R + row * p.K + c);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = ((int64_t)v * T + tid) * 8;
                h[v] = add<DT>(h[v], b[v]);
                if (p.H && c < p.K) *(u32x4*)(p.H + row * p.K + c) = h[v];
            }
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) s[0] = squares<DT>(h[v], s[0]);
        group_sum<1, T>(s, red[turn]);
        const float r = inverse_root(s[0], p.inv_k, p.eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = ((int64_t)v * T + tid) * 8;
            // (past the row's end 0 in the place of r, which may be NaN: the codes' padding is zeros)
            const u32x4 y = scaled<DT>(h[v], w[v], FORMAT == LLMINT8_CODES_NONE || c < p.K ? r : 0.0f);
            if (p.Y && c < p.K) *(u32x4*)(p.Y + row * p.K + c) = y;
            store_codes<DT, FORMAT>(p, row, c, y);
        }
    }
}

// Rows longer than a workgroup's registers: read twice (2000 x 65536 with a residual to 16 bits 238 us, 4.4 TB/s, to
// e4m3 224, to e2m1 213).
template <int DT, int FORMAT>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormArgs p) {
    constexpr int T = 1024;
    __shared__ float red[2][1][T / 64];
    const int64_t groups = norm_groups<FORMAT>(p, gridDim.x);
    if (FORMAT != LLMINT8_CODES_NONE && blockIdx.x >= groups) return clear_scales<FORMAT>(p);
    int turn = 0;
    for (int64_t row = in_runs(blockIdx.x, groups); row < p.M; row += groups, turn ^= 1) {
        float s[1] = {0.0f};
        for (int64_t c = 8 * threadIdx.x; c < p.K; c += 8192) {
            u32x4 h = *(const u32x4*)(p.X + row * p.K + c);
            if (p.R) {
                h = add<DT>(h, *(const u32x4*)(p.R + row * p.K + c));
                if (p.H) *(u32x4*)(p.H + row * p.K + c) = h;
            }
            s[0] = squares<DT>(h, s[0]);
        }
        group_sum<1, T>(s, red[turn]);
        const float r = inverse_root(s[0], p.inv_k, p.eps);
        for (int64_t base = 0; base < p.K; base += 8192) {
            const int64_t c = base + 8 * threadIdx.x;
            u32x4 y = {0u, 0u, 0u, 0u};
            if (c < p.K) {
                u32x4 h;  // (H may have taken the place of X or R)
                if (p.R && p.H) h = *(const u32x4*)(p.H + row * p.K + c);
                else h = *(const u32x4*)(p.X + row * p.K + c);
                if (p.R && !p.H) h = add<DT>(h, *(const u32x4*)(p.R + row * p.K + c));
                y = scaled<DT>(h, *(const u32x4*)(p.W + c), r);
                if (p.Y) *(u32x4*)(p.Y + row * p.K + c) = y;
            }
            store_codes<DT, FORMAT>(p, row, c, y);
        }
    }
}

// ---- gradient

// Pieces of a row of the gradient: sums over it, then dx and what the row adds to dw.
template <int DT>
__device__ __forceinline__ void row_sums(const u32x4& h, const u32x4& dy, const u32x4& w, float (&s)[2]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float a = low<DT>(h[d]), b = high<DT>(h[d]);
        s[0] = __builtin_fmaf(a, a, s[0]);
        s[0] = __builtin_fmaf(b, b, s[0]);
        s[1] = __builtin_fmaf(low<DT>(dy[d]) * low<DT>(w[d]), a, s[1]);
        s[1] = __builtin_fmaf(high<DT>(dy[d]) * high<DT>(w[d]), b, s[1]);
    }
}
// m = r mean(d h).  (r^2 is not formed: in a row of zeros it passes fp32 with an eps below 2^-128.)
template <int DT>
__device__ __forceinline__ u32x4 row_dx(const u32x4& h, const u32x4& dy, const u32x4& w, const u32x4& dh, float r, float m) {
    u32x4 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float a = r * (low<DT>(dy[d]) * low<DT>(w[d]) - low<DT>(h[d]) * r * m) + low<DT>(dh[d]);
        const float b = r * (high<DT>(dy[d]) * high<DT>(w[d]) - high<DT>(h[d]) * r * m) + high<DT>(dh[d]);
        o[d] = pack<DT>(a, b);
    }
    return o;
}
template <int DT>
__device__ __forceinline__ void row_dw(const u32x4& h, const u32x4& dy, float r, float* acc) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        acc[2 * d] = __builtin_fmaf(low<DT>(dy[d]), low<DT>(h[d]) * r, acc[2 * d]);
        acc[2 * d + 1] = __builtin_fmaf(high<DT>(dy[d]), high<DT>(h[d]) * r, acc[2 * d + 1]);
    }
}

// T threads take a row at a time, and a workgroup blockDim.x / T rows side by side; with AHEAD the next
// row's loads are under way while a row is summed.  dw's sums stay in registers over a thread's rows, and
// those of the workgroup's rows meet in LDS at the end.
template <int DT, int V, int T, bool DW, bool AHEAD>
__global__ __launch_bounds__(AHEAD ? 512 : T, AHEAD ? 2 : 4) void rmsnorm_backward_kernel(NormBackwardArgs p) {
    constexpr int kSide = AHEAD ? 512 / T : 1;  // rows side by side, at most
    __shared__ float red[2][kSide][2][T / 64];
    __shared__ v4f joined[DW && kSide > 1 ? 2 * V * T : 1];  // a row of dw's sums
    const int tid = threadIdx.x % T, side = kSide > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / T) : 0, sides = kSide > 1 ? (int)blockDim.x / T : 1;
    u32x4 w[V];
    float acc[V][8] = {};
    const u32x4 none = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + tid) * 8;
        w[v] = c < p.K ? *(const u32x4*)(p.W + c) : none;
    }
    struct Row {
        u32x4 h[V], dy[V], dh[V];
    };
    auto load = [&](int64_t row, Row& x) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + tid) * 8;
            const bool in = c < p.K && row < p.M;
            const int64_t at = row * p.K + c;
            x.h[v] = in ? *(const u32x4*)(p.H + at) : none;
            x.dy[v] = in ? *(const u32x4*)(p.dY + at) : none;
            x.dh[v] = in && p.dH ? *(const u32x4*)(p.dH + at) : none;
        }
    };
    const int64_t step = (int64_t)gridDim.x * sides;
    int64_t row = (int64_t)blockIdx.x * sides + side;
    Row x, next;
    load(row, x);
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * sides; first < p.M; first += step, row += step, turn ^= 1) {  // (every side as often)
        if (AHEAD) load(row + step, next);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) row_sums<DT>(x.h[v], x.dy[v], w[v], s);
        group_sum<2, T>(s, red[turn][side]);
        const float r = inverse_root(s[0], p.inv_k, p.eps), m = r * (float)(s[1] * p.inv_k);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + tid) * 8;
            if (c < p.K && row < p.M) *(u32x4*)(p.dX + row * p.K + c) = row_dx<DT>(x.h[v], x.dy[v], w[v], x.dh[v], r, m);
            if constexpr (DW) row_dw<DT>(x.h[v], x.dy[v], r, acc[v]);
        }
        if (AHEAD) x = next;
        else load(row + step, x);
    }
    if constexpr (DW) {
        if constexpr (kSide > 1) {
            for (int i = 1; i < sides; ++i) {  // the sides in their order, onto the first
                __syncthreads();
                if (side == i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        joined[(2 * v) * T + tid] = v4f{acc[v][0], acc[v][1], acc[v][2], acc[v][3]};
                        joined[(2 * v + 1) * T + tid] = v4f{acc[v][4], acc[v][5], acc[v][6], acc[v][7]};
                    }
                }
                __syncthreads();
                if (side == 0) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const v4f a = joined[(2 * v) * T + tid], b = joined[(2 * v + 1) * T + tid];
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[v][e] += a[e], acc[v][4 + e] += b[e];
                    }
                }
            }
            if (side) return;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + tid) * 8;
            if (c >= p.K) continue;
            float* to = p.partial + (int64_t)blockIdx.x * p.K + c;
            *(v4f*)to = v4f{acc[v][0], acc[v][1], acc[v][2], acc[v][3]};
            *(v4f*)(to + 4) = v4f{acc[v][4], acc[v][5], acc[v][6], acc[v][7]};
        }
    }
}

// Rows longer than a workgroup's registers: read twice, and H and dY once more for dw, for which r of each
// row is kept: 2000 x 32768 with dh 172 us, of which dw takes 49 and the join 5.
template <int DT>
__global__ __launch_bounds__(1024) void rmsnorm_backward_long_kernel(NormBackwardArgs p) {
    constexpr int T = 1024;
    __shared__ float red[2][2][T / 64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = 8 * threadIdx.x; c < p.K; c += 8192)
            row_sums<DT>(*(const u32x4*)(p.H + row * p.K + c), *(const u32x4*)(p.dY + row * p.K + c), *(const u32x4*)(p.W + c), s);
        group_sum<2, T>(s, red[turn]);
        const float r = inverse_root(s[0], p.inv_k, p.eps), m = r * (float)(s[1] * p.inv_k);
        if (threadIdx.x == 0 && p.rows) p.rows[row] = r;
        for (int64_t c = 8 * threadIdx.x; c < p.K; c += 8192) {
            const u32x4 none = {0u, 0u, 0u, 0u};
            const u32x4 dh = p.dH ? *(const u32x4*)(p.dH + row * p.K + c) : none;
            *(u32x4*)(p.dX + row * p.K + c) =
                row_dx<DT>(*(const u32x4*)(p.H + row * p.K + c), *(const u32x4*)(p.dY + row * p.K + c), *(const u32x4*)(p.W + c), dh, r, m);
        }
    }
}
// dw's sums over every gridDim.y-th row: 2048 columns a workgroup.
template <int DT>
__global__ __launch_bounds__(256) void rmsnorm_dw_long_kernel(NormBackwardArgs p) {
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= p.K) return;
    float acc[8] = {};
    for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y)
        row_dw<DT>(*(const u32x4*)(p.H + row * p.K + c), *(const u32x4*)(p.dY + row * p.K + c), p.rows[row], acc);
    float* to = p.partial + (int64_t)blockIdx.y * p.K + c;
    *(v4f*)to = v4f{acc[0], acc[1], acc[2], acc[3]};
    *(v4f*)(to + 4) = v4f{acc[4], acc[5], acc[6], acc[7]};
}

// dw from the partial sums (groups x K): a workgroup 32 columns, 32 runs of rows side by side, eight
// loads of a thread under way, then joined in their order.
template <int DT>
__global__ __launch_bounds__(256) void rmsnorm_dw_join_kernel(const float* __restrict__ partial, int groups, int64_t K, uint16_t* __restrict__ dW) {
    __shared__ v4f sums[32][8];
    constexpr int U = 8;
    const int cc = threadIdx.x & 7, rr = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 32 + 4 * cc;
    const int run = (int)ceil_div(groups, 32), first = rr * run, end = first + run < groups ? first + run : groups;
    v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < K) {
        for (int g = first; g < end; g += U) {
            v4f v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = *(const v4f*)(partial + (int64_t)(g + u < end ? g + u : g) * K + c);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (g + u < end) s += v[u];
        }
    }
    sums[rr][cc] = s;
    __syncthreads();
    if (rr == 0 && c < K) {
        for (int i = 1; i < 32; ++i) s += sums[i][cc];
        *(u32x2*)(dW + c) = u32x2{pack<DT>(s[0], s[1]), pack<DT>(s[2], s[3])};
    }
}

template <int DT, int FORMAT>
hipError_t norm_launch(const NormArgs& p, const NormPlan& plan, hipStream_t stream) {
    const unsigned grid = (unsigned)(p.M < kMaxGrid ? p.M : kMaxGrid) + (has_padding<FORMAT>(p) ? 1 : 0), threads = (unsigned)plan.threads;
    switch (16 * plan.threads + plan.vectors) {
#define LLMINT8_NORM(V, T) case 16 * T + V: rmsnorm_kernel<DT, V, FORMAT, T><<<grid, threads, 0, stream>>>(p); break
        LLMINT8_NORM(1, 64);
        LLMINT8_NORM(1, 128);
        LLMINT8_NORM(1, 256);
        LLMINT8_NORM(1, 512);
        LLMINT8_NORM(1, 1024);
        LLMINT8_NORM(2, 64);
        LLMINT8_NORM(2, 128);
        LLMINT8_NORM(2, 256);
        LLMINT8_NORM(2, 512);
        LLMINT8_NORM(2, 1024);
        LLMINT8_NORM(4, 512);
        LLMINT8_NORM(4, 1024);
#undef LLMINT8_NORM
        case 16 * 1024: rmsnorm_long_kernel<DT, FORMAT><<<grid, threads, 0, stream>>>(p); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t norm_launch(const NormArgs& p, const NormPlan& plan, hipStream_t stream) {
    if (p.format == LLMINT8_CODES_NONE) return norm_launch<DT, LLMINT8_CODES_NONE>(p, plan, stream);
    if (p.format == LLMINT8_CODES_FP8_BLOCK) return norm_launch<DT, LLMINT8_CODES_FP8_BLOCK>(p, plan, stream);
    return norm_launch<DT, LLMINT8_CODES_MXFP4>(p, plan, stream);
}

template <int DT, bool DW>
void backward_launch(const NormBackwardArgs& p, const NormBackwardPlan& plan, hipStream_t stream) {
    const unsigned grid = (unsigned)plan.groups, threads = (unsigned)plan.threads;
#define LLMINT8_BACKWARD(V, T, AHEAD) \
    if (plan.vectors == V && plan.row_threads == T && plan.ahead == AHEAD) rmsnorm_backward_kernel<DT, V, T, DW, AHEAD><<<grid, threads, 0, stream>>>(p)
    LLMINT8_BACKWARD(1, 64, false);
    LLMINT8_BACKWARD(1, 128, false);
    LLMINT8_BACKWARD(1, 256, false);
    LLMINT8_BACKWARD(1, 512, false);
    LLMINT8_BACKWARD(1, 1024, false);
    LLMINT8_BACKWARD(2, 1024, false);
    LLMINT8_BACKWARD(1, 64, true);
    LLMINT8_BACKWARD(2, 64, true);
    LLMINT8_BACKWARD(4, 64, true);
    LLMINT8_BACKWARD(4, 128, true);
    LLMINT8_BACKWARD(4, 256, true);
#undef LLMINT8_BACKWARD
}

template <int DT>
hipError_t backward_launch(const NormBackwardArgs& p, const NormBackwardPlan& plan, hipStream_t stream) {
    if (!plan.whole) {
        rmsnorm_backward_long_kernel<DT><<<(unsigned)(p.M < kMaxGrid ? p.M : kMaxGrid), 1024, 0, stream>>>(p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !p.dW) return e;
        rmsnorm_dw_long_kernel<DT><<<dim3((unsigned)ceil_div(p.K, 2048), (unsigned)plan.groups), 256, 0, stream>>>(p);
    } else if (p.dW) {
        backward_launch<DT, true>(p, plan, stream);
    } else {
        backward_launch<DT, false>(p, plan, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.dW) return e;
    rmsnorm_dw_join_kernel<DT><<<(unsigned)ceil_div(p.K, 32), 256, 0, stream>>>(p.partial, (int)plan.groups, p.K, p.dW);
    return hipGetLastError();
}

}  // namespace

// Pieces of 8 columns a thread: one while rows are few, since a row then takes its own latency (16 x
// 8192 with codes 4.6 us with one, 4.8 with two, 5.5 with four); two or four once rows fill the card
// several times over, so that a unit holds several workgroups (4096 x 8192, residual, to e2m1 53.1, 43.9
// and 42.0 us, to e4m3 52.1, 45.8 and 45.4, to 16 bits 47.3, 50.2 and 51.5; 16384 x 1024 to e2m1 13.1, 11.0
// and 14.8; 16384 x 256, residual, to e4m3 9.2, 11.1 and 17.6; 4096 x 16384 two 54.8, four 51.8).  From one to two
// pieces, all with a residual, around the border of 2048 rows: 2047 x 4096 to e4m3 12.3 and 11.4, 2047 x 8192 to e2m1
// 27.8 and 23.6, to 16 bits 24.5 and 25.6, 2047 x 1024 to e4m3 5.3 and 5.4; below it two are as good or better on wide
// rows with codes (1024 x 8192 14.3 and 12.1, 512 x 8192 8.9 and 8.2, 256 x 4096 3.9 and 4.2): not used.
NormPlan rmsnorm_plan(int64_t M, int64_t K, int format) {
    // the columns that a row's codes cover: the codes' padding is written by the threads past K
    const int64_t pieces = ceil_div(format == LLMINT8_CODES_NONE ? K : round_up(K, format == LLMINT8_CODES_MXFP4 ? 256 : 128), 8);
    if (pieces > 4096) return {0, 1024};
    const bool many = M >= 2048;
    const int V = pieces > (many ? 1024 : 2048) ? 4 : (pieces > (many ? 64 : 1024) ? 2 : 1);
    int T = 64;
    while (T * V < pieces) T *= 2;
    return {V, T};
}

hipError_t launch_rmsnorm(int dt, const NormArgs& p, const NormPlan& plan, hipStream_t stream) {
    if (p.M == 0 || p.K == 0) return hipSuccess;
    return dt == F16 ? norm_launch<F16>(p, plan, stream) : norm_launch<BF16>(p, plan, stream);
}

NormBackwardPlan rmsnorm_backward_plan(int64_t M, int64_t K) {
    if (K > 16384) return {false, 0, 0, false, 0, M < 64 ? M : 64};
    int columns = 512;
    while (columns < K) columns *= 2;
    // Few rows: a row over as many threads as it has pieces of 8 columns, and a workgroup a row, since
    // a row takes its own latency (333 x 1040 4.1 us, else 5.6; 100 x 4096 4.6 and 5.2).  So, too, rows that
    // with the next row ahead would not fit the registers (4096 x 16384 85 us, else 105).  There a row's partial sums
    // outweigh its data up to 511 rows: 511 x 16384 with dh 29.2 us and 22.4 with two rows a workgroup, 300 x 16384 20.2
    // and 17.6, 512 x 16384 (two) 22.2.
    if (columns > 8192 || M <= 512) {
        const int V = columns > 8192 ? 2 : 1, T = columns / 8 / V;
        return {true, V, T, false, T, M < 512 ? M : (columns > 8192 ? 256 : 512)};
    }
    // Many rows: 512 threads a compute unit, a wave or several a row, the next row's loads under way
    // (16384 x 1024 20.8 us, 43.7 with a workgroup of 128 threads a row and none ahead).  The border, both launches,
    // a workgroup a row and rows side by side: 256 x 8192 with dh 13.4 and 14.0 us, 512 x 4096 13.1 and 12.0, 512 x 8192
    // 17.6 and 17.9, 512 x 1040 8.0 and 8.3, 600 x 8192 20.0 and 18.3, 1024 x 8192 30.6 and 21.0.
    const int V = columns <= 2048 ? columns / 512 : 4, T = columns / 8 / V;
    int64_t sides = 512 / T;
    while (sides > 1 && M < 256 * sides) sides /= 2;
    const int64_t groups = ceil_div(M, sides);
    return {true, V, T, true, (int)(T * sides), groups < 256 ? groups : 256};
}

hipError_t launch_rmsnorm_backward(int dt, const NormBackwardArgs& p, const NormBackwardPlan& plan, hipStream_t stream) {
    if (p.M == 0 || p.K == 0) return hipSuccess;
    return dt == F16 ? backward_launch<F16>(p, plan, stream) : backward_launch<BF16>(p, plan, stream);
}

}  // namespace llmint8
