// Products of e2m1 codes with power-of-two scales per 32 values (the format: mxfp4_common.hpp):
//   Y[m,n] = RN_T( sum_g 2^(ea[m,g] + eb[n,g]) sum_{k in g} a[m,k] b[n,k] ),
// g over groups of 32 along K, a scale per row and group on both sides.
//
// The scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 takes 128 values, four groups, at a
// time: lane 16 q + i holds the 16 bytes and the scale of row i, group q.  n is its row side and m its
// column side: a lane's four results are neighbours along n.  A group's products are whole multiples
// of a quarter of its scales, at most 36, so their sum is exact; groups meet in fp32.
#include "launch.hpp"
#include "tile_gemm.hpp"

namespace llmint8 {

namespace {

#define LLMINT8_FP4_INLINE __attribute__((always_inline))

template <int DT, int WM, int WN, int NF, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN, 2) void mxfp4_tiled_kernel(TiledParams tp) {
    tiled_product<DT, WM, WN, NF, kFp4, SPLIT>(tp);
}
template <int DT>
__global__ __launch_bounds__(256, 1) void mxfp4_single_kernel(TiledParams tp) {
    single_product<DT, kFp4>(tp);
}

template <int DT, int WM, int WN, int NF>
hipError_t tiled(const Mxfp4GemmArgs& a, int split, hipStream_t stream) {
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    const int nk = (int)(a.pitch >> 7);
    const TiledParams p{a, (int)ceil_div(a.M, BM), (int)ceil_div(a.N, BN), split, (int)ceil_div(nk, split)};
    const int64_t T = (int64_t)p.tiles_m * p.tiles_n;
    if constexpr (NF == 8) {  // (tiles of 128 in parts run in mxfp4_single_kernel)
        if (split > 1) {
            mxfp4_tiled_kernel<DT, WM, WN, NF, true><<<(unsigned)(T * split), 64 * WM * WN, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    const int64_t G = (int64_t)(cus > 0 ? cus : 1) * (8 / (WM * WN));
    mxfp4_tiled_kernel<DT, WM, WN, NF, false><<<(unsigned)(T < G ? T : G), 64 * WM * WN, 0, stream>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t single(const Mxfp4GemmArgs& a, int split, hipStream_t stream) {
    const TiledParams p{a, (int)ceil_div(a.M, 128), (int)ceil_div(a.N, 128), split, (int)ceil_div(a.pitch >> 7, split)};
    mxfp4_single_kernel<DT><<<(unsigned)((int64_t)p.tiles_m * p.tiles_n * split), 256, 0, stream>>>(p);
    return hipGetLastError();
}

// ---- few rows: the product is bound by B's bytes, each read once straight into registers.  A
// workgroup takes 16 NF columns n and all rows m (at most 16 MG); its WV waves split the steps (wave w: w, w + WV,
// ...), U of them in flight while U are multiplied, and their fp32 sums meet in LDS in the order of
// the waves.  With FUSED (one piece of 16 rows), A is the 16-bit X itself: a lane codes its own groups.
// With few columns the steps are split over `split` workgroups too (grid.y, `part` steps each):
// their sums go through memory and the last one adds them up in their order.
template <int DT, int MG, int NF, int WV, bool FUSED, int U, int OCC>
__global__ __launch_bounds__(64 * WV, OCC) void mxfp4_small_kernel(Mxfp4GemmArgs p, int split, int part) {
    static_assert(!FUSED || MG == 1, "one piece of rows");
    constexpr int NA = FUSED ? 8 : 2 * MG;  // 16-byte pieces of A per lane and step
    constexpr int SN = (NF + 1) / 2, SM = FUSED ? 1 : (MG + 1) / 2;  // scale dwords
    __shared__ v4f red[WV][NF * MG][64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NF);
    const int all = (int)(p.pitch >> 7), g0 = blockIdx.y * part, nk = all - g0 < part ? all : g0 + part;
    const int64_t K = p.K, rows_n = p.N - n0 < 16 * NF ? p.N - n0 : 16 * NF;
    const int64_t sp = (int64_t)all * 256;  // bytes of the scales of 32 rows
    const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.B + n0 * p.pitch, rows_n * p.pitch);
    const __amdgpu_buffer_rsrc_t rsb = buffer_rsrc(p.sb + (n0 >> 5) * sp, ceil_div(rows_n, 32) * sp);
    const __amdgpu_buffer_rsrc_t ra = FUSED ? buffer_rsrc(p.X, p.M * K * 2) : buffer_rsrc(p.A, p.M * p.pitch);
    const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(p.sa, FUSED ? 0 : ceil_div(p.M, 32) * sp);
    const int nb = NF == 1 ? (int)(blockIdx.x & 1) : 0;  // the half of a tile of scales
    uint32_t b_off[NF], a_off[MG];
#pragma unroll
    for (int f = 0; f < NF; ++f) b_off[f] = (uint32_t)((16 * f + li) * p.pitch + 16 * q);
#pragma unroll
    for (int j = 0; j < MG; ++j) a_off[j] = (uint32_t)(FUSED ? (li * K + 32 * q) * 2 : (16 * j + li) * p.pitch + 16 * q);

    struct Step {
        u32x4 b[NF][2], a[NA];
        int eb[SN], ea[SM];
    };
    // The steps go round from a different one in each workgroup: in rows of a power of two bytes a
    // step's lines are in the same few memory channels.
    const int turn = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 5 % (unsigned)(nk - g0)));
    // the n-th step (past the last: nothing in reach, zeros)
    auto load = [&](int n, Step& r) LLMINT8_FP4_INLINE {
        const bool in = n < nk;
        const int g = n + turn < nk ? n + turn : n + turn - (nk - g0);
        const uint32_t far = in ? 0u : 0x80000000u;  // past every resource
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                r.b[f][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, (b_off[f] + (uint32_t)(g * 128 + 64 * h)) | far, 0, 0));
#pragma unroll
        for (int f = 0; f < SN; ++f)
            r.eb[f] = (int)__builtin_amdgcn_raw_buffer_load_b32(rsb, (uint32_t)(f * (int)sp + g * 256 + 4 * lane) | far, 0, 0);
        if constexpr (FUSED) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = g * 256 + 128 * (i >> 2) + 8 * (i & 3);
                const int64_t k = at + 32 * q;  // past K: the next row's, or nothing
                const uint32_t off = (a_off[0] + (uint32_t)at * 2) | (in && k < K && li < p.M ? 0u : 0x80000000u);
                r.a[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, off, 0, 0));
            }
        } else {
#pragma unroll
            for (int j = 0; j < MG; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    r.a[2 * j + h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, (a_off[j] + (uint32_t)(g * 128 + 64 * h)) | far, 0, 0));
#pragma unroll
            for (int j = 0; j < SM; ++j)
                r.ea[j] = (int)__builtin_amdgcn_raw_buffer_load_b32(rsa, (uint32_t)(j * (int)sp + g * 256 + 4 * lane) | far, 0, 0);
        }
    };
    v4f acc[NF][MG] = {};
    auto multiply = [&](const Step& r) LLMINT8_FP4_INLINE {
        u32x4 a[MG][2];
        int ea[SM], eb[SN];
#pragma unroll
        for (int f = 0; f < SN; ++f) eb[f] = NF == 1 ? (int)((uint32_t)r.eb[f] >> (8 * nb)) : r.eb[f];
        if constexpr (FUSED) {
            uint32_t e[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 v = magnitudes(r.a[4 * h]);
#pragma unroll
                for (int i = 1; i < 4; ++i)
#pragma unroll
                    for (int d = 0; d < 4; ++d) v[d] = max_patterns(v[d], r.a[4 * h + i][d] & 0x7fff7fffu);
                e[h] = fp4_scale_byte<DT>(max_pattern(v));
                const float s = e8m0_value(e[h]);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[0][h][i] = e2m1x8<DT>(r.a[4 * h + i], s);
            }
            ea[0] = (int)(e[0] | e[1] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < MG; ++j) a[j][0] = r.a[2 * j], a[j][1] = r.a[2 * j + 1];
#pragma unroll
            for (int j = 0; j < SM; ++j) ea[j] = r.ea[j];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MG; ++j)
                    acc[f][j] = mfma_fp4(__builtin_bit_cast(v4i, r.b[f][h]), __builtin_bit_cast(v4i, a[j][h]), acc[f][j], eb[f >> 1], 2 * h + (f & 1), ea[j >> 1], 2 * h + (j & 1));
    };
    Step x[U], y[U];
    int g = g0 + w;
#pragma unroll
    for (int u = 0; u < U; ++u) load(g + u * WV, x[u]);
    while (g < nk) {  // the steps are taken U at a time, two sets in turn
        g += U * WV;
#pragma unroll
        for (int u = 0; u < U; ++u) load(g + u * WV, y[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(x[u]);
        if (g >= nk) break;
        g += U * WV;
#pragma unroll
        for (int u = 0; u < U; ++u) load(g + u * WV, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(y[u]);
    }
    mfma_settle();
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < MG; ++j) red[w][f * MG + j][lane] = acc[f][j];
    __syncthreads();
    auto sum = [&](int t) LLMINT8_FP4_INLINE {
        v4f v[WV];  // all reads first
#pragma unroll
        for (int i = 0; i < WV; ++i) v[i] = red[i][t][lane];
        __builtin_amdgcn_sched_barrier(0);
        v4f s = v[0];
#pragma unroll
        for (int i = 1; i < WV; ++i) s += v[i];
        return s;
    };
    auto store = [&](int t, const v4f& s) LLMINT8_FP4_INLINE {
        const int64_t m = 16 * (t % MG) + li, n = n0 + 16 * (t / MG) + 4 * q;
        if (m < p.M && n < p.N) {  // N is a multiple of 8
            u32x2 v;
            v[0] = (uint32_t)from_f32<DT>(s[0]) | ((uint32_t)from_f32<DT>(s[1]) << 16);
            v[1] = (uint32_t)from_f32<DT>(s[2]) | ((uint32_t)from_f32<DT>(s[3]) << 16);
            *(u32x2*)(p.Y + m * p.N + n) = v;
        }
    };
    constexpr int kTiles = NF * MG;
    if (split == 1) {
        for (int t = w; t < kTiles; t += WV) store(t, sum(t));
        return;
    }
    const __amdgpu_buffer_rsrc_t rp = buffer_rsrc(p.partial + (int64_t)blockIdx.x * split * (kTiles * 256), (int64_t)split * kTiles * 1024);
    for (int t = w; t < kTiles; t += WV) store_part(rp, 16 * lane, (uint32_t)((blockIdx.y * kTiles + t) * 1024), sum(t));
    __shared__ int flag;
    if (!last_part(p.counters + blockIdx.x, split, &flag)) return;
    for (int t = w; t < kTiles; t += WV) {
        v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < split; ++i) s += load_part(rp, 16 * lane, (uint32_t)((i * kTiles + t) * 1024));
        store(t, s);
    }
}

template <int DT, int MG, int NF, int WV, bool FUSED, int U, int OCC>
hipError_t small_launch(const Mxfp4GemmArgs& a, int split, hipStream_t stream) {
    const int part = (int)ceil_div(a.pitch >> 7, split);
    const dim3 g((unsigned)ceil_div(a.N, 16 * NF), (unsigned)split);
    mxfp4_small_kernel<DT, MG, NF, WV, FUSED, U, OCC><<<g, 64 * WV, 0, stream>>>(a, split, part);
    return hipGetLastError();
}

template <int DT>
hipError_t small(const Mxfp4GemmArgs& a, const Mxfp4Plan& plan, hipStream_t stream) {
    if (plan.kind == Mxfp4Plan::kFused)
        return plan.columns == 1 ? small_launch<DT, 1, 1, 8, true, 1, 4>(a, plan.split, stream) : small_launch<DT, 1, 2, 8, true, 1, 4>(a, plan.split, stream);
    switch (4 * plan.pieces + plan.columns) {
        case 4 + 1: return small_launch<DT, 1, 1, 4, false, 2, 4>(a, plan.split, stream);
        case 4 + 2: return small_launch<DT, 1, 2, 4, false, 1, 4>(a, plan.split, stream);
        case 8 + 1: return small_launch<DT, 2, 1, 4, false, 1, 4>(a, plan.split, stream);
        case 8 + 2: return small_launch<DT, 2, 2, 8, false, 1, 2>(a, plan.split, stream);
        case 16 + 1: return small_launch<DT, 4, 1, 4, false, 1, 4>(a, plan.split, stream);
        default: return small_launch<DT, 4, 2, 4, false, 1, 2>(a, plan.split, stream);
    }
}

// Parts of the sum of `tiles` (at most 256) tiles of 128 x 128, one workgroup a compute unit.
int single_parts(int64_t tiles, int64_t lines) {
    auto cost = [&](int64_t i) {
        const int64_t wgs = tiles * i;
        return ceil_div(lines, i) * (4200 + 1200 * wgs / 256) + (i > 1 ? 20000 + 10000 * i + 110 * wgs : 0);
    };
    int64_t s = 1;
    for (int64_t i = 2; i * tiles <= 256 && i <= lines / 4; ++i)
        if (cost(i) < cost(s)) s = i;
    return (int)ceil_div(lines, ceil_div(lines, s));
}

}  // namespace

Mxfp4Plan mxfp4_plan(int64_t M, int64_t N, int64_t nk, bool x16) {
    Mxfp4Plan p{Mxfp4Plan::kTile256, 0, 0, 1, 0, 0};
    int64_t out = 256 * 256;
    if (M <= 32 || (M <= 64 && N * nk <= (int64_t)1 << 17)) {
        const bool fused = x16 && M <= 4 && N * nk <= (int64_t)1 << 19 && (N >= 2048 || nk < 32);
        p.kind = fused ? Mxfp4Plan::kFused : Mxfp4Plan::kSmall;
        p.pieces = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
        p.columns = N < 8192 ? 1 : 2;
        p.tiles = ceil_div(N, 16 * p.columns);
        if (!fused && (p.tiles < 128 || (p.tiles == 128 && p.pieces > 1))) p.split = sum_parts(nk, 256 / p.tiles, 4);
        out = 256 * p.columns * p.pieces;
    } else {
        const int64_t t256 = ceil_div(M, 256) * ceil_div(N, 256), t128 = ceil_div(M, 128) * ceil_div(N, 128);
        if (t128 <= 512 && !(t128 > 256 && nk >= 48)) {
            p.kind = t128 <= 256 ? Mxfp4Plan::kSingle : Mxfp4Plan::kTile128;
            out = 128 * 128;
            p.tiles = t128;
            if (t128 <= 256) p.split = single_parts(t128, nk);
        } else {
            p.tiles = t256;
            if (t256 <= 128) p.split = sum_parts(nk, 256 / t256, 16);
        }
    }
    p.partial_bytes = p.split > 1 ? p.tiles * p.split * out * 4 : 0;
    return p;
}

hipError_t launch_mxfp4_gemm(int dt, const Mxfp4GemmArgs& a, const Mxfp4Plan& plan, hipStream_t stream) {
    if (a.M == 0 || a.N == 0) return hipSuccess;
    if (plan.kind == Mxfp4Plan::kTile256) return dt == F16 ? tiled<F16, 4, 2, 8>(a, plan.split, stream) : tiled<BF16, 4, 2, 8>(a, plan.split, stream);
    if (plan.kind == Mxfp4Plan::kTile128) return dt == F16 ? tiled<F16, 2, 2, 4>(a, plan.split, stream) : tiled<BF16, 2, 2, 4>(a, plan.split, stream);
    if (plan.kind == Mxfp4Plan::kSingle) return dt == F16 ? single<F16>(a, plan.split, stream) : single<BF16>(a, plan.split, stream);
    return dt == F16 ? small<F16>(a, plan, stream) : small<BF16>(a, plan, stream);
}

}  // namespace llmint8
