// Products of e4m3 codes with power-of-two block scales:
//   Y[m,n] = RN_T( sum_g 2^(ea[m,g] + eb[n,g]) sum_{k in g} a[m,k] b[n,k] ),
// g over groups of 128 along K; ea per row, eb per row or per 128 rows.
// The forward product, the input gradient (b: the transposed weight codes) and the weight
// gradient (both operands per row, the sum over the tokens) are all this product.
//
// The scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 takes one group at a time and
// applies both scales itself, so the sums stay in the accumulators: no fold of partial sums.
// n is its row side and m its column side: a lane's four results are neighbours along n.
// The accumulators are fp32; within the instruction each run of 8 products is added at 13 bits below the
// largest of them before it meets the fp32 sum (measured), so a sum is off by less than 2^-10 of the sum of
// magnitudes, 2e-5 to 6e-5 of the norm in practice, where rounding to 16 bits costs 2e-4 (fp16) or more.
// That is what the instruction offers at its rate: the 16-bit one, whose sums are exact to fp32, has half.
//
// Tiled kernel: BM x BN outputs per workgroup, waves in WM x WN, each 64 rows m (MF = 4 pieces
// of 16) by 16 NF columns n.  A stage is one group: a 128-byte line per row of each operand,
// loaded straight into LDS (16-byte chunk c of row r at chunk c ^ swz(r), so that 8 lanes
// reading one chunk of 8 rows meet all banks), B two stages ahead (3 slots), A as soon as the
// stage two before is read (2 slots).
// Within a stage the n pieces stream from LDS two ahead of their MFMAs, the m pieces of the
// stage stay in registers.  The workgroup meets once per stage, after the stage's last LDS read
// and before the MFMAs of its last two n pieces; under those the next stage's m pieces and first
// n pieces are read.  The barrier waits for all but the newest B loads (counted), so the loads
// in flight are never drained.
// The scales of a row-scaled operand come as one dword per four pieces of 16 rows (the layout is
// the instruction's choice of a byte), one load per stage, a stage ahead; a block-scaled B's is
// one byte for all of a wave's columns.
// Persistent over the XCD's run of tiles, as the int8 product kernels: the next tile's first
// loads are in flight during a tile's last stages and its output.
// 4096 x 12288 x 36864: 1255 us, 2.95 PFLOP/s (the matrix units busy 75 % of the cycles at the 1.66 GHz
// that the power leaves; a register-only loop of the instruction on random operands reaches 4.3);
// 2048 x 4096 x 16384: 103 us, 2.67 PFLOP/s.  Weight gradient of that size: 118 us, 2.33 PFLOP/s: tiles of 16
// stages, whose output (4 us, as all units write at once) the next tile does not hide.
#include "launch.hpp"
#include "tile_gemm.hpp"

namespace llmint8 {

namespace {

template <int DT, int WM, int WN, int NF, bool ROWB, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tiled_kernel(TiledParams tp) {
    tiled_product<DT, WM, WN, NF, ROWB ? kRows : kBlocks, SPLIT>(tp);
}
template <int DT, bool ROWB>
__global__ __launch_bounds__(256, 1) void fp8_single_kernel(TiledParams tp) {
    single_product<DT, ROWB ? kRows : kBlocks>(tp);
}

// the stages of one of `split` parts: whole rounds of scales
int single_part(int64_t groups, int64_t split) { return (int)(split > 1 ? round_up(ceil_div(groups, split), 4) : groups); }

template <int DT, int WM, int WN, int NF, bool ROWB>
hipError_t tiled_launch(const Fp8GemmArgs& a, int split, hipStream_t stream) {
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    const int nk = (int)(a.pitch / BK);
    TiledParams p{a, (int)ceil_div(a.M, BM), (int)ceil_div(a.N, BN), split, (int)ceil_div(nk, split)};
    const int64_t T = (int64_t)p.tiles_m * p.tiles_n;
    if constexpr (NF == 8) {  // (tiles of 128 in parts run in fp8_single_kernel)
        if (split > 1) {
            fp8_tiled_kernel<DT, WM, WN, NF, ROWB, true><<<(unsigned)(T * split), 64 * WM * WN, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    const int64_t G = (int64_t)(cus > 0 ? cus : 1) * (8 / (WM * WN));
    fp8_tiled_kernel<DT, WM, WN, NF, ROWB, false><<<(unsigned)(T < G ? T : G), 64 * WM * WN, 0, stream>>>(p);
    return hipGetLastError();
}

template <int WM, int WN, int NF>
hipError_t tiled(int dt, const Fp8GemmArgs& a, int split, hipStream_t stream) {
    if (a.spitch == 0)
        return dt == F16 ? tiled_launch<F16, WM, WN, NF, true>(a, split, stream) : tiled_launch<BF16, WM, WN, NF, true>(a, split, stream);
    return dt == F16 ? tiled_launch<F16, WM, WN, NF, false>(a, split, stream) : tiled_launch<BF16, WM, WN, NF, false>(a, split, stream);
}

template <int DT>
hipError_t single(const Fp8GemmArgs& a, int split, hipStream_t stream) {
    const TiledParams p{a, (int)ceil_div(a.M, 128), (int)ceil_div(a.N, 128), split, single_part(a.pitch / BK, split)};
    const unsigned grid = (unsigned)((int64_t)p.tiles_m * p.tiles_n * split);
    if (a.spitch == 0) fp8_single_kernel<DT, true><<<grid, 256, 0, stream>>>(p);
    else fp8_single_kernel<DT, false><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

// ---- few rows (M <= 64): the product is bound by B's bytes, each read once straight into
// registers.  A workgroup takes 16 NF columns n; its WV waves split the groups (wave w: w, w + WV,
// ...), U of them in flight while U are multiplied, and their fp32 sums meet in LDS in the order of
// the waves.  With FUSED (one piece of 16 rows), A is the 16-bit X itself: a lane codes its 32
// values of the group (the row's largest magnitude over four lanes), which costs less than the
// launch and the round trip of a separate coding pass while there are few rows.
// With few columns the groups are split over `split` workgroups too (grid.y, `part` groups each):
// their sums go through memory and the last one adds them up in their order.
// 16 x 8192 x 8192: 14.8 us, 4.5 TB/s; 1 x 4096 x 4096 (FUSED) 5.7 us, 2.9 TB/s, of which about 3 us are
// the launch and the first load's way.
template <int DT, int MG, int NF, int WV, bool FUSED, int U, int OCC>
__global__ __launch_bounds__(64 * WV, OCC) void fp8_small_kernel(Fp8GemmArgs p, int split, int part) {
    static_assert(!FUSED || MG == 1, "one piece of rows");
    constexpr int NA = FUSED ? 4 : 2 * MG;  // 16-byte pieces of A per lane and group
    __shared__ v4f red[WV][NF * MG][64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NF);
    const int all = (int)(p.pitch / BK), g0 = blockIdx.y * part, nk = all - g0 < part ? all : g0 + part;
    const int64_t K = p.K;
    const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.B + n0 * p.pitch, (p.N - n0 < 16 * NF ? p.N - n0 : 16 * NF) * p.pitch);
    const __amdgpu_buffer_rsrc_t rsb = buffer_rsrc(p.sb + (n0 >> 7) * p.spitch, p.spitch);  // 16 NF divides 128: one block
    const __amdgpu_buffer_rsrc_t ra = FUSED ? buffer_rsrc(p.X, p.M * K * 2) : buffer_rsrc(p.A, p.M * p.pitch);
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(p.sa, FUSED ? 0 : (int64_t)all * 64);
    uint32_t b_off[NF], a_off[MG];
#pragma unroll
    for (int f = 0; f < NF; ++f) b_off[f] = (uint32_t)((16 * f + li) * p.pitch + 16 * q);
#pragma unroll
    for (int j = 0; j < MG; ++j) a_off[j] = (uint32_t)(FUSED ? (li * K + 16 * q) * 2 : (16 * j + li) * p.pitch + 16 * q);

    // (lane quarter q holds bytes 16 q .. + 15 and 64 + 16 q .. + 15 of a group of either operand, so that
    // a load takes half a line of a row)
    struct Group {
        u32x4 b[NF][2], a[NA];
        int eb, ea, shift;
    };
    // The groups go round from a different one in each workgroup: in rows of a power of two bytes a
    // group's lines are in the same few memory channels (16 x 8192 x 28672: 53 us, 60 from the first;
    // 4 x 16384 x 8192: 25.4 and 31.6).
    const int turn = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 5 % (unsigned)(nk - g0)));
    // the n-th group (past the last: nothing in reach, zeros)
    auto load = [&](int n, Group& r) LLMINT8_FP8_INLINE {
        const bool in = n < nk;
        const int g = n + turn < nk ? n + turn : n + turn - (nk - g0);
        const uint32_t far = in ? 0u : 0x80000000u;  // past every resource
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                r.b[f][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, (b_off[f] + (uint32_t)(g * BK + 64 * h)) | far, 0, 0));
        if constexpr (FUSED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = g * BK + 64 * (i >> 1) + 8 * (i & 1);
                const int64_t k = at + 16 * q;  // past K: the next row's, or nothing
                const uint32_t off = (a_off[0] + (uint32_t)at * 2) | (in && k < K && li < p.M ? 0u : 0x80000000u);
                r.a[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, off, 0, 0));
            }
        } else {
#pragma unroll
            for (int j = 0; j < MG; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    r.a[2 * j + h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, (a_off[j] + (uint32_t)(g * BK + 64 * h)) | far, 0, 0));
            r.ea = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(g * 64 + 4 * li) | far, 0, 0);
        }
        // the dword that holds the byte (of a byte load the compiler widens the value at once, and
        // waits for it there); the byte is shifted down where it is used
        r.eb = (int)__builtin_amdgcn_raw_buffer_load_b32(rsb, (uint32_t)(g & ~3) | far, 0, 0);
        r.shift = 8 * (g & 3);
    };
    v4f acc[NF][MG] = {};
    auto wide = [](const u32x4& lo, const u32x4& hi) LLMINT8_FP8_INLINE {
        return __builtin_bit_cast(v8i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto multiply = [&](const Group& r) LLMINT8_FP8_INLINE {
        v8i a[MG];
        int ea = r.ea, eb = r.eb;
        asm volatile("" : "+v"(eb));
        eb = (int)((uint32_t)eb >> r.shift);
        if constexpr (FUSED) {
            u32x4 v = magnitudes(r.a[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d) v[d] = max_patterns(v[d], r.a[i][d] & 0x7fff7fffu);
            const uint32_t m = max_patterns_rows(max_pattern(v));
            ea = (int)e8m0_of(to_f32<DT>((uint16_t)m));
            const float s = e8m0_value((uint32_t)ea);
            u32x2 c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = e4m3x8<DT>(r.a[i], s);
            a[0] = v8i{(int)c[0][0], (int)c[0][1], (int)c[1][0], (int)c[1][1], (int)c[2][0], (int)c[2][1], (int)c[3][0], (int)c[3][1]};
        } else {
#pragma unroll
            for (int j = 0; j < MG; ++j) a[j] = wide(r.a[2 * j], r.a[2 * j + 1]);
        }
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < MG; ++j) acc[f][j] = mfma_fp8(wide(r.b[f][0], r.b[f][1]), a[j], acc[f][j], eb, 0, ea, FUSED ? 0 : j);
    };
    Group x[U], y[U];
    int g = g0 + w;
#pragma unroll
    for (int u = 0; u < U; ++u) load(g + u * WV, x[u]);
    while (g < nk) {  // the groups are taken U at a time, two sets in turn
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
    auto sum = [&](int t) LLMINT8_FP8_INLINE {
        v4f v[WV];  // all reads first
#pragma unroll
        for (int i = 0; i < WV; ++i) v[i] = red[i][t][lane];
        __builtin_amdgcn_sched_barrier(0);
        v4f s = v[0];
#pragma unroll
        for (int i = 1; i < WV; ++i) s += v[i];
        return s;
    };
    auto store = [&](int t, const v4f& s) LLMINT8_FP8_INLINE {
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
hipError_t small_launch(const Fp8GemmArgs& a, int split, hipStream_t stream) {
    const int part = (int)ceil_div(a.pitch / BK, split);
    const dim3 g((unsigned)ceil_div(a.N, 16 * NF), (unsigned)split);
    fp8_small_kernel<DT, MG, NF, WV, FUSED, U, OCC><<<g, 64 * WV, 0, stream>>>(a, split, part);
    return hipGetLastError();
}

template <int DT>
hipError_t small(const Fp8GemmArgs& a, const Fp8Plan& plan, hipStream_t stream) {
    if (plan.kind == Fp8Plan::kFused) {
        if (plan.columns == 1) return small_launch<DT, 1, 1, 8, true, 1, 4>(a, plan.split, stream);
        // fewer waves once there are many workgroups: 1 x 4096 x 8192 7.6 us with 8, 8.7 with 4, 1 x 4096 x
        // 14336 14.3 and 12.1
        return a.N < 12288 ? small_launch<DT, 1, 2, 8, true, 1, 4>(a, plan.split, stream) : small_launch<DT, 1, 2, 4, true, 1, 4>(a, plan.split, stream);
    }
    switch (4 * plan.pieces + plan.columns) {
        case 4 + 1: return small_launch<DT, 1, 1, 4, false, 2, 4>(a, plan.split, stream);
        case 4 + 2: return small_launch<DT, 1, 2, 4, false, 1, 4>(a, plan.split, stream);
        case 8 + 1: return small_launch<DT, 2, 1, 4, false, 1, 4>(a, plan.split, stream);
        case 8 + 2: return small_launch<DT, 2, 2, 8, false, 1, 2>(a, plan.split, stream);
        case 8 + 4: return small_launch<DT, 2, 4, 4, false, 1, 2>(a, plan.split, stream);
        case 16 + 1: return small_launch<DT, 4, 1, 4, false, 1, 4>(a, plan.split, stream);
        default: return small_launch<DT, 4, 2, 4, false, 1, 2>(a, plan.split, stream);
    }
}

// Parts of the sum of `tiles` (at most 256) tiles of 128 x 128, one workgroup a compute unit.  The
// estimate, in units of 0.1 ns, from measurements over 5 to 256 tiles and 3 to 128 groups: a group
// takes 0.42 us, up to 0.54 us as more workgroups share the memory; joining s parts takes 2 us + 1 us
// a part + 11 ns a part and tile.  65 x 16384 x 4096 (32 tiles): 57.1 us unsplit, 37.3 in 2 parts,
// 27.3 in 4, 27.0 in 8; 200 x 8192 x 8192 (128 tiles): 35.7, 30.9 in 2; 512 x 4096 x 4096 (128
// tiles): 16.7, 19.1 in 2.
int single_parts(int64_t tiles, int64_t groups) {
    auto cost = [&](int64_t i) {
        const int64_t wgs = tiles * i;
        return single_part(groups, i) * (4200 + 1200 * wgs / 256) + (i > 1 ? 20000 + 10000 * i + 110 * wgs : 0);
    };
    int64_t s = 1;
    for (int64_t i = 2; i * tiles <= 256 && i <= groups / 4; ++i)
        if (cost(i) < cost(s)) s = i;
    return (int)ceil_div(groups, single_part(groups, s));
}

}  // namespace

Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t nk, bool x16, bool rowb) {
    Fp8Plan p{Fp8Plan::kTile256, 0, 0, 1, 0, 0};
    int64_t out = 256 * 256;
    // Few rows straight from memory; past 32 rows only while B is small, as there the tiles, whose rows
    // are shared, catch up: 64 x 16384 x 4096 38.1 us, in a tile's kernel 25.9, 48 x 8192 x 8192 24.0 and
    // 22.7; 64 x 4096 x 4096 11.4 and 13.7, 32 x 16384 x 4096 24.3 and 25.7.
    // (From 2^29 columns on their grid, of 8 threads a column, would pass the 2^32 threads of a launch.)
    if (!rowb && N < (int64_t)1 << 29 && (M <= 32 || (M <= 64 && N * nk <= (int64_t)1 << 17))) {
        // A coded in the kernel, or by a launch before it (every workgroup codes the rows that it
        // multiplies): 1 x 4096 x 4096 5.7 and 7.1 us, 4 x 8192 x 8192 14.9 and 16.8, 4 x 8192 x 28672 49.0 and
        // 48.4; not where a long sum wants parts (1 x 16384 x 1024: 13.2 us, in parts 11.6).
        const bool fused = x16 && M <= 4 && N * nk <= (int64_t)1 << 19 && (N >= 2048 || nk < 64);
        p.kind = fused ? Fp8Plan::kFused : Fp8Plan::kSmall;
        p.pieces = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
        // Pieces of 16 columns of a workgroup, while 256 workgroups are left: 16 x 4096 x 4096 6.1 us with one,
        // 7.7 with two, 16 x 8192 x 8192 18.4 and 14.8, 16 x 4096 x 16384 19.7 and 14.9; 32 x 4096 x 8192 14.0,
        // 10.3 and (four) 13.7, 32 x 4096 x 12288 20.1, 18.3 and 15.2; coded in the kernel, 1 x 4096 x 8192 9.3 and
        // 7.6, 1 x 4096 x 4096 5.7 and 7.0.
        p.columns = N < 8192 ? 1 : (p.pieces == 2 && N >= 12288 ? 4 : 2);
        p.tiles = ceil_div(N, 16 * p.columns);
        // Parts of the sum where columns alone leave units idle: 16 x 16384 x 1024 16.5 us, 9.1 in 4 parts;
        // 64 x 4096 x 2048 11.4 and (2) 9.1; 16 x 4096 x 2048 6.0 and 6.0.
        if (!fused && (p.tiles < 128 || (p.tiles == 128 && p.pieces > 1))) p.split = sum_parts(nk, 256 / p.tiles, 8);
        out = 256 * p.columns * p.pieces;
    } else {
        const int64_t t256 = ceil_div(M, 256) * ceil_div(N, 256), t128 = ceil_div(M, 128) * ceil_div(N, 128);
        // Tiles of 128 where all of them fit the card at once (two a compute unit): 2048 x 4096 x 4096
        // 33.8 us, with tiles of 256 42.1; 333 x 4096 x 16384 38.3 and 44.0; past that tiles of 256:
        // 2048 x 2064 x 7424 31.3 us, with tiles of 128 41.2; 1000 x 4096 x 16384 55.2 and 75.7.
        // Between half and all of that with a long sum, tiles of 256 in parts: 2048 x 16384 x 4096 116 us
        // in 2, with tiles of 128 136; 1000 x 8192 x 8192 (64 groups) 72.2 and 70.0.  One tile a unit:
        // the kernel that looks further ahead: 512 x 8192 x 8192 (256 tiles) 41.2 us, else 51.3; 200 x
        // 784 x 632 (10 tiles) 6.7 and 7.5.
        if (t128 <= 512 && !(t128 > 256 && nk >= 96)) {
            p.kind = t128 <= 256 ? Fp8Plan::kSingle : Fp8Plan::kTile128;
            out = 128 * 128;
            p.tiles = t128;
            if (t128 <= 256) p.split = single_parts(t128, nk);
        } else {
            p.tiles = t256;
            if (t256 <= 128) p.split = sum_parts(nk, 256 / t256, 32);
        }
    }
    p.partial_bytes = p.split > 1 ? p.tiles * p.split * out * 4 : 0;
    return p;
}

hipError_t launch_fp8_gemm(int dt, const Fp8GemmArgs& a, const Fp8Plan& plan, hipStream_t stream) {
    if (a.M == 0 || a.N == 0) return hipSuccess;
    if (plan.kind == Fp8Plan::kTile256) return tiled<4, 2, 8>(dt, a, plan.split, stream);
    if (plan.kind == Fp8Plan::kTile128) return tiled<2, 2, 4>(dt, a, plan.split, stream);
    if (plan.kind == Fp8Plan::kSingle) return dt == F16 ? single<F16>(a, plan.split, stream) : single<BF16>(a, plan.split, stream);
    return dt == F16 ? small<F16>(a, plan, stream) : small<BF16>(a, plan, stream);
}

}  // namespace llmint8
