// The tiled products of codes with power-of-two scales (gfx950), for e4m3 (fp8_gemm.hip) and e2m1
// (mxfp4_gemm.hip) alike: a stage is a line of 128 bytes of every row.
#pragma once

#include <type_traits>

#include "mxfp4_common.hpp"
#include "launch.hpp"

namespace llmint8 {

namespace {

constexpr int MF = 4;
constexpr int BK = 128;
constexpr int kXcds = 8;
constexpr int kGroupM = 8;

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// by value: a choice between the variables themselves would put them into memory
__device__ __forceinline__ __amdgpu_buffer_rsrc_t pick(int d, __amdgpu_buffer_rsrc_t a, __amdgpu_buffer_rsrc_t b,
                                                       __amdgpu_buffer_rsrc_t c) {
    return d == 0 ? a : (d == 1 ? b : c);
}

__device__ __forceinline__ int pick(int d, int a, int b) { return d == 0 ? a : b; }

__host__ __device__ constexpr int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

#define LLMINT8_FP8_INLINE __attribute__((always_inline))
// wait for this wave's LDS reads and all but the N newest loads, then the bare barrier
#define LLMINT8_FP8_WAIT_BARRIER(N)                                        \
    do {                                                                   \
        __builtin_amdgcn_s_waitcnt(0xC07F);                                \
        asm volatile("s_waitcnt vmcnt(" #N ")\n\ts_barrier" ::: "memory"); \
    } while (0)

struct TiledParams {
    Fp8GemmArgs a;
    int tiles_m, tiles_n;
    int split, part;  // parts of the sum and the stages of one (split 1: all of them)
};

// What the codes are and where their scales lie.  kBlocks, kRows: e4m3, lines of 128 values, a scale
// per line of A, and of B's 128 x 128 blocks or of its lines.  kFp4: e2m1, lines of 256 values, eight
// scales a line on both sides (tiles: mxfp4_common.hpp); the matrix instruction takes half a line.
enum Form { kBlocks, kRows, kFp4 };

// the instruction with bytes bn, bm of the scale dwords (constants after unrolling)
__device__ __forceinline__ v4f mfma_fp8(const v8i& n, const v8i& m, const v4f& c, int sn, int bn, int sm, int bm) {
#define LLMINT8_MFMA(BN_, BM_) \
    if (bn == BN_ && bm == BM_) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(n, m, c, 0, 0, BN_, sn, BM_, sm);
#define LLMINT8_MFMA4(BN_) LLMINT8_MFMA(BN_, 0) LLMINT8_MFMA(BN_, 1) LLMINT8_MFMA(BN_, 2) LLMINT8_MFMA(BN_, 3)
    LLMINT8_MFMA4(0) LLMINT8_MFMA4(1) LLMINT8_MFMA4(2) LLMINT8_MFMA4(3)
#undef LLMINT8_MFMA4
#undef LLMINT8_MFMA
    return c;
}
__device__ __forceinline__ v4f mfma_fp4(const v4i& n, const v4i& m, const v4f& c, int sn, int bn, int sm, int bm) {
    const v8i a = __builtin_shufflevector(n, n, 0, 1, 2, 3, -1, -1, -1, -1), b = __builtin_shufflevector(m, m, 0, 1, 2, 3, -1, -1, -1, -1);
#define LLMINT8_MFMA(BN_, BM_) \
    if (bn == BN_ && bm == BM_) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, BN_, sn, BM_, sm);
#define LLMINT8_MFMA4(BN_) LLMINT8_MFMA(BN_, 0) LLMINT8_MFMA(BN_, 1) LLMINT8_MFMA(BN_, 2) LLMINT8_MFMA(BN_, 3)
    LLMINT8_MFMA4(0) LLMINT8_MFMA4(1) LLMINT8_MFMA4(2) LLMINT8_MFMA4(3)
#undef LLMINT8_MFMA4
#undef LLMINT8_MFMA
    return c;
}
// half h (128 values) of a line's 16-byte pieces
__device__ __forceinline__ v4i half_of(const v8i& v, int h) {
    return h ? __builtin_shufflevector(v, v, 4, 5, 6, 7) : __builtin_shufflevector(v, v, 0, 1, 2, 3);
}

// A wave's 64 x 16 NF results from row m0, column n0 on, through its staging area `ys` in LDS, 16
// rows m at a time: row r's 16-byte piece c sits at piece c ^ r (mod the pieces of a row).
template <int DT, int NF>
__device__ __forceinline__ void store_tile(const Fp8GemmArgs& p, const v4f (&acc)[NF][MF], uint8_t* ys, int64_t m0, int64_t n0) {
    int lane = threadIdx.x & 63;  // opaque: nothing derived from it here is held through the stages
    asm volatile("" : "+v"(lane));
    const int li = lane & 15, q = lane >> 4;
    constexpr int kPieces = 2 * NF;
#pragma unroll
    for (int j = 0; j < MF; ++j) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            u32x2 v;
            v[0] = (uint32_t)from_f32<DT>(acc[f][j][0]) | ((uint32_t)from_f32<DT>(acc[f][j][1]) << 16);
            v[1] = (uint32_t)from_f32<DT>(acc[f][j][2]) | ((uint32_t)from_f32<DT>(acc[f][j][3]) << 16);
            const int c = (2 * f + (q >> 1)) ^ (li & (kPieces - 1));
            *(u32x2*)(ys + (li * kPieces + c) * 16 + 8 * (q & 1)) = v;
        }
#pragma unroll
        for (int it = 0; it < 16 * kPieces / 64; ++it) {
            const int row = it * (64 / kPieces) + lane / kPieces, ch = lane % kPieces;
            const u32x4 v = *(const u32x4*)(ys + (row * kPieces + (ch ^ (row & (kPieces - 1)))) * 16);
            const int64_t m = m0 + 16 * j + row, n = n0 + 8 * ch;
            if (m < p.M && n < p.N) *(u32x4*)(p.Y + m * p.N + n) = v;
        }
    }
}

// SPLIT: few tiles; a workgroup takes one part of one tile's stages, dumps its sums, and the last of the tile's parts
// to end adds them up in their order and writes the output.
template <int DT, int WM, int WN, int NF, int FORM, bool SPLIT>
__device__ __forceinline__ void tiled_product(const TiledParams& tp) {
    constexpr bool ROWB = FORM == kRows, FOUR = FORM == kFp4;
    constexpr int kWaves = WM * WN;
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    constexpr int kSlotA = BM * BK, kSlotB = BN * BK;
    constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = BN / 8 / kWaves;
    constexpr int NA = FOUR ? MF / 2 : 1;                      // scale dwords of a wave's rows
    constexpr int NS = FOUR ? NF / 2 : (ROWB ? NF / 4 : 1);  // and of its columns
    static_assert(NF % 4 == 0 && 16 * MF == 64, "a scale dword serves four pieces");
    static_assert(kLoadsA == 4 && kLoadsB == 4, "the barrier's wait leaves the four newest loads (B) in flight");
    static_assert(kWaves * 16 * 32 * NF <= kSlotB, "output staging");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kSlotA + 3 * kSlotB];
    const Fp8GemmArgs& p = tp.a;
    const int tid = threadIdx.x, lane = tid & 63, wu = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wu % WM, wn = wu / WM;
    const int li = lane & 15, q = lane >> 4;

    // ---- this workgroup's tiles: a strided part of its XCD's contiguous run (ids congruent mod
    // 8 share an XCD), in groups of kGroupM row tiles
    const int T1 = tp.tiles_m * tp.tiles_n, T = SPLIT ? T1 * tp.split : T1;  // SPLIT: part after part
    const int bid = blockIdx.x, nwg = gridDim.x;
    const int xcd = bid % kXcds, local = bid / kXcds;
    const int per = T / kXcds, rem = T % kXcds;
    const int x_start = xcd * per + (xcd < rem ? xcd : rem), x_cnt = per + (xcd < rem ? 1 : 0);
    const int on_xcd = (nwg - xcd + kXcds - 1) / kXcds;
    const int my_tiles = local < x_cnt ? (x_cnt - local + on_xcd - 1) / on_xcd : 0;
    if (my_tiles == 0) return;  // the same for every wave
    // SPLIT: one tile (T workgroups), its stages from k0
    // (a quotient comes from the vector unit: read back, or every load that it places would loop over lanes)
    const int part = SPLIT ? __builtin_amdgcn_readfirstlane((x_start + local) / T1) : 0, k0 = SPLIT ? part * tp.part : 0;
    const int all = (int)(p.pitch / BK), nk = SPLIT ? (all - k0 < tp.part ? all - k0 : tp.part) : all;
    auto tile_origin = [&](int i, int64_t& m0, int64_t& n0) LLMINT8_FP8_INLINE {
        const int t = SPLIT ? (x_start + local) - part * T1 : x_start + local + i * on_xcd;
        const int in_group = kGroupM * tp.tiles_n;
        const int first_m = (t / in_group) * kGroupM;
        const int gm = tp.tiles_m - first_m < kGroupM ? tp.tiles_m - first_m : kGroupM;
        m0 = (int64_t)__builtin_amdgcn_readfirstlane(first_m + (t % in_group) % gm) * BM;
        n0 = (int64_t)__builtin_amdgcn_readfirstlane((t % in_group) / gm) * BN;
    };

    // ---- operand loads: rows past M or N lie past the resources and read zero, as do all of
    // those past the last tile (they land in slots that no stage reads)
    auto tile_rsrc = [&](int i, __amdgpu_buffer_rsrc_t& ra, __amdgpu_buffer_rsrc_t& rb) LLMINT8_FP8_INLINE {
        int64_t m0 = 0, n0 = 0, rows_a = 0, rows_b = 0;
        if (i < my_tiles) {
            tile_origin(i, m0, n0);
            rows_a = p.M - m0 < BM ? p.M - m0 : BM;
            rows_b = p.N - n0 < BN ? p.N - n0 : BN;
        }
        ra = buffer_rsrc(p.A + m0 * p.pitch, rows_a * p.pitch);
        rb = buffer_rsrc(p.B + n0 * p.pitch, rows_b * p.pitch);
    };
    __amdgpu_buffer_rsrc_t ra0, rb0, ra1, rb1, ra2, rb2;  // (SPLIT: one tile, the first pair)
    tile_rsrc(0, ra0, rb0);
    if constexpr (!SPLIT) {
        tile_rsrc(1, ra1, rb1);
        tile_rsrc(2, ra2, rb2);
    }
    uint32_t off[4];  // of both operands: row 8 (4 wu + j) + lane / 8, its chunk lane % 8
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * (4 * wu + j) + lane / 8;
        off[j] = (uint32_t)(r * p.pitch + (((lane & 7) ^ swz(r)) << 4));
    }
    auto slot_a = [&](int s) LLMINT8_FP8_INLINE { return smem + s * kSlotA; };
    auto slot_b = [&](int s) LLMINT8_FP8_INLINE { return smem + 2 * kSlotA + s * kSlotB; };
    // `left`: the tiles from the current one on, so that a load d tiles ahead has one if d < left; a
    // load without one lies past its resource (which, empty, takes no scalar offset: the check
    // subtracts that)
    int left = my_tiles;
    auto issue = [&](int d, __amdgpu_buffer_rsrc_t r0, __amdgpu_buffer_rsrc_t r1, __amdgpu_buffer_rsrc_t r2, uint8_t* slot, int k,
                     int j) LLMINT8_FP8_INLINE {
        const __amdgpu_buffer_rsrc_t rs = SPLIT ? r0 : pick(d, r0, r1, r2);
        const uint32_t far = SPLIT && d ? 0x80000000u : 0u;
        const int at = __builtin_amdgcn_readfirstlane(d < left ? (k0 + k) * BK : 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(slot + (4 * wu + j) * 1024), 16, (int)(off[j] | far), at, 0, 0);
    };
    auto issue_a = [&](int d, uint8_t* slot, int k, int j) LLMINT8_FP8_INLINE { issue(d, ra0, ra1, ra2, slot, k, j); };
    auto issue_b = [&](int d, uint8_t* slot, int k, int j) LLMINT8_FP8_INLINE { issue(d, rb0, rb1, rb2, slot, k, j); };

    // ---- the scales of a stage: offsets and bytes of this tile's and the next tile's, held as
    // scalars (past the last tile: none, the loads return zeros)
    const int ta = (int)round_up(p.M, 64), tb = ROWB ? (int)round_up(p.N, 64) : 0;  // bytes of a group's scales
    int a_at0, a_at1, a_n0, a_n1, b_at0, b_at1, b_n0, b_n1;
    auto scale_range = [&](int i, int& a_at, int& a_n, int& b_at, int& b_n) LLMINT8_FP8_INLINE {
        int64_t m0 = 0, n0 = 0, rows_a = 0, rows_b = 0;
        if (i < my_tiles) {
            tile_origin(i, m0, n0);
            rows_a = p.M - m0 < BM ? p.M - m0 : BM;
            rows_b = p.N - n0 < BN ? p.N - n0 : BN;
        }
        a_at = (int)(FOUR ? m0 >> 5 : m0);
        a_n = (int)(FOUR ? ceil_div(rows_a, 32) : round_up(rows_a, 64));
        b_at = FOUR ? (int)(n0 >> 5) : (ROWB ? (int)n0 : (int)(n0 >> 7));
        b_n = FOUR ? (int)ceil_div(rows_b, 32) : (ROWB ? (int)round_up(rows_b, 64) : (int)ceil_div(rows_b, 128));
    };
    scale_range(0, a_at0, a_n0, b_at0, b_n0);
    if constexpr (!SPLIT) scale_range(1, a_at1, a_n1, b_at1, b_n1);
    auto load_scales = [&](int next, int kt, int (&sm)[NA], int (&sn)[NS]) LLMINT8_FP8_INLINE {
        int k = kt, a_at = a_at0, a_n = a_n0, b_at = b_at0, b_n = b_n0;
        if constexpr (SPLIT) {
            k = __builtin_amdgcn_readfirstlane(k0 + (next ? 0 : kt));  // past the part: any scales, unused
        } else {
            a_at = pick(next, a_at0, a_at1);
            a_n = pick(next, a_n0, a_n1);
            b_at = pick(next, b_at0, b_at1);
            b_n = pick(next, b_n0, b_n1);
        }
        if constexpr (FOUR) {
            int l = lane;  // opaque, as below
            asm volatile("" : "+v"(l));
            const int sp = all * 256;  // bytes of the scales of 32 rows
            const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(p.sa + (int64_t)a_at * sp + k * 256, a_n > 0 ? (int64_t)a_n * sp - k * 256 : 0);
            const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.sb + (int64_t)b_at * sp + k * 256, b_n > 0 ? (int64_t)b_n * sp - k * 256 : 0);
#pragma unroll
            for (int j = 0; j < NA; ++j) sm[j] = (int)__builtin_amdgcn_raw_buffer_load_b32(ra, (uint32_t)((NA * wm + j) * sp + 4 * l), 0, 0);
#pragma unroll
            for (int f = 0; f < NS; ++f) sn[f] = (int)__builtin_amdgcn_raw_buffer_load_b32(rb, (uint32_t)((NS * wn + f) * sp + 4 * l), 0, 0);
            return;
        }
        int li = lane & 15;  // opaque: the offsets are computed here, not held in registers
        asm volatile("" : "+v"(li));
        const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(p.sa + (int64_t)k * ta + a_at, a_n);
        sm[0] = (int)__builtin_amdgcn_raw_buffer_load_b32(ra, (uint32_t)(64 * wm + 4 * li), 0, 0);
        if constexpr (ROWB) {
            const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.sb + (int64_t)k * tb + b_at, b_n);
#pragma unroll
            for (int f = 0; f < NS; ++f)
                sn[f] = (int)__builtin_amdgcn_raw_buffer_load_b32(rb, (uint32_t)(16 * NF * wn + 64 * f + 4 * li), 0, 0);
        } else {
            const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.sb + b_at * p.spitch, b_n * p.spitch);
            sn[0] = (int)__builtin_amdgcn_raw_buffer_load_b8(rb, (uint32_t)(((16 * NF * wn) >> 7) * (int)p.spitch + k), 0, 0);
        }
    };

    // ---- operand reads: piece f of a slot holds rows 16 f + li, chunks 2q and 2q + 1 (kFp4: q of each half)
    const int rd = li * BK + (((FOUR ? q : 2 * q) ^ swz(li)) << 4);
    auto read = [&](const uint8_t* slot, int f) LLMINT8_FP8_INLINE {
        const v4i lo = *(const v4i*)(slot + f * 16 * BK + rd), hi = *(const v4i*)(slot + f * 16 * BK + (rd ^ (FOUR ? 64 : 16)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    v4f acc[NF][MF];
    v8i fm[2][MF], fn[2];      // m pieces of the stage and of the next, the next stage's first n pieces
    constexpr int R = 2 * NF, LA = 4;  // kFp4: pieces of half a line along n, read LA ahead
    v4i hm[2][MF], hn[LA];             // and by halves: m pieces of either half, the next n pieces
    int sm[NA], sn[NS], nsm[NA], nsn[NS];  // scales of the stage and of the next

    // Stage kt of a tile, in slots sa, sb; P = kt % 2.
    auto stage = [&](auto ptag, int sa, int sb, int kt) LLMINT8_FP8_INLINE {
        constexpr int P = decltype(ptag)::value;
        // both operands' loads are two stages ahead: stage k2 of the tile d ahead
        const int d = __builtin_amdgcn_readfirstlane(kt + 2 < nk ? 0 : (kt + 2 < 2 * nk ? 1 : 2));
        const int k2 = kt + 2 - d * nk;
        uint8_t* to_b = slot_b(sb == 0 ? 2 : sb - 1);
        const uint8_t* An = slot_a(sa ^ 1) + wm * (16 * MF * BK);
        const uint8_t* Bc = slot_b(sb) + wn * (16 * NF * BK);
        const uint8_t* Bn = slot_b(sb == 2 ? 0 : sb + 1) + wn * (16 * NF * BK);
        v8i w[NF];
        w[0] = fn[0];
        w[1] = fn[1];
        auto mfma_row = [&](int f) LLMINT8_FP8_INLINE {
#pragma unroll
            for (int j = 0; j < MF; ++j) acc[f][j] = mfma_fp8(w[f], fm[P][j], acc[f][j], sn[ROWB ? f / 4 : 0], ROWB ? f % 4 : 0, sm[0], j);
        };
        // the next stage's scales (before B's loads, which the barrier leaves in flight)
        const int next = __builtin_amdgcn_readfirstlane(kt + 1 < nk ? 0 : 1);
        load_scales(next, next ? 0 : kt + 1, nsm, nsn);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int kPhases = NF - 2;
#pragma unroll
        for (int f = 0; f < kPhases; ++f) {
#pragma unroll
            for (int l = 0; l < 4; ++l)
                if (l * kPhases / 4 == f) issue_b(d, to_b, k2, l);
            w[f + 2] = read(Bc, f + 2);
            mfma_row(f);
            __builtin_amdgcn_sched_barrier(0);
        }
        LLMINT8_FP8_WAIT_BARRIER(4);
        fn[0] = read(Bn, 0);
        fm[P ^ 1][0] = read(An, 0);
        fm[P ^ 1][1] = read(An, 1);
#pragma unroll
        for (int l = 0; l < 2; ++l) issue_a(d, slot_a(sa), k2, l);
        mfma_row(NF - 2);
        __builtin_amdgcn_sched_barrier(0);
        fm[P ^ 1][2] = read(An, 2);
        fm[P ^ 1][3] = read(An, 3);
        fn[1] = read(Bn, 1);
#pragma unroll
        for (int l = 2; l < 4; ++l) issue_a(d, slot_a(sa), k2, l);
        mfma_row(NF - 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NA; ++j) sm[j] = nsm[j];
#pragma unroll
        for (int f = 0; f < NS; ++f) sn[f] = nsn[f];
    };

    // The same by halves of a line (kFp4): the instruction takes half a line in half the time, so n pieces
    // are read LA = 4 ahead, and m pieces of one half while the other is multiplied, which takes half
    // the registers.
    auto half = [&](const uint8_t* slot, int f, int h) LLMINT8_FP8_INLINE { return *(const v4i*)(slot + f * 16 * BK + (h ? rd ^ 64 : rd)); };
    auto stage_by_halves = [&](int sa, int sb, int kt) LLMINT8_FP8_INLINE {
        const int d = __builtin_amdgcn_readfirstlane(kt + 2 < nk ? 0 : (kt + 2 < 2 * nk ? 1 : 2));
        const int k2 = kt + 2 - d * nk;
        uint8_t* to_b = slot_b(sb == 0 ? 2 : sb - 1);
        const uint8_t *Ac = slot_a(sa) + wm * (16 * MF * BK), *An = slot_a(sa ^ 1) + wm * (16 * MF * BK);
        const uint8_t *Bc = slot_b(sb) + wn * (16 * NF * BK), *Bn = slot_b(sb == 2 ? 0 : sb + 1) + wn * (16 * NF * BK);
        v4i w[R];
#pragma unroll
        for (int r = 0; r < LA; ++r) w[r] = hn[r];
        const int next = __builtin_amdgcn_readfirstlane(kt + 1 < nk ? 0 : 1);
        load_scales(next, next ? 0 : kt + 1, nsm, nsn);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r < R - LA) {
#pragma unroll
                for (int l = 0; l < 4; ++l)
                    if (l * (R - LA) / 4 == r) issue_b(d, to_b, k2, l);
                w[r + LA] = half(Bc, (r + LA) % NF, (r + LA) / NF);
                if (r < MF) hm[1][r] = half(Ac, r, 1);
            } else {
                if (r == R - LA) LLMINT8_FP8_WAIT_BARRIER(4);
                hn[r - (R - LA)] = half(Bn, r - (R - LA), 0);
                hm[0][r - (R - LA)] = half(An, r - (R - LA), 0);
                issue_a(d, slot_a(sa), k2, r - (R - LA));
            }
            const int f = r % NF, h = r / NF;
#pragma unroll
            for (int j = 0; j < MF; ++j) acc[f][j] = mfma_fp4(w[r], hm[h][j], acc[f][j], sn[f / 2], 2 * h + f % 2, sm[j / 2], 2 * h + j % 2);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < NA; ++j) sm[j] = nsm[j];
#pragma unroll
        for (int f = 0; f < NS; ++f) sn[f] = nsn[f];
    };

    // ---- prologue: stages 0 and 1 of both operands, the first scales
    load_scales(0, 0, sm, sn);
#pragma unroll
    for (int j = 0; j < 4; ++j) issue_a(0, slot_a(0), 0, j);
#pragma unroll
    for (int j = 0; j < 4; ++j) issue_b(0, slot_b(0), 0, j);
    const int d1 = nk > 1 ? 0 : 1, k1 = 1 - d1;
#pragma unroll
    for (int j = 0; j < 4; ++j) issue_b(d1, slot_b(1), k1, j);
#pragma unroll
    for (int j = 0; j < 4; ++j) issue_a(d1, slot_a(1), k1, j);
    LLMINT8_FP8_WAIT_BARRIER(8);
    auto first_reads = [&](int sa, int sb) LLMINT8_FP8_INLINE {
        if constexpr (FOUR) {
            static_assert(LA == MF && LA <= NF, "one n piece and one m piece a step");
#pragma unroll
            for (int j = 0; j < LA; ++j) {
                hn[j] = half(slot_b(sb) + wn * (16 * NF * BK), j, 0);
                hm[0][j] = half(slot_a(sa) + wm * (16 * MF * BK), j, 0);
            }
            return;
        }
        fn[0] = read(slot_b(sb) + wn * (16 * NF * BK), 0);
#pragma unroll
        for (int j = 0; j < MF; ++j) fm[0][j] = read(slot_a(sa) + wm * (16 * MF * BK), j);
        fn[1] = read(slot_b(sb) + wn * (16 * NF * BK), 1);
    };
    first_reads(0, 0);
    int sa = 0, sb = 0;
    auto advance = [&]() LLMINT8_FP8_INLINE {
        sa ^= 1;
        sb = sb == 2 ? 0 : sb + 1;
    };
    for (int ti = 0; ti < my_tiles; ++ti) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < MF; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        int kt = 0;
        if constexpr (FOUR) {
            for (; kt < nk; ++kt) {
                stage_by_halves(sa, sb, kt);
                advance();
            }
        }
        if constexpr (!FOUR) {
            for (; kt + 2 <= nk; kt += 2) {
                stage(std::integral_constant<int, 0>{}, sa, sb, kt);
                advance();
                stage(std::integral_constant<int, 1>{}, sa, sb, kt + 1);
                advance();
            }
            if (kt < nk) {
                stage(std::integral_constant<int, 0>{}, sa, sb, kt);
                advance();
            }
        }
        mfma_settle();
        if constexpr (SPLIT) {
            constexpr int H = ROWB ? 1 : 2;  // as the registers allow
            constexpr uint32_t kStep = 64 * kWaves * 16;  // bytes of one quad of every thread
            const int tile = x_start + local - part * T1;
            auto slot = [&](int i) LLMINT8_FP8_INLINE {
                return buffer_rsrc(p.partial + ((int64_t)tile * tp.split + i) * (BM * BN), (int64_t)BM * BN * 4);
            };
            const __amdgpu_buffer_rsrc_t own = slot(part);
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MF; ++j) store_part(own, 16 * tid, (f * MF + j) * kStep, acc[f][j]);
            if (!last_part(p.counters + tile, tp.split, (int*)slot_b(sb == 0 ? 2 : sb - 1))) break;
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MF; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            for (int i = 0; i < tp.split; ++i) {
                const __amdgpu_buffer_rsrc_t rs = slot(i);
#pragma unroll
                for (int f = 0; f < NF; f += H) {  // several loads under way
                    v4f v[H][MF];
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int j = 0; j < MF; ++j) v[h][j] = load_part(rs, 16 * tid, ((f + h) * MF + j) * kStep);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int j = 0; j < MF; ++j) acc[f + h][j] += v[h][j];
                }
            }
        }
        int64_t m0, n0;
        tile_origin(ti, m0, n0);  // out through the slot of the last stage
        store_tile<DT, NF>(p, acc, slot_b(sb == 0 ? 2 : sb - 1) + wu * (16 * 32 * NF), m0 + 64 * wm, n0 + 16 * NF * wn);
        if (!SPLIT && ti + 1 < my_tiles) {
            --left;
            ra0 = ra1;
            rb0 = rb1;
            ra1 = ra2;
            rb1 = rb2;
            tile_rsrc(ti + 3, ra2, rb2);
            a_at0 = a_at1;
            a_n0 = a_n1;
            b_at0 = b_at1;
            b_n0 = b_n1;
            scale_range(ti + 2, a_at1, a_n1, b_at1, b_n1);
            if (!FOUR && (nk & 1)) {
#pragma unroll
                for (int j = 0; j < MF; ++j) fm[0][j] = fm[1][j];
            }
            // every wave is done with its staging area: the next stage's loads go there
            __builtin_amdgcn_s_waitcnt(0xC07F);
            __builtin_amdgcn_s_barrier();
        }
    }
    // no load into this workgroup's LDS may outlive it
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---- at most one tile (or part of one) a compute unit: there a stage of the kernel above takes what
// a load from memory takes, divided by the two stages that it looks ahead.  Here a workgroup of four
// waves has the unit's LDS to itself and looks four stages ahead (4 slots of A, 5 of B); its tile of
// 128 x 128, its stage and its layout are the same.  Scales must not be waited for out of turn (loads
// return in order), so they come for four stages at a time, a round ahead: lane quarter q loads a
// row operand's dword of the round's stage q, which lane swaps then give to all quarters; a block
// operand's dword holds the four stages' bytes (a part's first stage is a multiple of 4).
// kFp4's scales, four dwords a stage, are loaded after the stage that used the registers, as far ahead
// as the operands.
template <int DT, int FORM>
__device__ __forceinline__ void single_product(const TiledParams& tp) {
    constexpr bool ROWB = FORM == kRows, FOUR = FORM == kFp4;
    constexpr int WM = 2, WN = 2, NF = 4, D = 4;
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    constexpr int kSlotA = BM * BK, kSlotB = BN * BK;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[D * kSlotA + (D + 1) * kSlotB];
    const Fp8GemmArgs& p = tp.a;
    const int tid = threadIdx.x, lane = tid & 63, wu = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wu % WM, wn = wu / WM;
    const int li = lane & 15, q = lane >> 4;

    // ---- this workgroup's tile and part: runs of tiles to an XCD, part after part, as above
    const int T1 = tp.tiles_m * tp.tiles_n, T = T1 * tp.split;
    const int xcd = blockIdx.x % kXcds, per = T / kXcds, rem = T % kXcds;
    const int id = xcd * per + (xcd < rem ? xcd : rem) + blockIdx.x / kXcds;
    const int part = __builtin_amdgcn_readfirstlane(id / T1), tile = id - part * T1;
    const int in_group = kGroupM * tp.tiles_n, first_m = tile / in_group * kGroupM;
    const int gm = tp.tiles_m - first_m < kGroupM ? tp.tiles_m - first_m : kGroupM;
    const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(first_m + tile % in_group % gm) * BM;
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(tile % in_group / gm) * BN;
    const int all = (int)(p.pitch / BK), k0 = part * tp.part, nk = all - k0 < tp.part ? all - k0 : tp.part;
    const int64_t rows_a = p.M - m0 < BM ? p.M - m0 : BM, rows_b = p.N - n0 < BN ? p.N - n0 : BN;

    // ---- operand loads; those past the part lie past the resources
    const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(p.A + m0 * p.pitch, rows_a * p.pitch);
    const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.B + n0 * p.pitch, rows_b * p.pitch);
    uint32_t off[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * (4 * wu + j) + lane / 8;
        off[j] = (uint32_t)(r * p.pitch + (((lane & 7) ^ swz(r)) << 4));
    }
    auto slot_a = [&](int s) LLMINT8_FP8_INLINE { return smem + s * kSlotA; };
    auto slot_b = [&](int s) LLMINT8_FP8_INLINE { return smem + D * kSlotA + s * kSlotB; };
    auto issue = [&](__amdgpu_buffer_rsrc_t rs, uint8_t* slot, int k, int j) LLMINT8_FP8_INLINE {
        const uint32_t far = k < nk ? 0u : 0x80000000u;
        const int at = __builtin_amdgcn_readfirstlane(k < nk ? (k0 + k) * BK : 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(slot + (4 * wu + j) * 1024), 16, (int)(off[j] | far), at, 0, 0);
    };

    // ---- scales of the stages k .. k + 3
    const int64_t ta = round_up(p.M, 64), tb = round_up(p.N, 64);
    struct Scales {
        int a, b;  // as loaded
    };
    auto row_scales = [&](const uint8_t* scales, int64_t t, int64_t r0, int64_t rows, int at, int k) LLMINT8_FP8_INLINE {
        const int g = __builtin_amdgcn_readfirstlane(k0 + k), n = all - g < 4 ? all - g : 4;
        const int64_t bytes = n > 0 ? (n - 1) * t + round_up(rows, 64) : 0;
        const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(scales + g * t + r0, bytes);
        return (int)__builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(q * (int)t + at + 4 * li), 0, 0);
    };
    auto load_scales = [&](int k) LLMINT8_FP8_INLINE {
        Scales r;
        r.a = row_scales(p.sa, ta, m0, rows_a, 64 * wm, k);
        if constexpr (ROWB) {
            r.b = row_scales(p.sb, tb, n0, rows_b, 64 * wn, k);
        } else {
            const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(p.sb + (n0 >> 7) * p.spitch, p.spitch);
            r.b = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(k0 + k), 0, 0);  // past the row: zeros
        }
        return r;
    };
    auto spread = [&](int v, int (&s)[D]) LLMINT8_FP8_INLINE {  // quarter q's to all, for each q
        const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
        s[0] = lo[0];
        s[1] = lo[1];
        s[2] = hi[0];
        s[3] = hi[1];
    };

    const int rd = li * BK + (((FOUR ? q : 2 * q) ^ swz(li)) << 4);
    auto read = [&](const uint8_t* slot, int f) LLMINT8_FP8_INLINE {
        const v4i lo = *(const v4i*)(slot + f * 16 * BK + rd), hi = *(const v4i*)(slot + f * 16 * BK + (rd ^ (FOUR ? 64 : 16)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    v4f acc[NF][MF] = {};
    v8i fm[2][MF], fn[2];
    int sm[D], sn[D];
    int s4m[D][2], s4n[D][2];  // kFp4: of the four stages under way
    Scales ahead;
    auto load_four = [&](int k, int (&m)[2], int (&n)[2]) LLMINT8_FP8_INLINE {
        const int sp = all * 256;  // bytes of the scales of 32 rows
        const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(p.sa + (m0 >> 5) * sp, ceil_div(rows_a, 32) * sp);
        const __amdgpu_buffer_rsrc_t rsb = buffer_rsrc(p.sb + (n0 >> 5) * sp, ceil_div(rows_b, 32) * sp);
        const uint32_t far = k < nk ? 0u : 0x80000000u;  // past the part
        const uint32_t at = (uint32_t)(k < nk ? (k0 + k) * 256 : 0) + 4 * lane;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(rsa, ((uint32_t)((2 * wm + i) * sp) + at) | far, 0, 0);
            n[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(rsb, ((uint32_t)((2 * wn + i) * sp) + at) | far, 0, 0);
        }
    };
    auto take_scales = [&]() LLMINT8_FP8_INLINE {
        spread(ahead.a, sm);
        if constexpr (ROWB) spread(ahead.b, sn);
        else sn[0] = ahead.b;
    };

    // Stage k, B in slot sb; P = k % 4, the slot of A; TAIL: past the last whole round, where no scales
    // are loaded.  The barrier leaves the loads after the next stage's in flight: B's and A's of two
    // stages and B's of a third, and the four stages' scales if they are among them.
    auto stage = [&](auto ptag, auto tail, int sb, int k) LLMINT8_FP8_INLINE {
        constexpr int P = decltype(ptag)::value;
        constexpr bool TAIL = decltype(tail)::value;
        uint8_t* to_b = slot_b(sb == 0 ? D : sb - 1);
        const uint8_t* An = slot_a((P + 1) % D) + wm * (16 * MF * BK);
        const uint8_t* Bc = slot_b(sb) + wn * (16 * NF * BK);
        const uint8_t* Bn = slot_b(sb == D ? 0 : sb + 1) + wn * (16 * NF * BK);
        v8i w[NF];
        w[0] = fn[0];
        w[1] = fn[1];
        auto mfma_row = [&](int f) LLMINT8_FP8_INLINE {
            if constexpr (FOUR) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < MF; ++j)
                        acc[f][j] = mfma_fp4(half_of(w[f], h), half_of(fm[P & 1][j], h), acc[f][j], s4n[P][f / 2], 2 * h + f % 2, s4m[P][j / 2], 2 * h + j % 2);
            } else {
#pragma unroll
                for (int j = 0; j < MF; ++j)
                    acc[f][j] = mfma_fp8(w[f], fm[P & 1][j], acc[f][j], sn[ROWB ? P : 0], ROWB ? f : P, sm[P], j);
            }
        };
        if constexpr (P == 0 && !TAIL && !FOUR) {
            ahead = load_scales(k + D);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int f = 0; f < NF - 2; ++f) {
#pragma unroll
            for (int l = 2 * f; l < 2 * f + 2; ++l) issue(rb, to_b, k + D, l);
            w[f + 2] = read(Bc, f + 2);
            mfma_row(f);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (FOUR) LLMINT8_FP8_WAIT_BARRIER(28);
        else if constexpr (P == 3 || TAIL) LLMINT8_FP8_WAIT_BARRIER(20);
        else LLMINT8_FP8_WAIT_BARRIER(22);
        fn[0] = read(Bn, 0);
        fm[(P & 1) ^ 1][0] = read(An, 0);
        fm[(P & 1) ^ 1][1] = read(An, 1);
#pragma unroll
        for (int l = 0; l < 2; ++l) issue(ra, slot_a(P), k + D, l);
        mfma_row(NF - 2);
        __builtin_amdgcn_sched_barrier(0);
        fm[(P & 1) ^ 1][2] = read(An, 2);
        fm[(P & 1) ^ 1][3] = read(An, 3);
        fn[1] = read(Bn, 1);
#pragma unroll
        for (int l = 2; l < 4; ++l) issue(ra, slot_a(P), k + D, l);
        mfma_row(NF - 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (FOUR) {
            load_four(k + D, s4m[P], s4n[P]);
            __builtin_amdgcn_sched_barrier(0);
        } else if constexpr (P == 3) {
            take_scales();
        }
    };

    // ---- the first four stages; the first one's are there when all but the other three's are
    if constexpr (!FOUR) {
        ahead = load_scales(0);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int k = 0; k < D; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) issue(rb, slot_b(k), k, j);
#pragma unroll
        for (int j = 0; j < 4; ++j) issue(ra, slot_a(k), k, j);
        if constexpr (FOUR) load_four(k, s4m[k], s4n[k]);
        __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (FOUR) {
        LLMINT8_FP8_WAIT_BARRIER(36);
    } else {
        LLMINT8_FP8_WAIT_BARRIER(24);
        take_scales();
    }
    fn[0] = read(slot_b(0) + wn * (16 * NF * BK), 0);
#pragma unroll
    for (int j = 0; j < MF; ++j) fm[0][j] = read(slot_a(0) + wm * (16 * MF * BK), j);
    fn[1] = read(slot_b(0) + wn * (16 * NF * BK), 1);
    int k = 0, sb = 0;
    auto advance = [&]() LLMINT8_FP8_INLINE {
        ++k;
        sb = sb == D ? 0 : sb + 1;
    };
    while (k + D <= nk) {
        stage(std::integral_constant<int, 0>{}, std::false_type{}, sb, k);
        advance();
        stage(std::integral_constant<int, 1>{}, std::false_type{}, sb, k);
        advance();
        stage(std::integral_constant<int, 2>{}, std::false_type{}, sb, k);
        advance();
        stage(std::integral_constant<int, 3>{}, std::false_type{}, sb, k);
        advance();
    }
    const int rest = nk - k;
    if (rest > 0) {
        stage(std::integral_constant<int, 0>{}, std::true_type{}, sb, k);
        advance();
    }
    if (rest > 1) {
        stage(std::integral_constant<int, 1>{}, std::true_type{}, sb, k);
        advance();
    }
    if (rest > 2) {
        stage(std::integral_constant<int, 2>{}, std::true_type{}, sb, k);
        advance();
    }
    mfma_settle();
    uint8_t* last = slot_b(sb == 0 ? D : sb - 1);  // the slot of the last stage, which no load is bound for
    if (tp.split > 1) {
        constexpr uint32_t kStep = 256 * 16;  // bytes of one quad of every thread
        auto slot = [&](int i) LLMINT8_FP8_INLINE {
            return buffer_rsrc(p.partial + ((int64_t)tile * tp.split + i) * (BM * BN), (int64_t)BM * BN * 4);
        };
        const __amdgpu_buffer_rsrc_t own = slot(part);
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < MF; ++j) store_part(own, 16 * tid, (f * MF + j) * kStep, acc[f][j]);
        if (!last_part(p.counters + tile, tp.split, (int*)last)) return;  // (which waited for all loads)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < MF; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < tp.split; ++i) {
            const __amdgpu_buffer_rsrc_t rs = slot(i);
            v4f v[NF][MF];
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MF; ++j) v[f][j] = load_part(rs, 16 * tid, (f * MF + j) * kStep);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MF; ++j) acc[f][j] += v[f][j];
        }
    }
    store_tile<DT, NF>(p, acc, last + wu * (16 * 32 * NF), m0 + 64 * wm, n0 + 16 * NF * wn);
    // no load into this workgroup's LDS may outlive it
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace

}  // namespace llmint8
