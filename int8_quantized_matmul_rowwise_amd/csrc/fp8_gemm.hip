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
#include <type_traits>

#include "fp8_common.hpp"
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

// ROWB: B has a scale per row (else per 128 rows, one for a wave's columns).  SPLIT: few tiles; a
// workgroup takes one part of one tile's stages, dumps its sums, and the last of the tile's parts
// to end adds them up in their order and writes the output.
template <int DT, int WM, int WN, int NF, bool ROWB, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tiled_kernel(TiledParams tp) {
    constexpr int kWaves = WM * WN;
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    constexpr int kSlotA = BM * BK, kSlotB = BN * BK;
    constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = BN / 8 / kWaves;
    constexpr int NS = ROWB ? NF / 4 : 1;  // scale dwords of a wave's columns
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
        a_at = (int)m0;
        a_n = (int)round_up(rows_a, 64);
        b_at = ROWB ? (int)n0 : (int)(n0 >> 7);
        b_n = ROWB ? (int)round_up(rows_b, 64) : (int)ceil_div(rows_b, 128);
    };
    scale_range(0, a_at0, a_n0, b_at0, b_n0);
    if constexpr (!SPLIT) scale_range(1, a_at1, a_n1, b_at1, b_n1);
    auto load_scales = [&](int next, int kt, int& sm, int (&sn)[NS]) LLMINT8_FP8_INLINE {
        int k = kt, a_at = a_at0, a_n = a_n0, b_at = b_at0, b_n = b_n0;
        if constexpr (SPLIT) {
            k = __builtin_amdgcn_readfirstlane(k0 + (next ? 0 : kt));  // past the part: any scales, unused
        } else {
            a_at = pick(next, a_at0, a_at1);
            a_n = pick(next, a_n0, a_n1);
            b_at = pick(next, b_at0, b_at1);
            b_n = pick(next, b_n0, b_n1);
        }
        int li = lane & 15;  // opaque: the offsets are computed here, not held in registers
        asm volatile("" : "+v"(li));
        const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(p.sa + (int64_t)k * ta + a_at, a_n);
        sm = (int)__builtin_amdgcn_raw_buffer_load_b32(ra, (uint32_t)(64 * wm + 4 * li), 0, 0);
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

    // ---- operand reads: piece f of a slot holds rows 16 f + li, chunks 2q and 2q + 1
    const int rd = li * BK + (((2 * q) ^ swz(li)) << 4);
    auto read = [&](const uint8_t* slot, int f) LLMINT8_FP8_INLINE {
        const v4i lo = *(const v4i*)(slot + f * 16 * BK + rd), hi = *(const v4i*)(slot + f * 16 * BK + (rd ^ 16));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    v4f acc[NF][MF];
    v8i fm[2][MF], fn[2];      // m pieces of the stage and of the next, the next stage's first n pieces
    int sm, sn[NS], nsm, nsn[NS];  // scales of the stage and of the next

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
            for (int j = 0; j < MF; ++j) acc[f][j] = mfma_fp8(w[f], fm[P][j], acc[f][j], sn[ROWB ? f / 4 : 0], ROWB ? f % 4 : 0, sm, j);
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
        sm = nsm;
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
            if (nk & 1) {
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
template <int DT, bool ROWB>
__global__ __launch_bounds__(256, 1) void fp8_single_kernel(TiledParams tp) {
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

    const int rd = li * BK + (((2 * q) ^ swz(li)) << 4);
    auto read = [&](const uint8_t* slot, int f) LLMINT8_FP8_INLINE {
        const v4i lo = *(const v4i*)(slot + f * 16 * BK + rd), hi = *(const v4i*)(slot + f * 16 * BK + (rd ^ 16));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    v4f acc[NF][MF] = {};
    v8i fm[2][MF], fn[2];
    int sm[D], sn[D];
    Scales ahead;
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
#pragma unroll
            for (int j = 0; j < MF; ++j)
                acc[f][j] = mfma_fp8(w[f], fm[P & 1][j], acc[f][j], sn[ROWB ? P : 0], ROWB ? f : P, sm[P], j);
        };
        if constexpr (P == 0 && !TAIL) {
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
        if constexpr (P == 3 || TAIL) LLMINT8_FP8_WAIT_BARRIER(20);
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
        if constexpr (P == 3) take_scales();
    };

    // ---- the first four stages; the first one's are there when all but the other three's are
    ahead = load_scales(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < D; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) issue(rb, slot_b(k), k, j);
#pragma unroll
        for (int j = 0; j < 4; ++j) issue(ra, slot_a(k), k, j);
        __builtin_amdgcn_sched_barrier(0);
    }
    LLMINT8_FP8_WAIT_BARRIER(24);
    take_scales();
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

// parts of `groups` groups such that none is empty and each has at least `least`
int parts(int64_t groups, int64_t wanted, int64_t least) {
    int64_t s = groups / least < wanted ? groups / least : wanted;
    if (s < 2) return 1;
    const int64_t part = ceil_div(groups, s);
    return (int)ceil_div(groups, part);
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
        if (!fused && (p.tiles < 128 || (p.tiles == 128 && p.pieces > 1))) p.split = parts(nk, 256 / p.tiles, 8);
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
            if (t256 <= 128) p.split = parts(nk, 256 / t256, 32);
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
