// Products of e2m1 codes with power-of-two scales per 32 values (the format: mxfp4_common.hpp):
//   Y[m,n] = RN_T( sum_g 2^(ea[m,g] + eb[n,g]) sum_{k in g} a[m,k] b[n,k] ),
// g over groups of 32 along K, a scale per row and group on both sides.
//
// The scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 takes 128 values, four groups, at a
// time: lane 16 q + i holds the 16 bytes and the scale of row i, group q.  n is its row side and m its
// column side: a lane's four results are neighbours along n.  A group's products are whole multiples
// of a quarter of its scales, at most 36, so their sum is exact; groups meet in fp32.
#include "launch.hpp"
#include "mxfp4_common.hpp"

namespace llmint8 {

namespace {

constexpr int MF = 4;   // pieces of 16 rows m of a wave
constexpr int BK = 128;  // bytes of a line
constexpr int kXcds = 8;
constexpr int kGroupM = 8;

typedef __attribute__((address_space(3))) void* lds_ptr_t;

#define LLMINT8_FP4_INLINE __attribute__((always_inline))
// wait for this wave's LDS reads and all but the N newest loads and stores, then the bare barrier
template <int N>
__device__ __forceinline__ void meet_once_read() {  // all but the N newest LDS reads
    asm volatile("s_waitcnt lgkmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// the instruction with bytes bn, bm of the scale dwords (constants after unrolling)
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

// Where chunk c (16 bytes) of row r's line lies in LDS: at chunk c ^ swz(r), so that the 16 lanes of a
// read meet the 64 banks once each (rows two apart at different chunks, odd rows in the other half).
__host__ __device__ constexpr int swz(int r) { return (r >> 1) & 7; }

struct TiledParams {
    Mxfp4GemmArgs a;
    int tiles_m, tiles_n;
    int split, part;  // parts of the sum and the stages of one (split 1: all of them)
};

// A wave's 64 x 16 NF results from row m0, column n0 on, through its 2 KB of LDS `ys`: 16 rows m x 64
// columns at a time, so that whole lines of 128 bytes leave (64 bytes of a row at a time, straight from
// the registers, took 2048 x 4096 x 16384 from 64 to 94 us).  Row r's 16-byte piece c is at c ^ (r / 2).
// Stores past the matrix lie past the resource.  Their offsets are all in the vector register (why: store_wide;
// opaque as a whole by way of the lane).
template <int DT, int NF>
__device__ __forceinline__ void store_tile(const Mxfp4GemmArgs& p, const v4f (&acc)[NF][MF], uint8_t* ys, int64_t m0, int64_t n0) {
    int lane = threadIdx.x & 63;  // opaque: nothing derived from it here is held through the stages
    asm volatile("" : "+v"(lane));
    const int li = lane & 15, q = lane >> 4, row = lane >> 3, ch = lane & 7;
    const int64_t rows = p.M - m0 < 64 ? p.M - m0 : 64;
    const __amdgpu_buffer_rsrc_t ry = buffer_rsrc(p.Y + (rows > 0 ? m0 * p.N : 0), rows > 0 ? rows * p.N * 2 : 0);
#pragma unroll
    for (int g = 0; g < NF; g += 4) {
        const int64_t n = n0 + 16 * g + 8 * ch;
        const uint32_t at = n < p.N ? (uint32_t)(row * p.N + n) * 2 : 0x80000000u;
#pragma unroll
        for (int j = 0; j < MF; ++j) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const v4f& a = acc[g + f][j];
                u32x2 v;
                v[0] = (uint32_t)from_f32<DT>(a[0]) | ((uint32_t)from_f32<DT>(a[1]) << 16);
                v[1] = (uint32_t)from_f32<DT>(a[2]) | ((uint32_t)from_f32<DT>(a[3]) << 16);
                *(u32x2*)(ys + li * 128 + (((2 * f + (q >> 1)) ^ (li >> 1)) << 4) + 8 * (q & 1)) = v;
            }
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const int r = 8 * it + row;
                const u32x4 v = *(const u32x4*)(ys + r * 128 + ((ch ^ (r >> 1)) << 4));
                __builtin_amdgcn_raw_buffer_store_b128(v, ry, at + (uint32_t)((16 * j + 8 * it) * p.N) * 2, 0, 0);
            }
        }
    }
}

// ---- tiles of BM x BN outputs, waves in WM x WN, each 64 rows m by 16 NF columns n.  A stage is a line
// (256 values) of every row, loaded straight into LDS with its scales (one tile of scales an
// instruction), D - 1 stages ahead: D sets of slots, and a set is loaded anew as soon as every wave has
// read it.  The workgroup meets once a stage, LA steps before its end.  D = 2 where several waves a SIMD
// cover for each other; with at most one tile (or part of one) a compute unit a workgroup of four waves
// has the unit's LDS to itself, and D = 4.
// A step is one n piece against the four m pieces, of half a line (128 values): n pieces are read LA
// steps ahead, m pieces of a half while the other one is multiplied, the scales in the steps after the
// barrier.  (With whole lines a step the m pieces of two stages take 32 registers more and the kernel
// spills: 2048 x 4096 x 16384 184 us.)  The loop is one block: a branch in it costs the registers too.
// Persistent over the XCD's run of tiles: the next tile's first loads are under way during a tile's last
// stage and its output.
// SPLIT: few tiles; a workgroup takes one part of one tile's stages, dumps its sums, and the last of the
// tile's parts (if there are several) to end adds them up in their order and writes the output.
// 4096 x 12288 x 36864: 870 to 890 us, 4.2 PFLOP/s (770 on another card); 8192 x 8192 x 8192 244 us, 4.5; 2048 x
// 4096 x 16384 64 to 74 us, 3.7 to 4.3.  The power sets the clock there (1.3 to 1.9 GHz): with codes that are all zero the first two take
// 593 and 188 us.  A loop of the instruction alone, from registers, reaches 7.1 PFLOP/s on random codes and
// 9.7 on zeros (32 x 32 x 64 6.4 and 9.8).  Of the 593 us, 470 are left without loads and LDS reads.
// Loads of A and of the scales from the middle of a stage on: zeros 666 to 593, random 880 and 887.
template <int DT, int WM, int WN, int NF, bool SPLIT, int D>
__global__ __launch_bounds__(64 * WM * WN, D == 2 ? 2 : 1) void mxfp4_tiled_kernel(TiledParams tp) {
    constexpr int kWaves = WM * WN, R = 2 * NF, LA = 4;
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    constexpr int kSlotA = BM * BK, kSlotB = BN * BK, kSlotS = (BM + BN) / 32 * 256, kSet = kSlotA + kSlotB + kSlotS;
    constexpr int NA = MF / 2, NS = NF / 2;  // scale dwords of a wave's rows and columns
    constexpr int kLoads = 10;
    // Tiles of 256: the m pieces and the scales are all read by step QB, where the workgroup meets once more,
    // and A and the scales are loaded from there on, B after the other barrier.
    constexpr int kEarly = NF == 8 ? 6 : 0, QB = 6;
    static_assert(!kEarly || (MF < QB && QB + 3 <= R - LA), "read before, loaded before the next barrier");
    static_assert(BM / 8 / kWaves == 4 && BN / 8 / kWaves == 4 && (BM + BN) / 32 / kWaves == 2 && BM == BN, "ten loads a wave and stage");
    static_assert(LA == MF && LA <= NF, "one n piece and one m piece a step");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[D * kSet + kWaves * 2048];
    const Mxfp4GemmArgs& p = tp.a;
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
    // (a quotient comes from the vector unit: read back, or every load that it places would loop over lanes)
    const int part = SPLIT ? __builtin_amdgcn_readfirstlane((x_start + local) / T1) : 0, k0 = SPLIT ? part * tp.part : 0;
    const int all = (int)(p.pitch / BK), nk = SPLIT ? (all - k0 < tp.part ? all - k0 : tp.part) : all;
    auto tile_origin = [&](int i, int64_t& m0, int64_t& n0) LLMINT8_FP4_INLINE {
        const int t = SPLIT ? (x_start + local) - part * T1 : x_start + local + i * on_xcd;
        const int in_group = kGroupM * tp.tiles_n;
        const int first_m = (t / in_group) * kGroupM;
        const int gm = tp.tiles_m - first_m < kGroupM ? tp.tiles_m - first_m : kGroupM;
        m0 = (int64_t)__builtin_amdgcn_readfirstlane(first_m + (t % in_group) % gm) * BM;
        n0 = (int64_t)__builtin_amdgcn_readfirstlane((t % in_group) / gm) * BN;
    };

    // ---- loads: a cursor over the stages of the tiles.  Rows past M or N lie past the resources and read
    // zero, and so does everything past the last tile (into slots that no stage reads; an empty resource
    // takes no scalar offset: the check subtracts that).
    const int sp = all * 256;  // bytes of the scales of 32 rows
    __amdgpu_buffer_rsrc_t ra, rb, rs;
    int ahead_tile = 0, ahead_k = 0;
    auto tile_rsrc = [&]() LLMINT8_FP4_INLINE {
        int64_t m0 = 0, n0 = 0, rows_a = 0, rows_b = 0;
        if (ahead_tile < my_tiles) {
            tile_origin(ahead_tile, m0, n0);
            rows_a = p.M - m0 < BM ? p.M - m0 : BM;
            rows_b = p.N - n0 < BN ? p.N - n0 : BN;
        }
        ra = buffer_rsrc(p.A + m0 * p.pitch, rows_a * p.pitch);
        rb = buffer_rsrc(p.B + n0 * p.pitch, rows_b * p.pitch);
        // half of the waves load A's scales, half B's
        rs = wu < kWaves / 2 ? buffer_rsrc(p.sa + (m0 >> 5) * sp, ceil_div(rows_a, 32) * sp) : buffer_rsrc(p.sb + (n0 >> 5) * sp, ceil_div(rows_b, 32) * sp);
    };
    uint32_t off[4];  // of both operands: row 8 (4 wu + j) + lane / 8, its chunk lane % 8
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * (4 * wu + j) + lane / 8;
        off[j] = (uint32_t)(r * p.pitch + (((lane & 7) ^ swz(r)) << 4));
    }
    const uint32_t off_s = (uint32_t)(2 * (wu % (kWaves / 2)) * sp + 4 * lane);
    auto issue = [&](uint8_t* set, int j) LLMINT8_FP4_INLINE {  // load j of the cursor's stage
        const int k = ahead_tile < my_tiles ? k0 + ahead_k : 0;
        if (j < 4) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(set + (4 * wu + j) * 1024), 16, (int)off[j], k * BK, 0, 0);
        else if (j < 8) __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(set + kSlotA + (4 * wu + j - 4) * 1024), 16, (int)off[j - 4], k * BK, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(set + kSlotA + kSlotB + (2 * wu + j - 8) * 256), 4, (int)(off_s + (j - 8) * sp), k * 256, 0, 0);
    };
    auto next_tile = [&]() LLMINT8_FP4_INLINE {  // once the tile's stages are loaded
        if (ahead_k == nk) {
            ahead_k = 0;
            ++ahead_tile;
            tile_rsrc();
        }
    };

    // ---- reads: piece f of a slot holds rows 16 f + li, chunk q of either half
    const int rd = li * BK + ((q ^ swz(li)) << 4);
    auto read_m = [&](const uint8_t* set, int j, int h) LLMINT8_FP4_INLINE { return *(const v4i*)(set + (wm * MF + j) * 16 * BK + (h ? rd ^ 64 : rd)); };
    auto read_n = [&](const uint8_t* set, int f, int h) LLMINT8_FP4_INLINE { return *(const v4i*)(set + kSlotA + (wn * NF + f) * 16 * BK + (h ? rd ^ 64 : rd)); };
    auto read_sm = [&](const uint8_t* set, int j) LLMINT8_FP4_INLINE { return *(const int*)(set + kSlotA + kSlotB + (wm * NA + j) * 256 + 4 * lane); };
    auto read_sn = [&](const uint8_t* set, int f) LLMINT8_FP4_INLINE { return *(const int*)(set + kSlotA + kSlotB + (BM / 32 + wn * NS + f) * 256 + 4 * lane); };

    v4f acc[NF][MF];
    v4i hm[2][MF], hn[LA];             // m pieces of either half; the next LA n pieces
    int sm[NA], sn[NS], nsm[NA], nsn[NS];  // scales of the stage and of the next

    auto stage = [&](int cur) LLMINT8_FP4_INLINE {
        uint8_t *set = smem + cur * kSet, *next = smem + (cur + 1 == D ? 0 : cur + 1) * kSet;
        v4i w[R];
#pragma unroll
        for (int r = 0; r < LA; ++r) w[r] = hn[r];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (kEarly && r >= QB && r < QB + 3) {
                if (r == QB) meet_once_read<QB - MF>();  // but the n pieces of the steps since the last m piece
                constexpr int order[6] = {0, 1, 2, 3, 8, 9};
                issue(set, order[2 * (r - QB)]);
                issue(set, order[2 * (r - QB) + 1]);
            }
            if (r < R - LA) {
                w[r + LA] = read_n(set, (r + LA) % NF, (r + LA) / NF);
                if (r < MF) hm[1][r] = read_m(set, r, 1);
            } else {
                const int i = r - (R - LA);
                if (i == 0) wait_and_meet<(D - 2) * kLoads + kEarly>();
                hn[i] = read_n(next, i, 0);
                hm[0][i] = read_m(next, i, 0);
#pragma unroll
                for (int s = i * (NA + NS) / LA; s < (i + 1) * (NA + NS) / LA; ++s) {
                    if (s < NA) nsm[s] = read_sm(next, s);
                    else nsn[s - NA] = read_sn(next, s - NA);
                }
#pragma unroll
                for (int l = kEarly ? 4 + i : i * kLoads / LA; l < (kEarly ? 5 + i : (i + 1) * kLoads / LA); ++l) issue(set, l);
            }
            const int f = r % NF, h = r / NF;
#pragma unroll
            for (int j = 0; j < MF; ++j) acc[f][j] = mfma_fp4(w[r], hm[h][j], acc[f][j], sn[f / 2], 2 * h + f % 2, sm[j / 2], 2 * h + j % 2);
            __builtin_amdgcn_sched_barrier(0);
        }
        ++ahead_k;
#pragma unroll
        for (int j = 0; j < NA; ++j) sm[j] = nsm[j];
#pragma unroll
        for (int f = 0; f < NS; ++f) sn[f] = nsn[f];
    };

    // ---- the first D stages, the first reads
    tile_rsrc();
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) issue(smem + d * kSet, j);
        ++ahead_k;
        next_tile();
    }
    wait_and_meet<(D - 1) * kLoads>();
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        hn[j] = read_n(smem, j, 0);
        hm[0][j] = read_m(smem, j, 0);
    }
#pragma unroll
    for (int j = 0; j < NA; ++j) sm[j] = read_sm(smem, j);
#pragma unroll
    for (int f = 0; f < NS; ++f) sn[f] = read_sn(smem, f);
    int cur = 0;
    for (int ti = 0; ti < my_tiles; ++ti) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < MF; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int kt = 0; kt < nk;) {  // (the inner loop stays one block: a branch in it costs the registers)
            const int end = nk - kt < nk - ahead_k ? nk : kt + nk - ahead_k;
            for (; kt < end; ++kt) {
                stage(cur);
                cur = cur + 1 == D ? 0 : cur + 1;
            }
            next_tile();
        }
        mfma_settle();
        if (SPLIT && tp.split > 1) {
            constexpr int H = 2;  // as the registers allow
            constexpr uint32_t kStep = 64 * kWaves * 16;  // bytes of one quad of every thread
            const int tile = x_start + local - part * T1;
            auto slot = [&](int i) LLMINT8_FP4_INLINE {
                return buffer_rsrc(p.partial + ((int64_t)tile * tp.split + i) * (BM * BN), (int64_t)BM * BN * 4);
            };
            const __amdgpu_buffer_rsrc_t own = slot(part);
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MF; ++j) store_part(own, 16 * tid, (f * MF + j) * kStep, acc[f][j]);
            if (!last_part(p.counters + tile, tp.split, (int*)(smem + D * kSet))) break;
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int j = 0; j < MF; ++j) acc[f][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            for (int i = 0; i < tp.split; ++i) {
                const __amdgpu_buffer_rsrc_t rp = slot(i);
#pragma unroll
                for (int f = 0; f < NF; f += H) {  // several loads under way
                    v4f v[H][MF];
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int j = 0; j < MF; ++j) v[h][j] = load_part(rp, 16 * tid, ((f + h) * MF + j) * kStep);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int j = 0; j < MF; ++j) acc[f + h][j] += v[h][j];
                }
            }
        }
        int64_t m0, n0;
        tile_origin(ti, m0, n0);
        store_tile<DT, NF>(p, acc, smem + D * kSet + wu * 2048, m0 + 64 * wm, n0 + 16 * NF * wn);
    }
    // no load into this workgroup's LDS may outlive it
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int DT, int WM, int WN, int NF>
hipError_t tiled(const Mxfp4GemmArgs& a, hipStream_t stream) {
    constexpr int BM = 16 * MF * WM, BN = 16 * NF * WN;
    const TiledParams p{a, (int)ceil_div(a.M, BM), (int)ceil_div(a.N, BN), 1, (int)(a.pitch >> 7)};
    const int64_t T = (int64_t)p.tiles_m * p.tiles_n;
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    const int64_t G = (int64_t)(cus > 0 ? cus : 1) * (8 / (WM * WN));
    mxfp4_tiled_kernel<DT, WM, WN, NF, false, 2><<<(unsigned)(T < G ? T : G), 64 * WM * WN, 0, stream>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t single(const Mxfp4GemmArgs& a, int split, hipStream_t stream) {
    const TiledParams p{a, (int)ceil_div(a.M, 128), (int)ceil_div(a.N, 128), split, (int)ceil_div(a.pitch >> 7, split)};
    mxfp4_tiled_kernel<DT, 2, 2, 4, true, 4><<<(unsigned)((int64_t)p.tiles_m * p.tiles_n * split), 256, 0, stream>>>(p);
    return hipGetLastError();
}

// ---- few rows: the product is bound by B's bytes, each read once straight into registers.  A
// workgroup takes 16 NF columns n and all rows m (at most 16 MG); its WV waves split the steps (wave w: w, w + WV,
// ...), U of them in flight while U are multiplied, and their fp32 sums meet in LDS in the order of
// the waves.  With FUSED (one piece of 16 rows), A is the 16-bit X itself: a lane codes its own groups.
// With few columns the steps are split over `split` workgroups too (grid.y, `part` steps each):
// their sums go through memory and the last one adds them up in their order.
// Bound by memory, and at the smallest sizes by a launch and one round of loads: 16 x 8192 x 8192 9.2 us (36
// MB, 3.9 TB/s), 16 x 8192 x 28672 27.3 (4.6), 1 x 4096 x 4096 4.2 and with the coding 5.6 (8.9 MB; the norm
// of a single row, a launch with one round trip to memory, takes 1.8).  Past 16 rows its waves wait for their loads:
// 36 MB take 10.8 us at 24 x 4096 x 16384, 11.0 at 32 x 8192 x 8192, 14.4 at 64 x 8192 x 8192 and 18.9 at 48 x 16384 x 4096,
// where waves, one a SIMD with one step under way, spend 84 % of their cycles waiting; 64 x 4096 x 4096 8.0.
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
    if (plan.kind == Mxfp4Plan::kFused) {
        if (plan.columns == 1) return small_launch<DT, 1, 1, 8, true, 1, 4>(a, plan.split, stream);
        // fewer waves once there are many workgroups: 1 x 8192 x 8192 9.4 us with 8, 10.5 with 4; 1 x 4096 x 14336 9.9
        // and 9.3
        return a.N < 12288 ? small_launch<DT, 1, 2, 8, true, 1, 4>(a, plan.split, stream) : small_launch<DT, 1, 2, 4, true, 1, 4>(a, plan.split, stream);
    }
    switch (4 * plan.pieces + plan.columns) {
        case 4 + 1: return small_launch<DT, 1, 1, 4, false, 2, 4>(a, plan.split, stream);
        case 4 + 2: return small_launch<DT, 1, 2, 8, false, 2, 2>(a, plan.split, stream);
        case 4 + 4: return small_launch<DT, 1, 4, 8, false, 1, 2>(a, plan.split, stream);
        case 8 + 1: return small_launch<DT, 2, 1, 4, false, 1, 4>(a, plan.split, stream);
        case 8 + 2: return small_launch<DT, 2, 2, 8, false, 1, 2>(a, plan.split, stream);
        case 16 + 1: return small_launch<DT, 4, 1, 4, false, 1, 4>(a, plan.split, stream);
        default: return small_launch<DT, 4, 2, 4, false, 1, 2>(a, plan.split, stream);
    }
}

// Parts of the sum of `tiles` (at most 256) tiles of 128 x 128, one workgroup a compute unit.  The
// estimate, in units of 0.1 ns, from measurements over 32 to 256 tiles and 16 to 64 lines: a line takes
// 0.44 us, up to 0.68 us as more workgroups share the memory; joining s parts takes 2 us + 1.6 us a
// part + 20 ns a part and tile.  128 x 16384 x 4096 (32 tiles): 32.5 us unsplit, 28.0 in 2 parts, 20.3 in 4,
// 29.6 in 8; 512 x 16384 x 4096 (128 tiles): 35.7, 34.1 in 2; 512 x 4096 x 4096 (128 tiles): 13.8, 20.4 in 2.
int single_parts(int64_t tiles, int64_t lines) {
    auto cost = [&](int64_t i) {
        const int64_t wgs = tiles * i;
        return ceil_div(lines, i) * (4400 + 2400 * wgs / 256) + (i > 1 ? 20000 + 16000 * i + 200 * wgs : 0);
    };
    int64_t s = 1;
    for (int64_t i = 2; i * tiles <= 256 && i <= lines / 4; ++i)
        if (cost(i) < cost(s)) s = i;
    return (int)ceil_div(lines, ceil_div(lines, s));
}

}  // namespace

Mxfp4Plan mxfp4_plan(int64_t M, int64_t N, int64_t nk, bool x16) {
    Mxfp4Plan p{Mxfp4Plan::kTile256, 0, 0, 1, 0, 0};
    int64_t out = 0;  // of a workgroup whose sum is split
    // Few rows straight from memory; past 32 rows while B is small, as there the tiles, whose rows are shared,
    // catch up: 64 x 8192 x 8192 14.7 us, in a tile's kernel 18.9, 64 x 4096 x 16384 15.5 and 13.0, 48 x 16384 x 4096
    // 19.0 and 19.5, 24 x 4096 x 16384 11.1 and 12.8.
    if (M <= 32 || (M <= 64 && (N * nk <= (int64_t)1 << 17 || (N <= 8192 && N * nk <= (int64_t)1 << 18)))) {
        // A coded in the kernel, or by a launch before it (every workgroup codes the rows that it multiplies;
        // both launches together): 1 x 4096 x 4096 5.6 and 7.0 us, 4 x 8192 x 8192 10.5 and 11.3, 4 x 8192 x 28672
        // 33.0 and 29.2, 8 x 4096 x 4096 6.5 and 7.3, 8 x 4096 x 14336 11.4 and 10.8, 16 x 2048 x 2048 5.0 and 6.4, 16 x
        // 4096 x 4096 8.3 and 7.8; not where a long sum wants parts (4 x 16384 x 1024: 13.3 us, in parts 9.6).
        const bool fused = x16 && M <= 16 && N * nk <= (int64_t)1 << (M <= 4 ? 19 : (M <= 8 ? 18 : 16)) && (N >= 2048 || nk < 32);
        p.kind = fused ? Mxfp4Plan::kFused : Mxfp4Plan::kSmall;
        p.pieces = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
        // Pieces of 16 columns of a workgroup: 16 x 4096 x 4096 4.8 us with one, 5.8 with two, 16 x 8192 x 8192 10.8,
        // 9.0 and (four) 12.4, 16 x 8192 x 28672 33.6, 30.2 and 27.3; coded in the kernel, 1 x 4096 x 4096 5.6 with one,
        // 6.5 with two, 1 x 8192 x 8192 12.2 and 9.4.
        p.columns = N < 8192 ? 1 : (p.pieces == 1 && !fused && N >= 24576 ? 4 : 2);
        p.tiles = ceil_div(N, 16 * p.columns);
        // Parts of the sum where columns alone leave units idle (with the coding): 16 x 16384 x 1024 13.2 us, in 4
        // parts 10.5; 64 x 8192 x 1024 15.4 and 11.5; 16 x 8192 x 1024 9.6 and 9.5.
        if (!fused && (p.tiles < 128 || (p.tiles == 128 && p.pieces > 1))) p.split = sum_parts(nk, 256 / p.tiles, 8);
        out = 256 * p.columns * p.pieces;
    } else if (const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128); t128 <= 512) {
        // Tiles of 128 where all of them fit the card at once (two a compute unit): 2048 x 4096 x 4096 23 us, with
        // tiles of 256 29.7, 2048 x 16384 x 4096 71.4 and 95.6; past that 700 x 4096 x 16384 35.8 and 31.7, 2048 x 8192 x
        // 8192 71.7 and 61.7.  One tile a unit: four sets of slots, and parts of the sum: 512 x 8192 x 8192 (256 tiles)
        // 23.6 us, with two sets 26.5.
        p.kind = t128 <= 256 ? Mxfp4Plan::kSingle : Mxfp4Plan::kTile128;
        p.tiles = t128;
        if (t128 <= 256) p.split = single_parts(t128, nk);
        out = 128 * 128;
    }
    p.partial_bytes = p.split > 1 ? p.tiles * p.split * out * 4 : 0;
    return p;
}

hipError_t launch_mxfp4_gemm(int dt, const Mxfp4GemmArgs& a, const Mxfp4Plan& plan, hipStream_t stream) {
    if (a.M == 0 || a.N == 0) return hipSuccess;
    if (plan.kind == Mxfp4Plan::kTile256) return dt == F16 ? tiled<F16, 4, 2, 8>(a, stream) : tiled<BF16, 4, 2, 8>(a, stream);
    if (plan.kind == Mxfp4Plan::kTile128) return dt == F16 ? tiled<F16, 2, 2, 4>(a, stream) : tiled<BF16, 2, 2, 4>(a, stream);
    if (plan.kind == Mxfp4Plan::kSingle) return dt == F16 ? single<F16>(a, plan.split, stream) : single<BF16>(a, plan.split, stream);
    return dt == F16 ? small<F16>(a, plan, stream) : small<BF16>(a, plan, stream);
}

}  // namespace llmint8
