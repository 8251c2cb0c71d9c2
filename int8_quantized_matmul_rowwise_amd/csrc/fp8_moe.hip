// A mixture-of-experts layer for few tokens, its weights e4m3 codes with a power-of-two scale
// per 128 x 128 block, its activations 16-bit.  Per token x (a row of X) with logits l:
//   experts e_0, e_1, ...: the top_k largest logits (ties to the lowest index; -inf and NaN are
//     never taken, +inf counts as the largest finite number);
//   p_j = exp(l[e_j] - l[e_0]) / Z, Z the sum of exp(l - l[e_0]) over the chosen experts
//     (renormalize) or over all;
//   [g; u] = W13hat_e x (2I values), h = RN_T(silu(g) u), y = RN_T(sum_j p_j W2hat_e h).
//
// Bound by the bytes of the experts met, each read once (once per 16 MG tokens of one expert).  Two
// launches: gate, up and SwiGLU (h goes to the workspace), then down and the weighted sum.  The
// experts are chosen by every workgroup of the first for itself, or, with more tokens or choices than
// kRouteTokens and kRouteChoices, by a launch before it: 4 tokens, top 8: 25.8 us and 3.5 + 25.0; 8
// tokens, top 8: 53.5 and 4.2 + 46.8.
// The products run on 16-bit matrix instructions (16x16x32): a code is exact in either 16-bit
// type, so nothing is lost against the coded weight, and the activations keep their 16 bits --
// few tokens leave the matrix units idle anyway.  Weights are the row side (16 rows), an expert's
// tokens the column side, 16 to a piece; a group of 128 takes four instructions, whose order of
// the terms is free as long as both operands agree.  bf16 takes the scale in the conversion: a
// shift of the exponent, exact wherever the product is a multiple of bf16's smallest step 2^-133 (which
// the instruction keeps).  Every product is at scales from 2^-124 on, as codes are multiples of 2^-9; at
// the three below, a converted weight's are (what it was coded from was such a multiple, and four bits
// of it are), and other codes would be rounded to that step.  fp16 could not hold the scale, so there
// each group's sum is added with it.  Sums are fp32; waves and workgroups split them and meet in a
// fixed order, so a result's bits follow from the inputs alone (where the splits lie depends on the
// sizes and on the experts that the tokens meet together).
//
// Three forms of both launches.  Light: the work is cut finer, so that small layers fill the compute
// units: the 16 rows of an instruction are 8 gate and the same 8 up columns in the first launch, and
// 8 columns of two experts in the second, whose tokens are the two halves of its columns (the
// products of one expert's rows with the other's tokens are not used).  Wide: 16 columns and MG
// pieces of tokens, the waves splitting the groups.  Many: 128 columns, a tile of 16 to a wave, which
// share the tokens' values in LDS.
//
// Read at: 8 tokens, 8 experts of 4096 x 14336, top 2: 165 and 78 us, 5.4 TB/s; 37 tokens, 60 experts of
// 2064 x 1424, top 4: 76 and 53 us, 3.8 TB/s; one token, 64 experts of 2048 x 768, top 8: 10 and 6.8 us
// (2.2 TB/s: the two launches' latencies).
#include <cmath>

#include "fp8_common.hpp"
#include "launch.hpp"

namespace llmint8 {

namespace {

constexpr int kMaxTokens = 128;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kUpWaves = 8, kLightUpWaves = 4;
constexpr int kRouteTokens = 8, kRouteChoices = 32;

#define LLMINT8_MOE_INLINE __attribute__((always_inline))

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off, int at = 0) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, at, 0));
}
constexpr uint32_t kFar = 0x80000000u;  // an offset past every resource: reads zero
typedef __attribute__((address_space(3))) void* lds_ptr_t;
__device__ const u32x4 kZeroLine[8] = {};  // a group's weights where there are none

// A step's instructions bound these kernels before its bytes do, so what a step computes is kept
// short: the group's place rides in the scalar offset, a step without a group has empty resources
// (it reads zeros), and only the last group of a ragged H selects other offsets per lane.

// The scale of group g of a row of scales: the dword that holds its byte, and the number where it
// is used (of a byte load the compiler widens the value at once, and waits for it there).
struct Scale {
    int dword, shift;
};
__device__ __forceinline__ Scale load_scale(const uint8_t* row, int g) {
    return Scale{*(const int*)(row + (g & ~3)), 8 * (g & 3)};
}
__device__ __forceinline__ Scale load_scale(__amdgpu_buffer_rsrc_t rs, uint32_t row, int g) {
    return Scale{(int)__builtin_amdgcn_raw_buffer_load_b32(rs, row, g & ~3, 0), 8 * (g & 3)};
}
__device__ __forceinline__ float scale_here(const Scale& s) {
    int d = s.dword;
    asm volatile("" : "+v"(d));
    return e8m0_value(((uint32_t)d >> s.shift) & 0xffu);
}

__device__ __forceinline__ float usable_logit(float l) {  // NaN as -inf, +inf as the largest number
    return l != l ? -__builtin_inff() : fminf(l, 3.4028234663852886e38f);
}

// Reductions over a wave with lane-to-lane operands (about 8 cycles a step; a shuffle takes about
// 100): the result comes from lane 63.
template <class F>
__device__ __forceinline__ float wave_reduce(float v, float none, F&& f) {
#define LLMINT8_DPP(CTRL, ROWS)                                                                                   \
    v = f(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), \
                                                                   CTRL, ROWS, 0xf, false)))
    LLMINT8_DPP(0x111, 0xf);  // from the lane 1, 2, 4, 8 below in the row of 16
    LLMINT8_DPP(0x112, 0xf);
    LLMINT8_DPP(0x114, 0xf);
    LLMINT8_DPP(0x118, 0xf);
    LLMINT8_DPP(0x142, 0xa);  // row 0's last lane to row 1, row 2's to row 3
    LLMINT8_DPP(0x143, 0xc);  // lane 31 to the upper rows
#undef LLMINT8_DPP
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The experts and (weigh) weights of one token, by one wave; lane j < k returns choice j.  A lane holds C
// neighbouring experts, so that among equal values the lowest lane, and in it the first expert,
// is the lowest index.
template <int C>
__device__ __forceinline__ void route_lanes(const float* __restrict__ l, int E, int k, int renormalize, bool weigh, int& id, float& p) {
    const float kNone = -__builtin_inff();
    const int lane = threadIdx.x & 63;
    float v[C], all[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        v[i] = C * lane + i < E ? usable_logit(l[C * lane + i]) : kNone;
        all[i] = v[i];
    }
    float mine = kNone;  // lane j: choice j's logit
    id = -1;
    for (int j = 0; j < k; ++j) {
        float best = v[0];
#pragma unroll
        for (int i = 1; i < C; ++i) best = v[i] > best ? v[i] : best;
        const float most = wave_reduce(best, kNone, [](float a, float b) { return a > b ? a : b; });
        if (!(most > kNone)) break;  // the same in every lane
        const int from = __builtin_ctzll(__ballot(best == most));
        int at = 0;
        bool taken = false;
#pragma unroll
        for (int i = 0; i < C; ++i) {  // the first of the winning lane's experts with that value
            const bool it = lane == from && !taken && v[i] == most;
            at = it ? i : at;
            v[i] = it ? kNone : v[i];
            taken = taken || it;
        }
        at = C * from + __builtin_amdgcn_readlane(at, from);
        if (lane == j) {
            id = at;
            mine = most;
        }
    }
    if (!weigh) return;
    const float top = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, mine)));
    p = id >= 0 ? expf(mine - top) : 0.0f;
    float own = p;
    if (!renormalize) {
        own = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) own += all[i] > kNone ? expf(all[i] - top) : 0.0f;
    }
    const float z = wave_reduce(own, 0.0f, [](float a, float b) { return a + b; });
    if (id >= 0) p /= z;
}

__device__ __forceinline__ void route_token(const float* __restrict__ l, int E, int k, int renormalize, bool weigh, int& id, float& p) {
    if (E <= 64) route_lanes<1>(l, E, k, renormalize, weigh, id, p);
    else if (E <= 256) route_lanes<4>(l, E, k, renormalize, weigh, id, p);
    else route_lanes<16>(l, E, k, renormalize, weigh, id, p);
}

__global__ __launch_bounds__(64) void moe_route_kernel(Fp8MoeArgs p) {
    const int t = blockIdx.x, lane = threadIdx.x;
    int id;
    float w;
    route_token(p.logits + (int64_t)t * p.E, (int)p.E, p.k, p.renormalize, true, id, w);
    if (lane < p.k) {
        p.ids[t * p.k + lane] = id;
        p.weights[t * p.k + lane] = w;
    }
}

// ---- the table of the second launch: entries of up to `chunk` tokens of one expert, experts
// ascending, an expert's tokens ascending.  table: [0] entries, then per entry expert, first,
// count; pairs: token * k + choice of each place.
__device__ __forceinline__ void build_table(const int32_t* ids, int T, int E, int k, int chunk, int32_t* table,
                                            int32_t* pairs, uint32_t (*mask)[4], int* first) {
    const int tid = threadIdx.x, lane = tid & 63, nt = blockDim.x;
    for (int i = tid; i < 4 * E; i += nt) mask[i >> 2][i & 3] = 0u;
    __syncthreads();
    for (int i = tid; i < T * k; i += nt) {
        const int e = ids[i], t = i / k;
        if (e >= 0) atomicOr(&mask[e][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    if (tid < 64) {  // exclusive sums over the experts of their tokens and entries
        int base = 0, entry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            int c = 0;
            if (e < E)
#pragma unroll
                for (int i = 0; i < 4; ++i) c += __popc(mask[e][i]);
            const int m = (c + chunk - 1) / chunk;
            int cs = c, ms = m;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int a = __shfl_up(cs, off, kWave), b = __shfl_up(ms, off, kWave);
                if (lane >= off) {
                    cs += a;
                    ms += b;
                }
            }
            if (e < E) first[e] = base + cs - c;
            for (int i = 0; i < m; ++i) {
                int32_t* r = table + 1 + 3 * (entry + ms - m + i);
                r[0] = e;
                r[1] = base + cs - c + i * chunk;
                r[2] = c - i * chunk < chunk ? c - i * chunk : chunk;
            }
            base += __shfl(cs, 63, kWave);
            entry += __shfl(ms, 63, kWave);
        }
        if (lane == 0) table[0] = entry;
    }
    __syncthreads();
    for (int i = tid; i < T * k; i += nt) {
        const int e = ids[i], t = i / k;
        if (e < 0) continue;
        int at = first[e];
        for (int j = 0; j < (t >> 5); ++j) at += __popc(mask[e][j]);
        at += __popc(mask[e][t >> 5] & ((1u << (t & 31)) - 1u));
        pairs[at] = i;
    }
}

// ---- the group product.  A weight row's 32 bytes against a token's 32 values: four steps of 8.
// Lane quarter q holds bytes 16 q .. + 15 and 64 + 16 q .. + 15 of the group, so that one load of
// 16 rows takes half a line of each.

template <int DT>
__device__ __forceinline__ u32x4 codes8(uint32_t lo, uint32_t hi, float s) {  // 8 codes as 16-bit values, times s
    u32x4 r;
    if constexpr (DT == F16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, false));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, true));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, false));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, true));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true));
    }
    return r;
}

// Byte offsets of this lane's values of a row of `n` (at `row`, kFar: none) in the first group, in its
// first and second half; past `n` in the last group the next row's are left out.
struct RowAt {
    uint32_t lo, hi, last_lo, last_hi;
    __device__ __forceinline__ void set(uint32_t row, int n, int ng, int q) {
        lo = row + 32 * q;
        hi = lo + 128;
        last_lo = 128 * (ng - 1) + 16 * q < n ? lo : kFar;
        last_hi = 128 * (ng - 1) + 64 + 16 * q < n ? hi : kFar;
    }
};
__device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t rs, const RowAt& a, int g, bool last, u32x4 (&x)[4]) {
    const uint32_t lo = last ? a.last_lo : a.lo, hi = last ? a.last_hi : a.hi;
    x[0] = load16(rs, lo, 256 * g);
    x[1] = load16(rs, lo + 16, 256 * g);
    x[2] = load16(rs, hi, 256 * g);
    x[3] = load16(rs, hi + 16, 256 * g);
}

template <int DT>
__device__ __forceinline__ v4f mfma_16(const u32x4& a, const u32x4& b, const v4f& c) {
    if constexpr (DT == F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// acc[j] += s * (codes of w) x[j].  Pieces without a token are multiplied too (their x is zero):
// skipping them would put a branch between a matrix instruction and the reader of its result,
// where the compiler (ROCm 7.2) leaves out the wait states that the reader needs.
template <int DT, int MG>
__device__ __forceinline__ void group_product(const u32x4 (&w)[2], float s, const u32x4 (&x)[MG][4], v4f (&acc)[MG]) {
    u32x4 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = codes8<DT>(w[i >> 1][2 * (i & 1)], w[i >> 1][2 * (i & 1) + 1], DT == F16 ? 1.0f : s);
#pragma unroll
    for (int j = 0; j < MG; ++j) {
        if constexpr (DT == F16) {
            v4f t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4; ++i) t = mfma_16<DT>(c[i], x[j][i], t);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(t[e], s, acc[j][e]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j] = mfma_16<DT>(c[i], x[j][i], acc[j]);
        }
    }
}

template <int DT>
__device__ __forceinline__ uint16_t swiglu(float gate, float up) {
    return from_f32<DT>(gate / (1.0f + expf(-gate)) * up);
}

// The rows of h are padded with zeros to whole groups: by the workgroup of the last tile.
__device__ __forceinline__ void pad_rows(const Fp8MoeArgs& p, const int* list, int from, int to, int64_t ip) {
    const int pad = (int)(ip - p.I);
    if (pad == 0) return;
    for (int i = threadIdx.x; i < (to - from) * pad; i += blockDim.x) p.h[(int64_t)list[from + i / pad] * ip + p.I + i % pad] = 0;
}

// ---- what a workgroup of the first launch sets up: the choices (ROUTE: it makes them itself,
// workgroup 0 writes them down) and its expert's tokens
template <bool ROUTE>
struct UpSetup {
    int32_t own[ROUTE ? kRouteChoices : 1];
    int list[kMaxTokens];  // the expert's tokens, ascending, as token * top_k + choice
    int part[2], dup;

    template <int WV>
    __device__ __forceinline__ const int32_t* route(const Fp8MoeArgs& p) {
        if (threadIdx.x == 0) dup = 0;
        if constexpr (ROUTE) {
            const int lane = threadIdx.x & 63;
            for (int t = threadIdx.x >> 6; t < p.T; t += WV) {
                int id;
                float wt = 0.0f;
                route_token(p.logits + t * p.E, (int)p.E, p.k, p.renormalize, blockIdx.x == 0, id, wt);
                if (lane < p.k) {
                    own[t * p.k + lane] = id;
                    if (blockIdx.x == 0) {
                        p.ids[t * p.k + lane] = id;
                        p.weights[t * p.k + lane] = wt;
                    }
                }
            }
        }
        __syncthreads();
        return ROUTE ? own : p.ids;
    }
    // This workgroup's expert, of pair y (by_pair; negative: none chosen) or expert y, and its
    // tokens (none if an earlier pair has the same expert, whose workgroups do it).
    __device__ __forceinline__ int expert(const int32_t* ids, int y, int by_pair) {
        return __builtin_amdgcn_readfirstlane(by_pair ? ids[y] : y);  // (from LDS it would count as a lane's value)
    }
    __device__ __forceinline__ int find(const Fp8MoeArgs& p, const int32_t* ids, int y, int by_pair, int e) {
        const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
        int mine = -1;
        if (tid < 128 && tid < p.T)
            for (int j = 0; j < p.k; ++j)
                if (ids[tid * p.k + j] == e) mine = tid * p.k + j;
        if (by_pair && mine >= 0 && mine < y) dup = 1;
        const uint64_t have = __ballot(mine >= 0);
        if (w < 2 && lane == 0) part[w] = __popcll(have);
        __syncthreads();
        const int count = __builtin_amdgcn_readfirstlane(dup ? 0 : part[0] + part[1]);
        if (mine >= 0) list[(w == 1 ? part[0] : 0) + __popcll(have & ((1ull << lane) - 1ull))] = mine;
        __syncthreads();
        return count;
    }
};

// ---- gate, up and SwiGLU: a workgroup takes `span` (at most its waves) tiles of 16 columns of I of
// one expert (16 gate rows and 16 up rows each).  Their groups of H, tile after tile, are split
// evenly over the waves and run through D sets of registers; what a wave has of a tile (it meets at
// most two) goes to LDS, and the waves meet once, after the last.  Workgroup 0 writes the table.
template <int DT, int MG>
__global__ __launch_bounds__(64 * kUpWaves, MG == 1 ? 4 : 2) void moe_up_kernel(Fp8MoeArgs p, int spans, int span, int by_pair, int chunk, int n_zero) {
    constexpr int WV = kUpWaves, D = 2;
    union Shared {
        v4f red[WV][2][2 * MG][64];  // of a wave's first tile and of its second
        struct {
            uint32_t mask[kMaxExperts][4];
            int first[kMaxExperts];
        } t;
    };
    __shared__ Shared sh;
    __shared__ UpSetup<false> setup;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int k = p.k;
    const int32_t* ids = setup.template route<WV>(p);
    if (blockIdx.x == 0) {
        for (int i = tid; i < n_zero; i += blockDim.x) p.counters[i] = 0;
        build_table(ids, (int)p.T, (int)p.E, k, chunk, p.table, p.pairs, sh.t.mask, sh.t.first);
        return;
    }
    const int y = (int)(blockIdx.x - 1) / spans, tile0 = (int)(blockIdx.x - 1) % spans * span;
    const int e = setup.expert(ids, y, by_pair);
    if (e < 0) return;  // the same in every thread, as below
    const int count = setup.find(p, ids, y, by_pair, e);
    if (count == 0) return;
    const int* list = setup.list;

    const int64_t hp = fp8_pitch(p.H), hsp = fp8_scale_pitch_of(p.H);
    const int tiles = (int)(p.I / 16), ng = (int)(hp / 128);
    const int my_tiles = tiles - tile0 < span ? tiles - tile0 : span;
    const int all = my_tiles * ng, from = all * w / WV, to = all * (w + 1) / WV;
    const uint8_t* W = p.W13 + (int64_t)e * 2 * p.I * hp;
    const uint8_t* S = p.s13 + (int64_t)e * ceil_div(2 * p.I, 128) * hsp;
    const int64_t ip = fp8_pitch(p.I);
    const uint32_t w_off = (uint32_t)(li * hp + 16 * q);

    struct Group {
        u32x4 g[2], u[2], x[MG][4];
        Scale eg, eu;
    };
    for (int c0 = 0; c0 < count; c0 += 16 * MG) {
        RowAt x_at[MG];
#pragma unroll
        for (int j = 0; j < MG; ++j) {
            const int i = c0 + 16 * j + li;
            x_at[j].set(i < count ? (uint32_t)((list[i] / k) * p.H) * 2 : kFar, (int)p.H, ng, q);
        }
        int lt = from / ng, lg = from - lt * ng, left = to - from;  // the next load's tile and group
        auto load = [&](Group& r) LLMINT8_MOE_INLINE {
            const bool in = left > 0;  // past the share: zeros
            const int64_t i0 = 16 * (int64_t)(in ? tile0 + lt : tile0);
            const int wg = in ? lg : 0, bytes = in ? 16 * (int)hp : 0;
            const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(W + i0 * hp, bytes), ru = buffer_rsrc(W + (p.I + i0) * hp, bytes);
            const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(p.X, in ? p.T * p.H * 2 : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                r.g[h] = load16(rg, w_off + 64 * h, wg * 128);
                r.u[h] = load16(ru, w_off + 64 * h, wg * 128);
            }
#pragma unroll
            for (int j = 0; j < MG; ++j) load_row(rx, x_at[j], wg, lg == ng - 1, r.x[j]);
            // the scales of the 16 rows (I is a multiple of 16: one block of rows each)
            r.eg = load_scale(S + (i0 >> 7) * hsp, wg);
            r.eu = load_scale(S + ((p.I + i0) >> 7) * hsp, wg);
            --left;
            if (++lg == ng) {
                lg = 0;
                ++lt;
            }
            __builtin_amdgcn_sched_barrier(0);  // the sets are issued, and so waited for, one after the other
        };
        v4f ag[MG] = {}, au[MG] = {};
        int slot = 0, cg = lg;  // of the tile and group being multiplied
        Group r[D];
#pragma unroll
        for (int d = 0; d < D; ++d) load(r[d]);
        // (whole rounds of D steps: a way out between them would make the compiler wait, at the top,
        // for every set instead of the first; steps past the last multiply zeros)
        const int steps = to - from;
        for (int s = 0; s < steps; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                group_product<DT, MG>(r[d].g, scale_here(r[d].eg), r[d].x, ag);
                group_product<DT, MG>(r[d].u, scale_here(r[d].eu), r[d].x, au);
                load(r[d]);
                if (s + d < steps && (++cg == ng || s + d + 1 == steps)) {
                    mfma_settle();
#pragma unroll
                    for (int j = 0; j < MG; ++j) {
                        sh.red[w][slot][j][lane] = ag[j];
                        sh.red[w][slot][MG + j][lane] = au[j];
                        ag[j] = au[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                    slot = 1;
                    cg = 0;
                }
            }
        }
        __syncthreads();
        // an output a thread at a time: its tile's sums in the order of the waves, SwiGLU, h
        const float* red = (const float*)sh.red;
        for (int t = 0; t < my_tiles; ++t) {
            for (int o = tid; o < 256 * MG; o += 64 * WV) {
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int i = 0; i < WV; ++i) {
                    const int a = all * i / WV, b = all * (i + 1) / WV, first = a / ng;
                    if (a < b && first <= t && t <= (b - 1) / ng) {
                        const float* at = red + (2 * i + (t - first)) * (512 * MG) + o;
                        gate += at[0];
                        up += at[256 * MG];
                    }
                }
                const int l = (o >> 2) & 63, i = c0 + 16 * (o >> 8) + (l & 15);
                if (i < count) p.h[(int64_t)list[i] * ip + 16 * (tile0 + t) + 4 * (l >> 4) + (o & 3)] = swiglu<DT>(gate, up);
            }
        }
        if (tile0 + my_tiles == tiles) pad_rows(p, list, c0, count < c0 + 16 * MG ? count : c0 + 16 * MG, ip);
        __syncthreads();
    }
}

// ---- the same in the light form: 8 columns of I a tile, rows 0 .. 7 of the instruction gate and
// 8 .. 15 up.
template <int DT, bool ROUTE>
__global__ __launch_bounds__(64 * kLightUpWaves, 4) void moe_up_light_kernel(Fp8MoeArgs p, int spans, int span, int by_pair, int chunk, int n_zero) {
    constexpr int WV = kLightUpWaves, D = 2;
    union Shared {
        v4f red[WV][64];
        struct {
            uint32_t mask[kMaxExperts][4];
            int first[kMaxExperts];
        } t;
    };
    __shared__ Shared sh;
    __shared__ UpSetup<ROUTE> setup;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int32_t* ids = setup.template route<WV>(p);
    if (blockIdx.x == 0) {
        for (int i = tid; i < n_zero; i += blockDim.x) p.counters[i] = 0;
        build_table(ids, (int)p.T, (int)p.E, p.k, chunk, p.table, p.pairs, sh.t.mask, sh.t.first);
        return;
    }
    const int y = (int)(blockIdx.x - 1) / spans, tile0 = (int)(blockIdx.x - 1) % spans * span;
    const int e = setup.expert(ids, y, by_pair);
    if (e < 0) return;  // the same in every thread, as below

    const int64_t hp = fp8_pitch(p.H), hsp = fp8_scale_pitch_of(p.H);
    const int tiles = (int)(p.I / 8), ng = (int)(hp / 128);
    const int my_tiles = tiles - tile0 < span ? tiles - tile0 : span;
    const int gw = (ng + WV - 1) / WV;  // groups of a wave (its last may lie past H: zeros)
    const int steps = my_tiles * gw;
    // this lane's row of the first tile; its scale is the one of the row that it converts (bf16), or
    // of the row of the results that it adds up (fp16)
    const int64_t row0 = 8 * (int64_t)tile0 + (li & 7) + (li >= 8 ? p.I : 0);
    const uint8_t* W = p.W13 + ((int64_t)e * 2 * p.I + row0) * hp + 16 * q;
    const int64_t s_bytes = ceil_div(2 * p.I, 128) * hsp, ip = fp8_pitch(p.I);
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(p.s13 + (int64_t)e * s_bytes, s_bytes);
    const bool up_scale = DT == F16 ? q >= 2 : li >= 8;
    struct Group {
        u32x4 w[2], x[1][4];
        Scale e;
    };
    RowAt x_at;
    struct At {
        int t, g;  // the next load's tile and group
    };
    At at{0, w};
    auto next = [&]() LLMINT8_MOE_INLINE {
        at.g += WV;
        if (at.g >= gw * WV) {
            at.g = w;
            ++at.t;
        }
        __builtin_amdgcn_sched_barrier(0);  // as above
    };
    // (read back: with the choices in LDS the compiler takes these for lanes' values)
    auto load_w = [&](Group& r) LLMINT8_MOE_INLINE {
        const bool in = at.t < my_tiles && at.g < ng;  // else zeros (no line of weights: NaN times zero is NaN)
        const int t = __builtin_amdgcn_readfirstlane(in ? at.t : 0), g = __builtin_amdgcn_readfirstlane(in ? at.g : 0);
        const uint8_t* from = in ? W + 8 * t * hp + g * 128 : (const uint8_t*)kZeroLine;
        r.w[0] = *(const u32x4*)from;
        r.w[1] = *(const u32x4*)(from + 64);
        // (I is a multiple of 16: a tile's gate rows, and its up rows, lie in one block)
        const int64_t i0 = 8 * (int64_t)(tile0 + t);
        r.e = load_scale(rs, up_scale ? (uint32_t)(((p.I + i0) >> 7) * hsp) : (uint32_t)((i0 >> 7) * hsp), g);
    };
    auto load_x = [&](Group& r) LLMINT8_MOE_INLINE {
        const bool in = at.t < my_tiles && at.g < ng;
        const int g = __builtin_amdgcn_readfirstlane(in ? at.g : 0);
        const int bytes = __builtin_amdgcn_readfirstlane(in ? (int)(p.T * p.H * 2) : 0);
        load_row(buffer_rsrc(p.X, bytes), x_at, g, g == ng - 1, r.x[0]);
    };
    // the first weights are on their way while the expert's tokens are looked up
    Group r[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load_w(r[d]);
        next();
    }
    const int count = setup.find(p, ids, y, by_pair, e);
    if (count == 0) return;
    for (int c0 = 0; c0 < count; c0 += 16) {
        x_at.set(c0 + li < count ? (uint32_t)((setup.list[c0 + li] / p.k) * p.H) * 2 : kFar, (int)p.H, ng, q);
        at = At{0, w};
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (c0 > 0) load_w(r[d]);
            load_x(r[d]);
            next();
        }
        v4f acc[1] = {};
        int tile = tile0, done = 0;
        auto finish = [&]() LLMINT8_MOE_INLINE {
            mfma_settle();
            sh.red[w][lane] = acc[0];
            acc[0] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            __syncthreads();
            if (tid < 128) {  // an output a thread (up: two lane quarters on)
                const float* red = (const float*)sh.red;
                float gate = red[tid], up = red[128 + tid];
#pragma unroll
                for (int i = 1; i < WV; ++i) {
                    gate += red[256 * i + tid];
                    up += red[256 * i + 128 + tid];
                }
                const int l = tid >> 2, i = c0 + (l & 15);
                if (i < count)
                    p.h[(int64_t)setup.list[i] * ip + 8 * tile + 4 * (l >> 4) + (tid & 3)] = swiglu<DT>(gate, up);
            }
            if (tile == tiles - 1) pad_rows(p, setup.list, c0, count < c0 + 16 ? count : c0 + 16, ip);
            __syncthreads();
            ++tile;
        };
        for (int s = 0; s < steps; s += D) {  // whole rounds, as above
#pragma unroll
            for (int d = 0; d < D; ++d) {
                group_product<DT, 1>(r[d].w, scale_here(r[d].e), r[d].x, acc);
                load_w(r[d]);
                load_x(r[d]);
                next();
                if (s + d < steps && ++done == gw) {
                    done = 0;
                    finish();
                }
            }
        }
    }
}

// ---- the second launch's work: blocks of columns, each of `steps` steps, one block after the other
// split evenly over the workgroups: each takes a run of steps, whole blocks and parts of its first
// and last.  With as many workgroups as blocks a run is a block.
struct Runs {
    int64_t steps, total, groups;
    int64_t from, to;  // this workgroup's

    __device__ __forceinline__ void set(int64_t blocks, int64_t n) {
        steps = n;
        total = blocks * n;
        groups = gridDim.x < total ? gridDim.x : total;  // (none without a step: the shares of a block are counted)
        from = start(blockIdx.x);
        to = start(blockIdx.x + 1);
    }
    __device__ __forceinline__ int64_t start(int64_t group) const {
        if (group >= groups) return total;
        return groups * steps == total ? group * steps : total * group / groups;
    }
    __device__ __forceinline__ int64_t owner(int64_t step) const { return ((step + 1) * groups - 1) / total; }
};

// The end of a run's share of a block of 4 Q columns: of every token the waves' sums in their order.
// A block of several shares has those go through memory (`most` places a block), and the last one to
// end adds them up in their order.
template <int DT, int Q, int MAXT, int WV>
__device__ __forceinline__ void put_tokens(const Fp8MoeArgs& p, const v4f (&ysum)[WV][MAXT][Q], const Runs& runs, int block,
                                           bool whole, int most, int* flag) {
    const int n = (int)p.T * Q;
    auto store = [&](int i, const v4f& y) LLMINT8_MOE_INLINE {
        u32x2 o;
        o[0] = (uint32_t)from_f32<DT>(y[0]) | ((uint32_t)from_f32<DT>(y[1]) << 16);
        o[1] = (uint32_t)from_f32<DT>(y[2]) | ((uint32_t)from_f32<DT>(y[3]) << 16);
        *(u32x2*)(p.Y + (int64_t)(i / Q) * p.H + (int64_t)block * (4 * Q) + 4 * (i % Q)) = o;
    };
    auto sum = [&](int i) LLMINT8_MOE_INLINE {
        v4f y = ysum[0][i / Q][i % Q];
#pragma unroll
        for (int v = 1; v < WV; ++v) y += ysum[v][i / Q][i % Q];
        return y;
    };
    __syncthreads();
    if (whole) {
        for (int i = threadIdx.x; i < n; i += 64 * WV) store(i, sum(i));
        return;
    }
    const int first = (int)runs.owner(block * runs.steps), parts = (int)runs.owner(block * runs.steps + runs.steps - 1) - first + 1;
    const __amdgpu_buffer_rsrc_t rp = buffer_rsrc(p.partial + (int64_t)block * most * n * 4, (int64_t)most * n * 16);
    const int own = __builtin_amdgcn_readfirstlane(16 * n * ((int)blockIdx.x - first));
    for (int i = threadIdx.x; i < n; i += 64 * WV) store_part(rp, 16 * i, own, sum(i));
    if (!last_part(p.counters + block, parts, flag)) return;
    for (int i = threadIdx.x; i < n; i += 64 * WV) {
        v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int v = 0; v < parts; ++v) y += load_part(rp, 16 * i, 16 * n * v);
        store(i, y);
    }
}

// ---- down and the weighted sum: blocks of 16 columns of H, all entries.  A share's groups of I,
// entry after entry, are split evenly over the waves and run through D sets of registers;
// a wave ends an entry (or its share of it) by adding p times its sums to its own rows of token
// sums in LDS.
template <int DT, int MG, int MAXT, int WV>
__global__ __launch_bounds__(64 * WV) void moe_down_kernel(Fp8MoeArgs p, int blocks, int most) {
    constexpr int D = MG == 1 ? (WV == 8 ? 4 : 3) : 2, MAXN = MAXT * kMaxTopK;
    __shared__ v4f ysum[WV][MAXT][4];  // a wave's sums of 16 columns per token
    __shared__ int32_t table[3 * MAXN], pairs[MAXN];
    __shared__ float weights[MAXN];
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int T = (int)p.T, k = p.k, n = T * k;
    const int64_t ip = fp8_pitch(p.I), isp = fp8_scale_pitch_of(p.I);
    const int ng = (int)(ip / 128);
    const int entries = __builtin_amdgcn_readfirstlane(p.table[0]);
    for (int i = tid; i < 3 * n; i += 64 * WV) table[i] = p.table[1 + i];  // past the entries: unread
    for (int i = tid; i < n; i += 64 * WV) {
        pairs[i] = p.pairs[i];
        weights[i] = p.weights[i];
    }
    Runs runs;
    runs.set(blocks, entries * ng > 0 ? entries * ng : 1);
    for (int64_t at = runs.from; at < runs.to;) {
        const int block = __builtin_amdgcn_readfirstlane((int)(at / runs.steps));
        const int64_t ends = (block + 1) * runs.steps < runs.to ? (block + 1) * runs.steps : runs.to;
        const int begin = __builtin_amdgcn_readfirstlane((int)(at - block * runs.steps)), end = __builtin_amdgcn_readfirstlane((int)(ends - block * runs.steps));
        at = ends;
        const int64_t n0 = 16 * (int64_t)block;
        for (int i = tid; i < WV * T * 4; i += 64 * WV) ysum[i / (4 * T)][(i >> 2) % T][i & 3] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        __syncthreads();
        const int from = begin + (int)((int64_t)(end - begin) * w / WV), to = begin + (int)((int64_t)(end - begin) * (w + 1) / WV);
        if (from < to && entries * ng > 0) {
            const uint32_t w_off = (uint32_t)(li * ip + 16 * q);
            const int64_t h_bytes = (int64_t)n * ip * 2;
            const int64_t scale_rows = ceil_div(p.H, 128);
            struct Group {
                u32x4 w[2], x[MG][4];
                Scale s;
            };
            // the next load's entry and group, and that entry's expert and rows of h
            int le = from / ng, lg = from - le * ng, expert = 0, left = to - from;
            uint32_t h_off[MG];
            auto open = [&]() LLMINT8_MOE_INLINE {
                if (le >= entries) return;
                expert = __builtin_amdgcn_readfirstlane(table[3 * le]);
                const int first = table[3 * le + 1], count = table[3 * le + 2];
#pragma unroll
                for (int j = 0; j < MG; ++j) {
                    const int i = 16 * j + li;
                    h_off[j] = i < count ? (uint32_t)(pairs[first + i] * ip + 16 * q) * 2 : kFar;
                }
            };
            auto load = [&](Group& r) LLMINT8_MOE_INLINE {
                const bool in = left > 0;  // past the share: zeros
                const int g = in ? lg : 0;  // (an empty resource takes no scalar offset: the check subtracts it)
                const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(p.W2 + ((int64_t)expert * p.H + n0) * ip, in ? 16 * ip : 0);
                const __amdgpu_buffer_rsrc_t rh = buffer_rsrc(p.h, in ? h_bytes : 0);
#pragma unroll
                for (int h = 0; h < 2; ++h) r.w[h] = load16(rw, w_off + 64 * h, g * 128);
#pragma unroll
                for (int j = 0; j < MG; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) r.x[j][i] = load16(rh, h_off[j] + 128 * (i >> 1) + 16 * (i & 1), g * 256);
                r.s = load_scale(p.s2 + (expert * scale_rows + (n0 >> 7)) * isp, lg);
                __builtin_amdgcn_sched_barrier(0);  // as above
                --left;
                if (++lg == ng) {
                    lg = 0;
                    ++le;
                    open();
                }
            };
            v4f acc[MG] = {};
            int ce = le, cg = lg;  // the entry and group being multiplied
            auto flush = [&]() LLMINT8_MOE_INLINE {
                mfma_settle();
                const int first = table[3 * ce + 1], count = table[3 * ce + 2];
#pragma unroll
                for (int j = 0; j < MG; ++j) {
                    const int i = 16 * j + li;
                    if (i < count) {
                        const int pair = pairs[first + i];
                        const float pt = weights[pair];
                        v4f y = ysum[w][pair / k][q];
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(pt, acc[j][r], y[r]);
                        ysum[w][pair / k][q] = y;
                    }
                    acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                }
            };
            Group r[D];
            open();
#pragma unroll
            for (int d = 0; d < D; ++d) load(r[d]);
            const int steps = to - from;
            for (int s = 0; s < steps; s += D) {  // whole rounds, as above
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    group_product<DT, MG>(r[d].w, scale_here(r[d].s), r[d].x, acc);
                    load(r[d]);
                    if (s + d < steps && (++cg == ng || s + d + 1 == steps)) {
                        flush();
                        cg = 0;
                        ++ce;
                    }
                }
            }
        }
        put_tokens<DT, 4, MAXT, WV>(p, ysum, runs, block, end - begin == runs.steps, most, &flag);
        __syncthreads();  // before the sums are cleared
    }
}

// ---- the same in the light form: 8 columns of H, two entries (of up to 8 tokens) at a time, the
// even one in rows and columns 0 .. 7 of the instruction, the odd one in 8 .. 15.
template <int DT, int MAXT, int WV, int C, int D>
__global__ __launch_bounds__(64 * WV) void moe_down_light_kernel(Fp8MoeArgs p, int blocks, int most) {
    constexpr int MAXN = MAXT * kMaxTopK;
    __shared__ v4f ysum[WV][MAXT][2];  // a wave's sums of 8 columns per token
    __shared__ int32_t table[3 * MAXN], pairs[MAXN];
    __shared__ float weights[MAXN];
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4, half = li >> 3;
    const int T = (int)p.T, k = p.k, n = T * k;
    const int64_t ip = fp8_pitch(p.I), isp = fp8_scale_pitch_of(p.I);
    const int ng = (int)(ip / 128);
    const int entries = __builtin_amdgcn_readfirstlane(p.table[0]), twos = (entries + 1) / 2;
    for (int i = tid; i < 3 * n; i += 64 * WV) table[i] = p.table[1 + i];  // past the entries: unread
    for (int i = tid; i < n; i += 64 * WV) {
        pairs[i] = p.pairs[i];
        weights[i] = p.weights[i];
    }
    Runs runs;
    runs.set(blocks, twos * ng > 0 ? twos * ng : 1);
    for (int64_t run = runs.from; run < runs.to;) {
        const int block = __builtin_amdgcn_readfirstlane((int)(run / runs.steps));
        const int64_t ends = (block + 1) * runs.steps < runs.to ? (block + 1) * runs.steps : runs.to;
        const int begin = __builtin_amdgcn_readfirstlane((int)(run - block * runs.steps)), end = __builtin_amdgcn_readfirstlane((int)(ends - block * runs.steps));
        run = ends;
        const int64_t n0 = 8 * (int64_t)block;
        for (int i = tid; i < WV * T * 2; i += 64 * WV) ysum[i / (2 * T)][(i >> 1) % T][i & 1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        __syncthreads();
        // this share's steps (groups of I, two entries after two entries) go round the waves C at a time,
        // so that what the workgroup reads at a time lies together
        const int total = end - begin, round = WV * C, own = total - total / round * round - w * C;
        const int steps = total / round * C + (own < 0 ? 0 : (own < C ? own : C));
        if (steps > 0 && twos * ng > 0) {
            const int64_t h_bytes = (int64_t)n * ip * 2;
            const int64_t scale_rows = ceil_div(p.H, 128);
            struct Group {
                u32x4 w[2], x[1][4];
                Scale s;
            };
            // the next load's two entries and group; of this lane's entry its row of W2, its scales
            // and its token's row of h (an odd count: the last entry's weights times zeros)
            struct At {
                int two, g, c;  // the entries, the group, the place among C
                __device__ __forceinline__ bool next(int ng) {  // true: other entries
                    const int was = two;
                    g += ++c == C ? (WV - 1) * C + 1 : 1;
                    c = c == C ? 0 : c;
                    while (g >= ng) {
                        g -= ng;
                        ++two;
                    }
                    return two != was;
                }
            };
            At l{(begin + w * C) / ng, (begin + w * C) % ng, 0}, m = l;  // of the next load, and of the next product
            int left = steps;
            const uint8_t *row = nullptr, *scales = nullptr;
            uint32_t h_off = kFar;
            auto open = [&]() LLMINT8_MOE_INLINE {
                const int mine = 2 * l.two + half, at = mine < entries ? mine : entries - 1;
                const int e = table[3 * at], first = table[3 * at + 1], count = mine < entries ? table[3 * at + 2] : 0;
                row = p.W2 + ((int64_t)e * p.H + n0 + (li & 7)) * ip + 16 * q;
                scales = p.s2 + (e * scale_rows + (n0 >> 7)) * isp;
                h_off = (li & 7) < count ? (uint32_t)(pairs[first + (li & 7)] * ip + 16 * q) * 2 : kFar;
            };
            auto load = [&](Group& r) LLMINT8_MOE_INLINE {
                const uint8_t* from = row + l.g * 128;
                r.w[0] = *(const u32x4*)from;
                r.w[1] = *(const u32x4*)(from + 64);
                const __amdgpu_buffer_rsrc_t rh = buffer_rsrc(p.h, left > 0 ? h_bytes : 0);  // past the share: zeros
#pragma unroll
                for (int i = 0; i < 4; ++i) r.x[0][i] = load16(rh, h_off + 128 * (i >> 1) + 16 * (i & 1), l.g * 256);
                r.s = load_scale(scales, l.g);
                __builtin_amdgcn_sched_barrier(0);  // as above
                if (--left > 0) {
                    if (l.next(ng)) open();
                } else {  // from here on one line of weights
                    row = p.W2;
                    l.g = 0;
                }
            };
            v4f acc[1] = {};
            // The results of an entry's rows with its own tokens; the even entry first, then the odd one: a
            // token may be in both, on lanes of either half, whose sums are one word of LDS.  One lane takes
            // part in one of the two at most, so without the fence the compiler might join them.
            auto flush = [&](int two) LLMINT8_MOE_INLINE {
                mfma_settle();
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int at = 2 * two + t;
                    if (half == t && (q >> 1) == t && at < entries && (li & 7) < table[3 * at + 2]) {
                        const int pair = pairs[table[3 * at + 1] + (li & 7)];
                        const float pt = weights[pair];
                        v4f y = ysum[w][pair / k][q & 1];
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(pt, acc[0][r], y[r]);
                        ysum[w][pair / k][q & 1] = y;
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
                acc[0] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            };
            Group r[D];
            open();
#pragma unroll
            for (int d = 0; d < D; ++d) load(r[d]);
            for (int s = 0; s < steps; s += D) {  // whole rounds, as above
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    group_product<DT, 1>(r[d].w, scale_here(r[d].s), r[d].x, acc);
                    load(r[d]);
                    if (s + d < steps) {
                        const int two = m.two;
                        if (m.next(ng) || s + d + 1 == steps) flush(two);
                    }
                }
            }
        }
        put_tokens<DT, 2, MAXT, WV>(p, ysum, runs, block, end - begin == runs.steps, most, &flag);
        __syncthreads();  // before the sums are cleared
    }
}

// ---- many tokens an expert (16 MG at a time) in a large layer: there the tokens' values, which every wave of the
// kernels above reads for itself, are most of what a compute unit reads (12 TB/s from the L2s in all).
// Here the eight waves of a workgroup take a tile of 16 columns each, and share the tokens: a group's
// values come straight into LDS (16-byte chunk c of token t at chunk c ^ t, so that 16 tokens' reads
// of one chunk meet all banks), two groups ahead in three slots.  The waves meet once per group;
// each has whole sums, so nothing is joined.
template <int MG>
struct Tokens {
    static constexpr int kLoads = MG / 2;  // of a wave: 4 tokens each
    static constexpr int kSlot = 16 * MG * 256;
    uint32_t off[kLoads], past[kLoads];  // this lane's chunks in the first group; kFar: none in the last

    // row: of token t its offset, or kFar; n: values of a row (past them the last group reads zeros)
    template <class F>
    __device__ __forceinline__ void set(F&& row, int n, int ng) {
        const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int t = 4 * (kLoads * w + j) + lane / 16, c = (lane ^ t) & 15;
            off[j] = row(t) + 16 * c;
            past[j] = 128 * (ng - 1) + 8 * c < n ? 0u : kFar;
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint8_t* slot, int g, int ng) const {
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int at = __builtin_amdgcn_readfirstlane(g < ng ? 256 * g : 0);
        const uint32_t far = g < ng ? 0u : kFar, tail = g == ng - 1 ? kFar : 0u;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t o = off[j] | far | (tail & past[j]);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(slot + (kLoads * w + j) * 1024), 16, (int)o, at, 0, 0);
        }
    }
    static __device__ __forceinline__ void read(const uint8_t* slot, u32x4 (&x)[MG][4]) {
        const int li = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
#pragma unroll
        for (int j = 0; j < MG; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[j][i] = *(const u32x4*)(slot + (16 * j + li) * 256 + (((8 * (i >> 1) + 2 * q + (i & 1)) ^ li) << 4));
    }
};

// wait for this wave's LDS reads and all but the N newest loads, then the bare barrier
template <int N>
__device__ __forceinline__ void wait_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int DT, int MG>
__global__ __launch_bounds__(512, 2) void moe_up_many_kernel(Fp8MoeArgs p, int spans, int chunk, int n_zero) {
    constexpr int D = 2, S = 3, kWeightLoads = 6;  // (of a step: vector loads all, as the waits count them)
    struct Shared {  // (one variable: with several the compiler waits for all loads at each read)
        union {
            __attribute__((aligned(1024))) uint8_t x[S][Tokens<MG>::kSlot];
            struct {
                uint32_t mask[kMaxExperts][4];
                int first[kMaxExperts];
            } t;
        };
        UpSetup<false> setup;
    };
    __shared__ Shared sh;
    auto& setup = sh.setup;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int32_t* ids = setup.template route<8>(p);
    if (blockIdx.x == 0) {
        for (int i = tid; i < n_zero; i += blockDim.x) p.counters[i] = 0;
        build_table(ids, (int)p.T, (int)p.E, p.k, chunk, p.table, p.pairs, sh.t.mask, sh.t.first);
        return;
    }
    const int e = (int)(blockIdx.x - 1) / spans, span = (int)(blockIdx.x - 1) % spans;
    const int count = setup.find(p, ids, e, 0, e);
    if (count == 0) return;  // the same in every thread
    const int* list = setup.list;
    const int64_t hp = fp8_pitch(p.H), hsp = fp8_scale_pitch_of(p.H), ip = fp8_pitch(p.I);
    const int tiles = (int)(p.I / 16), ng = (int)(hp / 128), tile = 8 * span + w;
    const bool has = tile < tiles;
    const int64_t i0 = 16 * (int64_t)(has ? tile : 0), s_bytes = ceil_div(2 * p.I, 128) * hsp;
    const uint8_t* W = p.W13 + (int64_t)e * 2 * p.I * hp;
    const uint8_t *Wg = W + i0 * hp, *Wu = W + (p.I + i0) * hp;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(p.X, p.T * p.H * 2), rs = buffer_rsrc(p.s13 + (int64_t)e * s_bytes, s_bytes);
    const uint32_t w_off = (uint32_t)(li * hp + 16 * q), sg = (uint32_t)((i0 >> 7) * hsp), su = (uint32_t)(((p.I + i0) >> 7) * hsp);
    struct Group {
        u32x4 g[2], u[2];
        Scale eg, eu;
    };
    // Workgroups start at different groups: rows of 4096 bytes have a group's lines in the same few
    // memory channels (64 tokens, 16 experts of 4096 x 2048, top 4: 53.7 us, from the first group 69).
    const int g0 = __builtin_amdgcn_readfirstlane((int)((blockIdx.x - 1) * 5 % ng));
    auto group_at = [&](int s) LLMINT8_MOE_INLINE { return s >= ng ? ng : (s + g0 >= ng ? s + g0 - ng : s + g0); };
    for (int c0 = 0; c0 < count; c0 += 16 * MG) {
        Tokens<MG> tokens;
        tokens.set([&](int t) { return c0 + t < count ? (uint32_t)((list[c0 + t] / p.k) * p.H) * 2 : kFar; }, (int)p.H, ng);
        auto load_w = [&](Group& r, int s) LLMINT8_MOE_INLINE {
            const bool in = s < ng && has;  // else zeros
            const int at = in ? group_at(s) : 0, bytes = in ? 16 * (int)hp : 0;
            const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(Wg, bytes), ru = buffer_rsrc(Wu, bytes);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                r.g[h] = load16(rg, w_off + 64 * h, at * 128);
                r.u[h] = load16(ru, w_off + 64 * h, at * 128);
            }
            r.eg = load_scale(rs, sg, at);
            r.eu = load_scale(rs, su, at);
            __builtin_amdgcn_sched_barrier(0);  // as above
        };
        auto load_x = [&](int s, int slot) LLMINT8_MOE_INLINE {
            tokens.load(rx, sh.x[slot], group_at(s), ng);
            __builtin_amdgcn_sched_barrier(0);
        };
        v4f ag[MG] = {}, au[MG] = {};
        Group r[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load_x(d, d);
            load_w(r[d], d);
        }
        int slot = 0;
        for (int s = 0; s < ng; s += D) {  // whole rounds, as above
#pragma unroll
            for (int d = 0; d < D; ++d) {
                // the group's values are in, and every wave is done with the slot before it
                wait_barrier<2 * kWeightLoads + Tokens<MG>::kLoads>();
                load_x(s + d + 2, slot == 0 ? 2 : slot - 1);
                u32x4 x[MG][4];
                Tokens<MG>::read(sh.x[slot], x);
                group_product<DT, MG>(r[d].g, scale_here(r[d].eg), x, ag);
                group_product<DT, MG>(r[d].u, scale_here(r[d].eu), x, au);
                load_w(r[d], s + d + 2);
                slot = slot == 2 ? 0 : slot + 1;
            }
        }
        mfma_settle();
#pragma unroll
        for (int j = 0; j < MG; ++j) {
            const int i = c0 + 16 * j + li;
            if (has && i < count) {
                u32x2 o;
                o[0] = (uint32_t)swiglu<DT>(ag[j][0], au[j][0]) | ((uint32_t)swiglu<DT>(ag[j][1], au[j][1]) << 16);
                o[1] = (uint32_t)swiglu<DT>(ag[j][2], au[j][2]) | ((uint32_t)swiglu<DT>(ag[j][3], au[j][3]) << 16);
                *(u32x2*)(p.h + (int64_t)list[i] * ip + i0 + 4 * q) = o;
            }
        }
        if (span == spans - 1) pad_rows(p, list, c0, count < c0 + 16 * MG ? count : c0 + 16 * MG, ip);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load is bound for the slots any more
        __syncthreads();
    }
}

// The second launch: 128 columns of H, an entry after the other.
template <int DT, int MG, int MAXT>
__global__ __launch_bounds__(512, 2) void moe_down_many_kernel(Fp8MoeArgs p) {
    constexpr int D = 2, S = 3, kWeightLoads = 3, MAXN = MAXT * kMaxTopK;
    struct Shared {  // one variable, as above
        __attribute__((aligned(1024))) uint8_t x[S][Tokens<MG>::kSlot];
        v4f ysum[8][MAXT][4];  // a wave's 16 columns of every token
        int32_t table[3 * MAXN / 8], pairs[MAXN];
        float weights[MAXN];
        int flag;
    };
    __shared__ Shared sh;
    auto& xs = sh.x;
    auto& ysum = sh.ysum;
    auto& table = sh.table;
    auto& pairs = sh.pairs;
    auto& weights = sh.weights;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int T = (int)p.T, k = p.k, n = T * k;
    const bool has = 128 * (int64_t)blockIdx.x + 16 * w < p.H;
    const int64_t n0 = has ? 128 * (int64_t)blockIdx.x + 16 * w : 0;
    const int64_t ip = fp8_pitch(p.I), isp = fp8_scale_pitch_of(p.I);
    const int ng = (int)(ip / 128);
    const int entries = __builtin_amdgcn_readfirstlane(p.table[0]);  // (at most E + n / (16 MG), which the plan holds to MAXN / 8)
    for (int i = tid; i < 3 * entries; i += 512) table[i] = p.table[1 + i];
    for (int i = tid; i < n; i += 512) {
        pairs[i] = p.pairs[i];
        weights[i] = p.weights[i];
    }
    for (int i = tid; i < 8 * T * 4; i += 512) ysum[i / (4 * T)][(i >> 2) % T][i & 3] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    const int total = entries * ng, parts = gridDim.y, part = blockIdx.y;
    const int from = (int)((int64_t)total * part / parts), to = (int)((int64_t)total * (part + 1) / parts);
    if (from < to) {
        const __amdgpu_buffer_rsrc_t rh = buffer_rsrc(p.h, (int64_t)n * ip * 2);
        const int64_t scale_rows = ceil_div(p.H, 128), e_scales = scale_rows * isp;
        const uint32_t w_off = (uint32_t)(li * ip + 16 * q), s_row = (uint32_t)((n0 >> 7) * isp);
        struct Group {
            u32x4 w[2];
            Scale s;
        };
        // the next load's entry and group, and that entry's expert and rows of h
        int le = from / ng, lg = from - le * ng, expert = 0, left = to - from;
        Tokens<MG> tokens;
        auto open = [&]() LLMINT8_MOE_INLINE {
            if (le >= entries) return;
            expert = __builtin_amdgcn_readfirstlane(table[3 * le]);
            const int first = table[3 * le + 1], count = table[3 * le + 2];
            tokens.set([&](int t) { return t < count ? (uint32_t)(pairs[first + t] * ip) * 2 : kFar; }, (int)ip, ng);
        };
        auto load_x = [&](int slot) LLMINT8_MOE_INLINE {
            tokens.load(rh, xs[slot], left > 0 ? lg : ng, ng);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto load_w = [&](Group& r) LLMINT8_MOE_INLINE {
            const bool in = left > 0 && has;  // else zeros
            const int g = in ? lg : 0;
            const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(p.W2 + ((int64_t)expert * p.H + n0) * ip, in ? 16 * ip : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) r.w[h] = load16(rw, w_off + 64 * h, g * 128);
            r.s = load_scale(buffer_rsrc(p.s2 + expert * e_scales, e_scales), s_row, g);
            __builtin_amdgcn_sched_barrier(0);
            --left;
            if (++lg == ng) {
                lg = 0;
                ++le;
                open();
            }
        };
        v4f acc[MG] = {};
        int ce = le, cg = lg;  // the entry and group being multiplied
        auto flush = [&]() LLMINT8_MOE_INLINE {
            mfma_settle();
            const int first = table[3 * ce + 1], count = table[3 * ce + 2];
#pragma unroll
            for (int j = 0; j < MG; ++j) {
                const int i = 16 * j + li;
                if (i < count) {
                    const int pair = pairs[first + i];
                    const float pt = weights[pair];
                    v4f y = ysum[w][pair / k][q];
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(pt, acc[j][r], y[r]);
                    ysum[w][pair / k][q] = y;
                }
                acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            }
        };
        Group r[D];
        open();
        // (the two parts of a load take the same place: load_w moves on)
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load_x(d);
            load_w(r[d]);
        }
        const int steps = to - from;
        int slot = 0;
        for (int s = 0; s < steps; s += D) {  // whole rounds, as above
#pragma unroll
            for (int d = 0; d < D; ++d) {
                wait_barrier<2 * kWeightLoads + Tokens<MG>::kLoads>();  // as above
                load_x(slot == 0 ? 2 : slot - 1);
                u32x4 x[MG][4];
                Tokens<MG>::read(xs[slot], x);
                group_product<DT, MG>(r[d].w, scale_here(r[d].s), x, acc);
                load_w(r[d]);
                slot = slot == 2 ? 0 : slot + 1;
                if (s + d < steps && (++cg == ng || s + d + 1 == steps)) {
                    flush();
                    cg = 0;
                    ++ce;
                }
            }
        }
    }
    auto store = [&](int i, const v4f& y) LLMINT8_MOE_INLINE {
        u32x2 o;
        o[0] = (uint32_t)from_f32<DT>(y[0]) | ((uint32_t)from_f32<DT>(y[1]) << 16);
        o[1] = (uint32_t)from_f32<DT>(y[2]) | ((uint32_t)from_f32<DT>(y[3]) << 16);
        if (has) *(u32x2*)(p.Y + (int64_t)(i >> 2) * p.H + n0 + 4 * (i & 3)) = o;
    };
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into this workgroup's LDS may outlive it
    if (parts == 1) {
        for (int i = lane; i < 4 * T; i += 64) store(i, ysum[w][i >> 2][i & 3]);
        return;
    }
    // a part's sums, wave after wave; the last part to end adds them up in their order
    const int64_t block_bytes = (int64_t)8 * 4 * T * 16;
    const __amdgpu_buffer_rsrc_t rp = buffer_rsrc((const uint8_t*)p.partial + (int64_t)blockIdx.x * parts * block_bytes, parts * block_bytes);
    const uint32_t own = (uint32_t)(w * 4 * T * 16);
    for (int i = lane; i < 4 * T; i += 64) store_part(rp, own + 16 * i, (uint32_t)(part * block_bytes), ysum[w][i >> 2][i & 3]);
    if (!last_part(p.counters + blockIdx.x, parts, &sh.flag)) return;
    for (int i = lane; i < 4 * T; i += 64) {
        v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int v = 0; v < parts; ++v) y += load_part(rp, own + 16 * i, (uint32_t)(v * block_bytes));
        store(i, y);
    }
}

// The first launch's grid: workgroup 0 (the table), then `rows` (pairs or experts) of `spans` spans
// of `span` tiles.  A workgroup's setup (choosing the experts or reading them, the list) is paid
// once per span, as long as about `enough` workgroups are left: 4 tokens, 64 experts of 2048 x 768,
// top 8: 25.5 us with spans of 3, 32.6 with single tiles; longer ones gain nothing (8 tokens, 128
// such experts: 48.3 us with spans of 3, 47.3 with 6, 59.6 with 1; 16 tokens, top 4: 38.6, 44.9, 47.2).
// The wide form, 37 tokens, 60 experts of 2064 x 1424, top 4 (where the form for many tokens runs now): 78
// us with 1024 workgroups left, 89 with 512 and with 2048; 64 tokens, 160 experts of 5120 x 1536, top 6:
// 451, 451 and 456.
struct UpGrid {
    int by_pair, spans, span;
    int64_t grid;
};
UpGrid up_grid(const Fp8MoeArgs& p, int columns, int64_t enough, int64_t longest) {
    UpGrid g;
    g.by_pair = p.T * p.k < p.E;
    const int64_t rows = g.by_pair ? p.T * p.k : p.E, tiles = p.I / columns;
    int64_t span = tiles * rows / enough;
    span = span < 1 ? 1 : (span > longest ? longest : span);
    g.span = (int)span;
    g.spans = (int)ceil_div(tiles, span);
    g.grid = 1 + g.spans * rows;
    return g;
}

// MG: pieces of 16 tokens multiplied at once; 0: the light form
template <int DT, int MG, bool MANY = false>
hipError_t launch_up(const Fp8MoeArgs& p, const Fp8MoePlan& plan, hipStream_t stream) {
    const int chunk = plan.chunk, n_zero = plan.parts > 1 ? (int)plan.blocks : 0;
    const bool routes = MG == 0 && p.T <= kRouteTokens && p.T * p.k <= kRouteChoices;
    if (!routes) {  // (what comes next reads the experts that this one writes)
        moe_route_kernel<<<(unsigned)p.T, 64, 0, stream>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if constexpr (MG == 0) {
        const UpGrid g = up_grid(p, 8, 1024, 3);
        constexpr int kThreads = 64 * kLightUpWaves;
        if (routes) moe_up_light_kernel<DT, true><<<(unsigned)g.grid, kThreads, 0, stream>>>(p, g.spans, g.span, g.by_pair, chunk, n_zero);
        else moe_up_light_kernel<DT, false><<<(unsigned)g.grid, kThreads, 0, stream>>>(p, g.spans, g.span, g.by_pair, chunk, n_zero);
    } else {
        if constexpr (MANY) {
            const int spans = (int)ceil_div(p.I, 128);
            moe_up_many_kernel<DT, MG><<<(unsigned)(1 + p.E * spans), 512, 0, stream>>>(p, spans, chunk, n_zero);
        } else {
            const UpGrid g = up_grid(p, 16, 1024, 8);
            moe_up_kernel<DT, MG><<<(unsigned)g.grid, 64 * kUpWaves, 0, stream>>>(p, g.spans, g.span, g.by_pair, chunk, n_zero);
        }
    }
    return hipGetLastError();
}

template <int DT, int MG, bool MANY = false>
hipError_t launch_down(const Fp8MoeArgs& p, const Fp8MoePlan& plan, hipStream_t stream) {
    const int blocks = (int)plan.blocks, most = plan.parts;
    if constexpr (MG == 0) {
        if (p.T <= 16) moe_down_light_kernel<DT, 16, 8, 3, 2><<<plan.groups, 512, 0, stream>>>(p, blocks, most);
        else moe_down_light_kernel<DT, 128, 8, 3, 2><<<plan.groups, 512, 0, stream>>>(p, blocks, most);
    } else if constexpr (MANY) {
        const dim3 grid((unsigned)blocks, (unsigned)plan.parts);
        if (p.T <= 64) moe_down_many_kernel<DT, MG, 64><<<grid, 512, 0, stream>>>(p);
        else moe_down_many_kernel<DT, MG, 128><<<grid, 512, 0, stream>>>(p);
    } else {
        if (p.T <= 64) moe_down_kernel<DT, MG, 64, 16><<<plan.groups, 1024, 0, stream>>>(p, blocks, most);
        else moe_down_kernel<DT, MG, 128, 8><<<plan.groups, 512, 0, stream>>>(p, blocks, most);
    }
    return hipGetLastError();
}

template <int DT>
hipError_t moe_launch(const Fp8MoeArgs& p, const Fp8MoePlan& plan, hipStream_t stream) {
    const hipError_t e = plan.up == Fp8MoePlan::kLight  ? launch_up<DT, 0>(p, plan, stream)
                         : plan.up == Fp8MoePlan::kWide ? (plan.up_pieces == 1 ? launch_up<DT, 1>(p, plan, stream) : launch_up<DT, 2>(p, plan, stream))
                         : plan.up_pieces == 2          ? launch_up<DT, 2, true>(p, plan, stream)
                                                        : launch_up<DT, 4, true>(p, plan, stream);
    if (e != hipSuccess) return e;
    return plan.down == Fp8MoePlan::kLight  ? launch_down<DT, 0>(p, plan, stream)
           : plan.down == Fp8MoePlan::kWide ? (plan.down_pieces == 1 ? launch_down<DT, 1>(p, plan, stream) : launch_down<DT, 2>(p, plan, stream))
           : plan.down_pieces == 2          ? launch_down<DT, 2, true>(p, plan, stream)
                                            : launch_down<DT, 4, true>(p, plan, stream);
}

// Workgroups of the second launch (light or wide).  A compute unit reads about 20 bytes a nanosecond
// whether it holds one of them or two, so a few blocks past a multiple of 256 would cost a whole round:
// there 256 workgroups share the blocks' steps evenly; and half as many blocks or fewer are taken in
// parts.  The estimate, in 10 ns, has 3 us for joining and 1.5 us for setting up a run.  37 tokens, 60
// experts, top 4: 2064 x 1424 (258 blocks) 78.1 us a block each, shared by 256 53.2, by 512 54.5; 8 tokens,
// 64 experts of 1024 x 768, top 4 (128 blocks) 11.9 and 11.1; 4 tokens, 64 of 2048 x 768 (256) 12.8.
unsigned down_groups(int64_t blocks, int64_t steps) {
    const int64_t work = steps * 11;  // of one block's steps of 16 rows of 128 bytes
    const int64_t plain = ceil_div(blocks, 256) * (work + 150);
    if (blocks > 256) return (unsigned)(blocks * work / 256 + 700 < plain ? 256 : blocks);
    const int64_t parts = blocks > 0 ? 256 / blocks : 1;
    return (unsigned)(parts > 1 && work / parts + 600 < plain ? blocks * parts : blocks);
}

}  // namespace

Fp8MoePlan fp8_moe_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
    Fp8MoePlan plan{};
    const int64_t n = T * k, mean16 = 16 * n / E;  // 16 times the tokens that an expert has on average
    const int64_t some = k == E ? E : (int64_t)((double)E * -expm1((double)T * log1p(-(double)k / (double)E))) + 1;  // of even choices
    const int64_t met = T == 0 ? 0 : (some < E ? some : E);
    const int pieces = mean16 <= 28 * 16 || T <= 32 ? 2 : 4;
    // The first launch, by estimates in 10 ns (from 45 layers of 4 to 256 experts, 1 to 128 tokens):
    //   light: bytes at 3.1 TB/s, + 3 us; it chooses the experts itself where they are few (the others: + 3.5);
    //   wide: bytes at 5.5 TB/s (with two pieces 3.2: every wave reads the tokens), + 15 us (12);
    //   many: 11.3 ns a value of H for each 256 workgroups of 128 columns, + 3 us; it needs most experts
    //     met, as workgroups without tokens leave the others unevenly on the card.
    // 64 tokens, 32 experts of 2048 x 768, top 4: 33.6 light, 40.1 wide, 25.5 many; 4 tokens, 64 such, top 8:
    // 25.9, 36.4, 40.8; 16 tokens, 64 of 4096 x 1408, top 6: 137, 124, 129; 64 tokens, 160 of 5120 x 1536, top
    // 6: 496, 450, 413; 44 tokens, 16 of 2752 x 448, top 6: 27.6, 24.7, 28.4.
    const int64_t bytes = met * 2 * I * fp8_pitch(H), wgs = met * ceil_div(I, 128);
    const int64_t route = T <= kRouteTokens && n <= kRouteChoices ? 350 : 0;
    plan.up_pieces = mean16 <= 14 * 16 || T <= 16 ? 1 : 2;
    const int64_t light = bytes / 31000 + 300;
    const int64_t wide = (plan.up_pieces == 1 ? bytes / 55000 + 1500 : bytes / 32000 + 1200) + route;
    const int64_t many = ceil_div(wgs, 256) * H * 113 / 100 + 300 + route;
    plan.up = Fp8MoePlan::kWide;
    if (n >= E && many <= wide) {
        plan.up = Fp8MoePlan::kMany;
        plan.up_pieces = pieces;
    }
    if ((mean16 <= 8 * 16 || T <= 16) && light < (plan.up == Fp8MoePlan::kMany ? many : wide)) plan.up = Fp8MoePlan::kLight;
    // The second launch.  Many: most experts met, at least 20 blocks of 128 columns (8 parts of each are 160
    // workgroups), and at most as many entries as its table holds.  Parts: 64 tokens, 16 experts of 4096 x
    // 2048, top 4: 39.3 us in 8, 48.8 in 4, 52.6 in 16.  8 tokens, 8 of 4096 x 14336, top 2: 77.6 us, wide 91.0,
    // light 104; 40 tokens, 32 of 2880 x 2880, top 6: 65 and wide 96.  Whole calls with this form and with the
    // better of the others, by blocks: 64 tokens, 64 experts, I = 1024, top 6: 16 blocks 108.7 us and 96.3, 18
    // 114.4 and 119.5, 19 117.3 and 127.9, 20 122.6 and 133.2; 32 tokens, 16, 2048, top 4: 16 blocks 65.0 and
    // 60.2, 19 68.0 and 75.5, 20 70.4 and 77.4.  By experts, groups and blocks multiplied: 2048 (16 tokens, 8 of 4096 x
    // 1024, top 2) 39.5 and 41.3, 2560 55.2 and 56.0, 3520 58.9 and 62.3, 4096 60.5 and 64.4, 8192 90.5 and 94.8: below
    // the border too it gains a little.
    // Light where most experts have few tokens: 16 tokens, 64 of 2048 x 768, top 4: 18.1, wide 21.2; 64 tokens,
    // 64 of 2048 x 1024, top 6: 49.6 and 41.9; and while wide blocks are under one a compute unit, from where on
    // either may be ahead by up to 5 %.  Whole calls: one token, top 8 of 64, I = 1024: H = 3584 29.0 and 30.3, 4096
    // 30.1 and 31.1; one token, top 6 of 64, 5120 x 1536: 54.8 and 57.8; 4 tokens, top 8 of 128, 4096 x 1408: 133.2
    // and 131.5; 8 tokens, top 4 of 32, 4096 x 1024: 75.8 and 74.9; 16 tokens, top 2 of 128, 4096 x 1024: 93.6 and 91.0.
    const int64_t entries = (E < n ? E : n) + n / (16 * pieces), blocks128 = ceil_div(H, 128);
    if (n >= E && blocks128 >= 20 && E * ceil_div(I, 128) * blocks128 >= 4096 && entries <= (T <= 64 ? 64 : 128) * kMaxTopK / 8) {
        plan.down = Fp8MoePlan::kMany;
        plan.down_pieces = pieces;
        plan.chunk = 16 * pieces;
        plan.blocks = blocks128;
        plan.parts = blocks128 >= 32 ? (int)(blocks128 <= 256 ? 256 / blocks128 : 1) : 8;
        plan.partial_bytes = plan.parts > 1 ? T * blocks128 * 128 * plan.parts * 4 : 0;
        return plan;
    }
    plan.down = (T <= 8 || mean16 <= 3 * 16) && H / 16 < 256 ? Fp8MoePlan::kLight : Fp8MoePlan::kWide;
    plan.down_pieces = mean16 <= 14 * 16 || T <= 16 ? 1 : 2;
    const int64_t columns = plan.down == Fp8MoePlan::kLight ? 8 : 16;
    plan.chunk = plan.down == Fp8MoePlan::kLight ? 8 : 16 * plan.down_pieces;
    plan.blocks = H / columns;
    plan.groups = down_groups(plan.blocks, (plan.down == Fp8MoePlan::kLight ? ceil_div(met, 2) : met) * ceil_div(I, 128));
    plan.parts = plan.groups == plan.blocks ? 1 : (int)(plan.groups / (plan.blocks > 0 ? plan.blocks : 1)) + 2;
    plan.partial_bytes = plan.parts > 1 ? T * H * plan.parts * 4 : 0;
    return plan;
}

hipError_t launch_fp8_moe(int dt, const Fp8MoeArgs& p, const Fp8MoePlan& plan, hipStream_t stream) {
    return dt == F16 ? moe_launch<F16>(p, plan, stream) : moe_launch<BF16>(p, plan, stream);
}

}  // namespace llmint8
