// A mixture-of-experts layer for few tokens, its weights e4m3 codes with a power-of-two scale
// per 128 x 128 block, its activations 16-bit.  Per token x (a row of X) with logits l:
//   experts e_0, e_1, ...: the top_k largest logits (ties to the lowest index; -inf and NaN are
//     never taken, +inf counts as the largest finite number);
//   p_j = exp(l[e_j] - l[e_0]) / Z, Z the sum of exp(l - l[e_0]) over the chosen experts
//     (renormalize) or over all;
//   [g; u] = W13hat_e x (2I values), h = RN_T(silu(g) u), y = RN_T(sum_j p_j W2hat_e h).
//
// Bound by the bytes of the experts met, each read once (once per kMaxPieces * 16 tokens of one
// expert).  Two launches: gate, up and SwiGLU (h goes to the workspace), then down and the
// weighted sum; with more than kRouteTokens tokens a third one before them chooses the experts,
// which otherwise every workgroup of the first does for itself (that costs less than a launch).
//
// The products run on 16-bit matrix instructions (16x16x32): a code is exact in either 16-bit
// type, so nothing is lost against the coded weight, and the activations keep their 16 bits --
// few tokens leave the matrix units idle anyway.  Weights are the row side (16 rows), an expert's
// tokens the column side, 16 to a piece; lane l holds bytes 32 (l / 16) .. + 31 of its row's
// group of 128, and instruction s of a group takes 8 s .. 8 s + 7 of them from both operands (the
// order of a sum's terms is free, as long as both agree).  bf16 takes the scale in the
// conversion (an exact shift of the exponent); fp16 could not hold it, so there each group's sum
// is added with its scale.  Sums are fp32; the waves of a workgroup split them and meet in LDS in
// a fixed order, and every token has a column of its own, so neither the order of atomics nor a
// token's neighbours change its bits.
#include "fp8_common.hpp"
#include "launch.hpp"

namespace llmint8 {

namespace {

constexpr int kMaxTokens = 128;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kUpWaves = 8;
constexpr int kRouteTokens = kUpWaves;  // a wave per token

#define LLMINT8_MOE_INLINE __attribute__((always_inline))

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}
constexpr uint32_t kFar = 0x80000000u;  // an offset past every resource: reads zero

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

// The experts and weights of one token, by one wave; lane j < k returns choice j.  A lane holds C
// neighbouring experts, so that among equal values the lowest lane, and in it the first expert,
// is the lowest index.
template <int C>
__device__ __forceinline__ void route_lanes(const float* __restrict__ l, int E, int k, int renormalize, int& id, float& p) {
    const float kNone = -__builtin_inff();
    const int lane = threadIdx.x & 63;
    float v[C], all[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        v[i] = C * lane + i < E ? usable_logit(l[C * lane + i]) : kNone;
        all[i] = v[i];
    }
    float top = 0.0f, chosen = 0.0f;
    id = -1;
    p = 0.0f;
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
        if (j == 0) top = most;
        const float x = expf(most - top);
        chosen += x;
        if (lane == j) {
            id = at;
            p = x;
        }
    }
    float z = chosen;
    if (!renormalize) {
        float own = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) own += expf(all[i] - top);
        z = wave_reduce(own, 0.0f, [](float a, float b) { return a + b; });
    }
    if (id >= 0) p /= z;
}

__device__ __forceinline__ void route_token(const float* __restrict__ l, int E, int k, int renormalize, int& id, float& p) {
    if (E <= 64) route_lanes<1>(l, E, k, renormalize, id, p);
    else if (E <= 256) route_lanes<4>(l, E, k, renormalize, id, p);
    else route_lanes<16>(l, E, k, renormalize, id, p);
}

__global__ __launch_bounds__(64) void moe_route_kernel(Fp8MoeArgs p) {
    const int t = blockIdx.x, lane = threadIdx.x;
    int id;
    float w;
    route_token(p.logits + (int64_t)t * p.E, (int)p.E, p.k, p.renormalize, id, w);
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

// ---- gate, up and SwiGLU: a workgroup takes `span` tiles of 16 columns of I of one expert (16
// gate rows and 16 up rows each), its waves split the groups of H.  A wave's groups, tile after
// tile, run through D sets of registers, so that the next tile's weights are on their way while
// a tile's sums meet.  Workgroup 0 writes the table.  by_pair: workgroups go by pair of token and
// choice (each expert at its first pair), else by expert.
template <int DT, int MG, bool ROUTE>
__global__ __launch_bounds__(64 * kUpWaves, MG == 1 ? 4 : 2) void moe_up_kernel(Fp8MoeArgs p, int spans, int span, int by_pair) {
    constexpr int WV = kUpWaves, D = 2;
    union Shared {
        v4f red[WV][2 * MG][64];
        struct {
            uint32_t mask[kMaxExperts][4];
            int first[kMaxExperts];
        } t;
    };
    __shared__ Shared sh;
    __shared__ int32_t own_ids[ROUTE ? kRouteTokens * kMaxTopK : 1];
    __shared__ int list[kMaxTokens];
    __shared__ int part[2], dup;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int T = (int)p.T, E = (int)p.E, k = p.k;
    const int32_t* ids = p.ids;
    if (tid == 0) dup = 0;
    if constexpr (ROUTE) {
        if (w < T) {
            int id;
            float wt;
            route_token(p.logits + (int64_t)w * E, E, k, p.renormalize, id, wt);
            if (lane < k) {
                own_ids[w * k + lane] = id;
                if (blockIdx.x == 0) {
                    p.ids[w * k + lane] = id;
                    p.weights[w * k + lane] = wt;
                }
            }
        }
        ids = own_ids;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        build_table(ids, T, E, k, 16 * MG, p.table, p.pairs, sh.t.mask, sh.t.first);
        return;
    }
    const int y = (int)(blockIdx.x - 1) / spans, tile0 = (int)(blockIdx.x - 1) % spans * span;
    int e = y;
    if (by_pair) {
        e = ids[y];
        if (e < 0) return;
    }
    // the expert's tokens, ascending: list[place] = token * k + choice
    int mine = -1;
    if (tid < 128 && tid < T)
        for (int j = 0; j < k; ++j)
            if (ids[tid * k + j] == e) mine = tid * k + j;
    if (by_pair && mine >= 0 && mine < y) dup = 1;  // an earlier pair's workgroups do this expert
    const uint64_t have = __ballot(mine >= 0);
    if (w < 2 && lane == 0) part[w] = __popcll(have);
    __syncthreads();
    const int count = part[0] + part[1];
    if (count == 0 || dup) return;  // the same in every thread
    if (mine >= 0) list[(w == 1 ? part[0] : 0) + __popcll(have & ((1ull << lane) - 1ull))] = mine;
    __syncthreads();

    const int64_t hp = fp8_pitch(p.H), hsp = fp8_scale_pitch_of(p.H);
    const int tiles = (int)(p.I / 16), ng = (int)(hp / 128);
    const int my_tiles = tiles - tile0 < span ? tiles - tile0 : span;
    const int gw = (ng + WV - 1) / WV;  // groups of a wave (its last may lie past H: zeros)
    const int steps = my_tiles * gw;
    const uint8_t* W = p.W13 + (int64_t)e * 2 * p.I * hp;
    const uint8_t* S = p.s13 + (int64_t)e * ceil_div(2 * p.I, 128) * hsp;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(p.X, p.T * p.H * 2);
    const uint32_t w_off = (uint32_t)(li * hp + 32 * q);

    struct Group {
        u32x4 g[2], u[2], x[MG][4];
        float eg, eu;
    };
    for (int c0 = 0; c0 < count; c0 += 16 * MG) {
        uint32_t x_off[MG];
#pragma unroll
        for (int j = 0; j < MG; ++j) {
            const int i = c0 + 16 * j + li;
            x_off[j] = i < count ? (uint32_t)((list[i] / k) * p.H + 32 * q) * 2 : kFar;
        }
        int lt = 0, lg = w;  // the next load's tile and group
        auto load = [&](Group& r) LLMINT8_MOE_INLINE {
            const bool in = lt < my_tiles && lg < ng;
            const uint32_t far = in ? 0u : kFar;
            const int64_t i0 = 16 * (int64_t)(lt < my_tiles ? tile0 + lt : tile0);
            const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(W + i0 * hp, 16 * hp), ru = buffer_rsrc(W + (p.I + i0) * hp, 16 * hp);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t off = (w_off + (uint32_t)(lg * 128 + 16 * h)) | far;
                r.g[h] = load16(rg, off);
                r.u[h] = load16(ru, off);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t out = lg * 128 + 32 * q + 8 * i < p.H ? far : kFar;  // past H: the next row's
#pragma unroll
                for (int j = 0; j < MG; ++j) r.x[j][i] = load16(rx, (x_off[j] + (uint32_t)(lg * 128 + 8 * i) * 2) | out);
            }
            // the scales of the 16 rows (I is a multiple of 16: one block of rows each)
            r.eg = in ? e8m0_value(S[(i0 >> 7) * hsp + lg]) : 0.0f;
            r.eu = in ? e8m0_value(S[((p.I + i0) >> 7) * hsp + lg]) : 0.0f;
            lg += WV;
            if (lg >= gw * WV) {
                lg = w;
                ++lt;
            }
        };
        v4f ag[MG] = {}, au[MG] = {};
        int tile = tile0, done = 0;
        // after a tile's last group: the waves' sums meet, SwiGLU, h
        auto finish = [&]() LLMINT8_MOE_INLINE {
            mfma_settle();
#pragma unroll
            for (int j = 0; j < MG; ++j) {
                sh.red[w][j][lane] = ag[j];
                sh.red[w][MG + j][lane] = au[j];
                ag[j] = au[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            }
            __syncthreads();
            if (w < MG) {  // piece w: sums in the order of the waves
                v4f sgate = sh.red[0][w][lane], sup = sh.red[0][MG + w][lane];
#pragma unroll
                for (int i = 1; i < WV; ++i) {
                    sgate += sh.red[i][w][lane];
                    sup += sh.red[i][MG + w][lane];
                }
                const int i = c0 + 16 * w + li;
                if (i < count) {
                    uint16_t h[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) h[r] = from_f32<DT>(sgate[r] / (1.0f + expf(-sgate[r])) * sup[r]);
                    u32x2 v;
                    v[0] = (uint32_t)h[0] | ((uint32_t)h[1] << 16);
                    v[1] = (uint32_t)h[2] | ((uint32_t)h[3] << 16);
                    *(u32x2*)(p.h + (int64_t)list[i] * p.I + 16 * tile + 4 * q) = v;
                }
            }
            __syncthreads();
            ++tile;
        };
        Group r[D];
#pragma unroll
        for (int d = 0; d < D; ++d) load(r[d]);
        for (int s = 0; s < steps; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (s + d >= steps) break;
                group_product<DT, MG>(r[d].g, r[d].eg, r[d].x, ag);
                group_product<DT, MG>(r[d].u, r[d].eu, r[d].x, au);
                load(r[d]);
                if (++done == gw) {
                    done = 0;
                    finish();
                }
            }
        }
    }
}

// ---- down and the weighted sum: a workgroup takes 16 columns of H of all entries.  Their groups
// of I, entry after entry, are split evenly over the waves and run through D sets of registers;
// a wave ends an entry (or its share of it) by adding p times its sums to its own rows of token
// sums in LDS.
template <int DT, int MG, int MAXT, int WV>
__global__ __launch_bounds__(64 * WV) void moe_down_kernel(Fp8MoeArgs p) {
    constexpr int D = MG == 1 ? (WV == 8 ? 4 : 3) : 2, MAXN = MAXT * kMaxTopK;
    __shared__ v4f ysum[WV][MAXT][4];  // a wave's sums of 16 columns per token
    __shared__ int32_t table[3 * MAXN], pairs[MAXN];
    __shared__ float weights[MAXN];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int T = (int)p.T, k = p.k, n = T * k;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t ip = fp8_pitch(p.I), isp = fp8_scale_pitch_of(p.I);
    const int ng = (int)(ip / 128);
    const int entries = __builtin_amdgcn_readfirstlane(p.table[0]);
    for (int i = tid; i < 3 * n; i += 64 * WV) table[i] = p.table[1 + i];  // past the entries: unread
    for (int i = tid; i < n; i += 64 * WV) {
        pairs[i] = p.pairs[i];
        weights[i] = p.weights[i];
    }
    for (int i = tid; i < WV * T * 4; i += 64 * WV) ysum[i / (4 * T)][(i >> 2) % T][i & 3] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    const int64_t total = (int64_t)entries * ng;
    const int64_t from = total * w / WV, to = total * (w + 1) / WV;
    if (from < to) {
        const uint32_t w_off = (uint32_t)(li * ip + 32 * q);
        const __amdgpu_buffer_rsrc_t rh = buffer_rsrc(p.h, (int64_t)n * p.I * 2);
        const int64_t scale_rows = ceil_div(p.H, 128);
        struct Group {
            u32x4 w[2], x[MG][4];
            float s;
        };
        // the next load's entry and group, and that entry's expert and rows of h
        int le = (int)(from / ng), lg = (int)(from - (int64_t)le * ng), expert = 0;
        int64_t left = to - from;
        uint32_t h_off[MG];
        auto open = [&]() LLMINT8_MOE_INLINE {
            if (le >= entries) return;
            expert = __builtin_amdgcn_readfirstlane(table[3 * le]);
            const int first = table[3 * le + 1], count = table[3 * le + 2];
#pragma unroll
            for (int j = 0; j < MG; ++j) {
                const int i = 16 * j + li;
                h_off[j] = i < count ? (uint32_t)(pairs[first + i] * p.I + 32 * q) * 2 : kFar;
            }
        };
        auto load = [&](Group& r) LLMINT8_MOE_INLINE {
            const bool in = left > 0;
            const uint32_t far = in ? 0u : kFar;
            const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(p.W2 + ((int64_t)expert * p.H + n0) * ip, 16 * ip);
#pragma unroll
            for (int h = 0; h < 2; ++h) r.w[h] = load16(rw, (w_off + (uint32_t)(lg * 128 + 16 * h)) | far);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t out = lg * 128 + 32 * q + 8 * i < p.I ? far : kFar;  // past I: the next row's
#pragma unroll
                for (int j = 0; j < MG; ++j) r.x[j][i] = load16(rh, (h_off[j] + (uint32_t)(lg * 128 + 8 * i) * 2) | out);
            }
            r.s = in ? e8m0_value(p.s2[(expert * scale_rows + (n0 >> 7)) * isp + lg]) : 0.0f;
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
        const int steps = (int)(to - from);
        for (int s = 0; s < steps; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (s + d >= steps) break;
                group_product<DT, MG>(r[d].w, r[d].s, r[d].x, acc);
                load(r[d]);
                if (++cg == ng || s + d + 1 == steps) {
                    flush();
                    cg = 0;
                    ++ce;
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < T * 4; i += 64 * WV) {
        v4f y = ysum[0][i >> 2][i & 3];
#pragma unroll
        for (int v = 1; v < WV; ++v) y += ysum[v][i >> 2][i & 3];
        u32x2 o;
        o[0] = (uint32_t)from_f32<DT>(y[0]) | ((uint32_t)from_f32<DT>(y[1]) << 16);
        o[1] = (uint32_t)from_f32<DT>(y[2]) | ((uint32_t)from_f32<DT>(y[3]) << 16);
        *(u32x2*)(p.Y + (int64_t)(i >> 2) * p.H + n0 + 4 * (i & 3)) = o;
    }
}

template <int DT, int MG>
hipError_t moe_launch(const Fp8MoeArgs& p, hipStream_t stream) {
    const int by_pair = p.T * p.k < p.E;
    const int64_t rows = by_pair ? p.T * p.k : p.E, tiles = p.I / 16;
    // tiles of a workgroup: its setup (choosing the experts or reading them, the list) is paid
    // once, as long as enough workgroups are left
    int64_t span = tiles * rows / 1024;
    span = span < 1 ? 1 : (span > 8 ? 8 : span);
    const int64_t spans = ceil_div(tiles, span), grid = 1 + spans * rows;
    if (MG == 1 && p.T <= kRouteTokens && grid <= 2048) {
        moe_up_kernel<DT, MG, MG == 1><<<(unsigned)grid, 64 * kUpWaves, 0, stream>>>(p, (int)spans, (int)span, by_pair);
    } else {
        moe_route_kernel<<<(unsigned)p.T, 64, 0, stream>>>(p);
        moe_up_kernel<DT, MG, false><<<(unsigned)grid, 64 * kUpWaves, 0, stream>>>(p, (int)spans, (int)span, by_pair);
    }
    const unsigned cols = (unsigned)(p.H / 16);
    if constexpr (MG == 1) {
        if (p.T <= 16) {
            moe_down_kernel<DT, MG, 16, 16><<<cols, 1024, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
    if constexpr (MG < 4) {
        if (p.T <= 64) {
            moe_down_kernel<DT, MG, 64, 16><<<cols, 1024, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
    moe_down_kernel<DT, MG, 128, 8><<<cols, 512, 0, stream>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t moe_pieces(const Fp8MoeArgs& p, hipStream_t stream) {
    // pieces of 16 tokens multiplied at once: by the tokens that an expert has on average (one
    // that has more is read once per 16 MG of them)
    const int64_t mean16 = 16 * p.T * p.k / p.E;
    if (mean16 <= 12 * 16 || p.T <= 16) return moe_launch<DT, 1>(p, stream);
    if (mean16 <= 28 * 16 || p.T <= 32) return moe_launch<DT, 2>(p, stream);
    return moe_launch<DT, 4>(p, stream);
}

}  // namespace

hipError_t launch_fp8_moe(int dt, const Fp8MoeArgs& p, hipStream_t stream) {
    return dt == F16 ? moe_pieces<F16>(p, stream) : moe_pieces<BF16>(p, stream);
}

}  // namespace llmint8
