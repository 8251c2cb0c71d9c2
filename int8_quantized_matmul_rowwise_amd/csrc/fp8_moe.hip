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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// The experts and weights of one token, by one wave; lane j < k returns choice j.
__device__ __forceinline__ void route_token(const float* __restrict__ l, int E, int k, int renormalize, int& id, float& p) {
    const int lane = threadIdx.x & 63;
    float prev = __builtin_inff(), top = 0.0f, chosen = 0.0f;
    int prev_e = -1;
    id = -1;
    p = 0.0f;
    for (int j = 0; j < k; ++j) {
        // the best of those after (prev, prev_e) in the order (value descending, index ascending)
        float best = -__builtin_inff();
        int at = 0x7fffffff;
        for (int e = lane; e < E; e += kWave) {
            const float v = usable_logit(l[e]);
            if ((v < prev || (v == prev && e > prev_e)) && v > best) {
                best = v;
                at = e;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const float v = __shfl_xor(best, off, kWave);
            const int e = __shfl_xor(at, off, kWave);
            if (v > best || (v == best && e < at)) {
                best = v;
                at = e;
            }
        }
        if (!(best > -__builtin_inff())) break;  // the same in every lane
        if (j == 0) top = best;
        const float x = expf(best - top);
        chosen += x;
        if (lane == j) {
            id = at;
            p = x;
        }
        prev = best;
        prev_e = at;
    }
    float z = chosen;
    if (!renormalize) {
        z = 0.0f;
        for (int e = lane; e < E; e += kWave) z += expf(usable_logit(l[e]) - top);
        z = wave_sum(z);
    }
    if (id >= 0) p /= z;
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

// ---- gate, up and SwiGLU: a workgroup takes 16 columns of I of one expert (16 gate rows and 16
// up rows), its waves split the groups of H.  Workgroup 0 writes the table.  by_pair: workgroups
// go by pair of token and choice (each expert at its first pair), else by expert.
template <int DT, int MG, bool ROUTE>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(Fp8MoeArgs p, int tiles, int by_pair) {
    constexpr int WV = kUpWaves, U = MG == 1 ? 2 : 1;
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
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        build_table(ids, T, E, k, 16 * MG, p.table, p.pairs, sh.t.mask, sh.t.first);
        return;
    }
    const int y = (int)(blockIdx.x - 1) / tiles, tile = (int)(blockIdx.x - 1) % tiles;
    int e = y;
    if (by_pair) {
        e = ids[y];
        if (e < 0) return;
    }
    // the expert's tokens, ascending: list[place] = token * k + choice
    if (tid == 0) dup = 0;
    __syncthreads();
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
    const int i0 = 16 * tile, ng = (int)(hp / 128);
    const uint8_t* W = p.W13 + (int64_t)e * 2 * p.I * hp;
    const uint8_t* S = p.s13 + (int64_t)e * ceil_div(2 * p.I, 128) * hsp;
    const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(W + (int64_t)i0 * hp, 16 * hp);
    const __amdgpu_buffer_rsrc_t ru = buffer_rsrc(W + (p.I + i0) * hp, 16 * hp);
    const uint8_t* sg = S + (int64_t)(i0 >> 7) * hsp;
    const uint8_t* su = S + ((p.I + i0) >> 7) * hsp;  // I is a multiple of 16: one block
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
        auto load = [&](int g, Group& r) LLMINT8_MOE_INLINE {
            const uint32_t far = g < ng ? 0u : kFar;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t off = (w_off + (uint32_t)(g * 128 + 16 * h)) | far;
                r.g[h] = load16(rg, off);
                r.u[h] = load16(ru, off);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t out = g * 128 + 32 * q + 8 * i < p.H ? far : kFar;  // past H: the next row's
#pragma unroll
                for (int j = 0; j < MG; ++j)
                    r.x[j][i] = load16(rx, (x_off[j] + (uint32_t)(g * 128 + 8 * i) * 2) | out);
            }
            r.eg = g < ng ? e8m0_value(sg[g]) : 0.0f;
            r.eu = g < ng ? e8m0_value(su[g]) : 0.0f;
        };
        v4f ag[MG] = {}, au[MG] = {};
        auto multiply = [&](const Group& r) LLMINT8_MOE_INLINE {
            group_product<DT, MG>(r.g, r.eg, r.x, ag);
            group_product<DT, MG>(r.u, r.eu, r.x, au);
        };
        Group a[U], b[U];
        int g = w;
#pragma unroll
        for (int u = 0; u < U; ++u) load(g + u * WV, a[u]);
        while (g < ng) {
            g += U * WV;
#pragma unroll
            for (int u = 0; u < U; ++u) load(g + u * WV, b[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) multiply(a[u]);
            if (g >= ng) break;
            g += U * WV;
#pragma unroll
            for (int u = 0; u < U; ++u) load(g + u * WV, a[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) multiply(b[u]);
        }
        mfma_settle();
#pragma unroll
        for (int j = 0; j < MG; ++j) {
            sh.red[w][j][lane] = ag[j];
            sh.red[w][MG + j][lane] = au[j];
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
                *(u32x2*)(p.h + (int64_t)list[i] * p.I + i0 + 4 * q) = v;
            }
        }
        __syncthreads();
    }
}

// ---- down and the weighted sum: a workgroup takes 16 columns of H of all entries.  Their groups
// of I, entry after entry, are split evenly over the waves; a wave ends an entry (or its share of
// it) by adding p times its sums to its own rows of token sums in LDS.
template <int DT, int MG, int WV>
__global__ __launch_bounds__(64 * WV) void moe_down_kernel(Fp8MoeArgs p) {
    extern __shared__ v4f ysum[];  // [WV][T][4] quads: a wave's sums of 16 columns per token
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, q = lane >> 4;
    const int T = (int)p.T, k = p.k;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t ip = fp8_pitch(p.I), isp = fp8_scale_pitch_of(p.I);
    const int ng = (int)(ip / 128);
    const int entries = __builtin_amdgcn_readfirstlane(p.table[0]);
    for (int i = tid; i < WV * T * 4; i += 64 * WV) ysum[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();
    const int64_t total = (int64_t)entries * ng;
    const int64_t from = total * w / WV, to = total * (w + 1) / WV;
    const uint32_t w_off = (uint32_t)(li * ip + 32 * q);
    const __amdgpu_buffer_rsrc_t rh = buffer_rsrc(p.h, p.T * k * p.I * 2);
    v4f* mine = ysum + (int64_t)w * T * 4;
    for (int64_t at = from; at < to;) {
        const int entry = __builtin_amdgcn_readfirstlane((int)(at / ng));
        const int g0 = (int)(at - (int64_t)entry * ng);
        const int g1 = to - at < ng - g0 ? g0 + (int)(to - at) : ng;
        const int e = __builtin_amdgcn_readfirstlane(p.table[1 + 3 * entry]);
        const int off = __builtin_amdgcn_readfirstlane(p.table[2 + 3 * entry]);
        const int count = __builtin_amdgcn_readfirstlane(p.table[3 + 3 * entry]);
        uint32_t h_off[MG];
        int token[MG];
        float pt[MG];
#pragma unroll
        for (int j = 0; j < MG; ++j) {
            const int i = 16 * j + li;
            const int pair = i < count ? p.pairs[off + i] : -1;
            token[j] = pair >= 0 ? pair / k : -1;
            pt[j] = pair >= 0 ? p.weights[pair] : 0.0f;
            h_off[j] = pair >= 0 ? (uint32_t)(pair * p.I + 32 * q) * 2 : kFar;
        }
        const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(p.W2 + ((int64_t)e * p.H + n0) * ip, 16 * ip);
        const uint8_t* s = p.s2 + ((int64_t)e * ceil_div(p.H, 128) + (n0 >> 7)) * isp;
        struct Group {
            u32x4 w[2], x[MG][4];
            float s;
        };
        auto load = [&](int g, Group& r) LLMINT8_MOE_INLINE {
            const uint32_t far = g < g1 ? 0u : kFar;
#pragma unroll
            for (int h = 0; h < 2; ++h) r.w[h] = load16(rw, (w_off + (uint32_t)(g * 128 + 16 * h)) | far);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t out = g * 128 + 32 * q + 8 * i < p.I ? far : kFar;
#pragma unroll
                for (int j = 0; j < MG; ++j)
                    r.x[j][i] = load16(rh, (h_off[j] + (uint32_t)(g * 128 + 8 * i) * 2) | out);
            }
            r.s = g < g1 ? e8m0_value(s[g]) : 0.0f;
        };
        constexpr int U = MG <= 2 ? 2 : 1;
        v4f acc[MG] = {};
        Group a[U], b[U];
        int g = g0;
#pragma unroll
        for (int u = 0; u < U; ++u) load(g + u, a[u]);
        while (g < g1) {
            g += U;
#pragma unroll
            for (int u = 0; u < U; ++u) load(g + u, b[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) group_product<DT, MG>(a[u].w, a[u].s, a[u].x, acc);
            if (g >= g1) break;
            g += U;
#pragma unroll
            for (int u = 0; u < U; ++u) load(g + u, a[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) group_product<DT, MG>(b[u].w, b[u].s, b[u].x, acc);
        }
        mfma_settle();
#pragma unroll
        for (int j = 0; j < MG; ++j)
            if (token[j] >= 0) {
                v4f y = mine[token[j] * 4 + q];
#pragma unroll
                for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(pt[j], acc[j][r], y[r]);
                mine[token[j] * 4 + q] = y;
            }
        at += g1 - g0;
    }
    __syncthreads();
    for (int i = tid; i < T * 4; i += 64 * WV) {
        v4f y = ysum[i];
#pragma unroll
        for (int v = 1; v < WV; ++v) y += ysum[v * T * 4 + i];
        u32x2 o;
        o[0] = (uint32_t)from_f32<DT>(y[0]) | ((uint32_t)from_f32<DT>(y[1]) << 16);
        o[1] = (uint32_t)from_f32<DT>(y[2]) | ((uint32_t)from_f32<DT>(y[3]) << 16);
        *(u32x2*)(p.Y + (int64_t)(i >> 2) * p.H + n0 + 4 * (i & 3)) = o;
    }
}

template <int DT, int MG>
hipError_t moe_launch(const Fp8MoeArgs& p, hipStream_t stream) {
    const bool route = p.T <= kRouteTokens;
    const int by_pair = p.T * p.k < p.E;
    const int tiles = (int)(p.I / 16);
    const int64_t grid = 1 + (int64_t)tiles * (by_pair ? p.T * p.k : p.E);
    if (!route) moe_route_kernel<<<(unsigned)p.T, 64, 0, stream>>>(p);
    if (route && MG == 1) moe_up_kernel<DT, MG, MG == 1><<<(unsigned)grid, 64 * kUpWaves, 0, stream>>>(p, tiles, by_pair);
    else moe_up_kernel<DT, MG, false><<<(unsigned)grid, 64 * kUpWaves, 0, stream>>>(p, tiles, by_pair);
    constexpr int WV = 8;
    moe_down_kernel<DT, MG, WV><<<(unsigned)(p.H / 16), 64 * WV, WV * p.T * 64, stream>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t moe_pieces(const Fp8MoeArgs& p, hipStream_t stream) {
    if (p.T <= 16) return moe_launch<DT, 1>(p, stream);
    if (p.T <= 32) return moe_launch<DT, 2>(p, stream);
    return moe_launch<DT, 4>(p, stream);
}

}  // namespace

hipError_t launch_fp8_moe(int dt, const Fp8MoeArgs& p, hipStream_t stream) {
    return dt == F16 ? moe_pieces<F16>(p, stream) : moe_pieces<BF16>(p, stream);
}

}  // namespace llmint8
