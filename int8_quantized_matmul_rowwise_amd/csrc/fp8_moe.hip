// A mixture-of-experts layer for few tokens, its weights e4m3 codes with a power-of-two scale
// per 128 x 128 block, its activations 16-bit.  Per token x (a row of X) with logits l:
//   experts e_0, e_1, ...: the top_k largest logits (ties to the lowest index; -inf and NaN are
//     never taken, +inf counts as the largest finite number);
//   p_j = exp(l[e_j] - l[e_0]) / Z, Z the sum of exp(l - l[e_0]) over the chosen experts
//     (renormalize) or over all;
//   [g; u] = W13hat_e x (2I values), h = RN_T(silu(g) u), y = RN_T(sum_j p_j W2hat_e h).
#include "fp8_common.hpp"
#include "launch.hpp"

namespace llmint8 {

namespace {

__device__ __forceinline__ float usable_logit(float l) {  // NaN as -inf, +inf as the largest number
    return l != l ? -__builtin_inff() : fminf(l, 3.4028234663852886e38f);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// one wave per token
__global__ __launch_bounds__(64) void moe_route_kernel(const float* __restrict__ logits, int E, int k, int renormalize,
                                                       int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int t = blockIdx.x, lane = threadIdx.x;
    const float* l = logits + (int64_t)t * E;
    float prev = __builtin_inff(), top = 0.0f, chosen = 0.0f, z = 0.0f;
    int prev_e = -1;
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
        const bool open = best > -__builtin_inff();
        if (j == 0) top = best;
        const float x = open ? expf(best - top) : 0.0f;
        chosen += x;
        if (lane == 0) {
            ids[t * k + j] = open ? at : -1;
            weights[t * k + j] = x;
        }
        if (open) {
            prev = best;
            prev_e = at;
        } else {
            prev = -__builtin_inff();
        }
    }
    if (renormalize) {
        z = chosen;
    } else {
        for (int e = lane; e < E; e += kWave) z += expf(usable_logit(l[e]) - top);
        z = wave_sum(z);
    }
    if (lane == 0 && ids[t * k] >= 0)
        for (int j = 0; j < k; ++j) weights[t * k + j] = weights[t * k + j] / z;
}

__device__ __forceinline__ float code_value(uint8_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }

// sum_k code[k] s[k / 128] x[k], lanes over k
template <class F>
__device__ __forceinline__ float row_dot(const uint8_t* code, const uint8_t* s, int64_t K, F&& x) {
    float sum = 0.0f;
    for (int64_t k = threadIdx.x & 63; k < K; k += kWave)
        sum = __fadd_rn(sum, __fmul_rn(__fmul_rn(code_value(code[k]), e8m0_value(s[k >> 7])), x(k)));
    return wave_sum(sum);
}

// one wave per (pair of token and choice, column of I)
template <int DT>
__global__ __launch_bounds__(256) void moe_up_kernel(Fp8MoeArgs p) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), pair = blockIdx.y;
    const int e = p.ids[pair];
    if (e < 0 || i >= p.I) return;
    const uint16_t* x = p.X + (pair / p.k) * p.H;
    const int64_t hp = fp8_pitch(p.H), hsp = fp8_scale_pitch_of(p.H);
    const uint8_t* W = p.W13 + (int64_t)e * 2 * p.I * hp;
    const uint8_t* S = p.s13 + (int64_t)e * ceil_div(2 * p.I, 128) * hsp;
    auto xv = [&](int64_t k) { return to_f32<DT>(x[k]); };
    const float g = row_dot(W + i * hp, S + (i >> 7) * hsp, p.H, xv);
    const float u = row_dot(W + (p.I + i) * hp, S + ((p.I + i) >> 7) * hsp, p.H, xv);
    if ((threadIdx.x & 63) == 0) p.h[pair * p.I + i] = from_f32<DT>(g / (1.0f + expf(-g)) * u);
}

// one wave per (token, column of H)
template <int DT>
__global__ __launch_bounds__(256) void moe_down_kernel(Fp8MoeArgs p) {
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), t = blockIdx.y;
    if (n >= p.H) return;
    const int64_t ip = fp8_pitch(p.I), isp = fp8_scale_pitch_of(p.I);
    float y = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int64_t pair = t * p.k + j;
        const int e = p.ids[pair];
        if (e < 0) continue;
        const uint16_t* h = p.h + pair * p.I;
        const float d = row_dot(p.W2 + ((int64_t)e * p.H + n) * ip, p.s2 + ((int64_t)e * ceil_div(p.H, 128) + (n >> 7)) * isp,
                                p.I, [&](int64_t k) { return to_f32<DT>(h[k]); });
        y = __fadd_rn(y, __fmul_rn(p.weights[pair], d));
    }
    if ((threadIdx.x & 63) == 0) p.Y[t * p.H + n] = from_f32<DT>(y);
}

template <int DT>
hipError_t moe_launch(const Fp8MoeArgs& p, hipStream_t stream) {
    moe_route_kernel<<<(unsigned)p.T, 64, 0, stream>>>(p.logits, (int)p.E, p.k, p.renormalize, p.ids, p.weights);
    if (p.I > 0) moe_up_kernel<DT><<<dim3((unsigned)ceil_div(p.I, 4), (unsigned)(p.T * p.k)), 256, 0, stream>>>(p);
    moe_down_kernel<DT><<<dim3((unsigned)ceil_div(p.H, 4), (unsigned)p.T), 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_moe(int dt, const Fp8MoeArgs& p, hipStream_t stream) {
    return dt == F16 ? moe_launch<F16>(p, stream) : moe_launch<BF16>(p, stream);
}

}  // namespace llmint8
