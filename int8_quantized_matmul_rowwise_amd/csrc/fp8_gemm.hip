// Products of e4m3 codes with power-of-two block scales:
//   Y[m,n] = RN_T( sum_g 2^(ea[m,g] + eb[n,g]) sum_{k in g} a[m,k] b[n,k] ),
// g over groups of 128 along K; ea per row, eb per row (n >> 0) or per 128 rows (n >> 7).
// The forward product, the input gradient (b: the transposed weight codes) and the weight
// gradient (both operands per row, the sum over the tokens) are all this product.
#include "fp8_common.hpp"
#include "launch.hpp"

namespace llmint8 {

namespace {

// One workgroup per 64 x 64 outputs, each wave 16 columns n by 64 rows m; operands from global
// memory straight into the matrix unit's registers (16x16x128: lane l holds row l % 16, bytes
// 32 (l / 16) .. + 31 of the group).  n is the instruction's row side, so a lane's four results
// are four neighbours along n of one row m.
template <int DT>
__global__ __launch_bounds__(256) void fp8_gemm_kernel(Fp8GemmArgs p) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int li = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 64 + 16 * w, m0 = (int64_t)blockIdx.y * 64;
    const int64_t n = n0 + li < p.N ? n0 + li : p.N - 1;
    const uint8_t* b = p.B + n * p.pitch + 32 * q;
    const uint8_t* sb = p.sb + (n >> p.bshift) * p.spitch;
    const uint8_t* a[4];
    const uint8_t* sa[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + 16 * j + li < p.M ? m0 + 16 * j + li : p.M - 1;
        a[j] = p.A + m * p.pitch + 32 * q;
        sa[j] = p.sa + m * p.spitch;
    }
    v4f acc[4] = {};
    for (int64_t g = 0; g < p.pitch / 128; ++g) {
        const v8i fb = *(const v8i*)(b + g * 128);
        const int eb = sb[g];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, *(const v8i*)(a[j] + g * 128), acc[j], 0, 0, 0,
                                                                      eb, 0, (int)sa[j][g]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + 16 * j + li;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (m < p.M && n0 + 4 * q + e < p.N) p.Y[m * p.N + n0 + 4 * q + e] = from_f32<DT>(acc[j][e]);
    }
}

}  // namespace

hipError_t launch_fp8_gemm(int dt, const Fp8GemmArgs& p, hipStream_t stream) {
    if (p.M == 0 || p.N == 0) return hipSuccess;
    const dim3 g((unsigned)ceil_div(p.N, 64), (unsigned)ceil_div(p.M, 64));
    if (dt == F16) fp8_gemm_kernel<F16><<<g, 256, 0, stream>>>(p);
    else fp8_gemm_kernel<BF16><<<g, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace llmint8
