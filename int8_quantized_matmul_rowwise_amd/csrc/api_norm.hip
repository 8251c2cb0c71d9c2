// C-ABI entry points of the root-mean-square norm (declared and documented in include/llmint8.h).
// Validation happens before anything is enqueued.
#include "api_common.hpp"
#include "launch.hpp"
#include "mxfp4_common.hpp"

using namespace llmint8;

namespace {

constexpr int64_t kMaxSide = (int64_t)1 << 22;

int check_norm(int64_t M, int64_t K, int dtype) {
    if (dtype != LLMINT8_F16 && dtype != LLMINT8_BF16) return LLMINT8_EINVAL;
    if (M < 0 || K < 0 || K % 16 != 0) return LLMINT8_EINVAL;
    if (M > kMaxSide || K > kMaxSide) return LLMINT8_ERANGE;
    return LLMINT8_OK;
}

bool eps_ok(float eps) { return eps > 0.0f && isfinite(eps); }
bool in_ok(const void* p) { return p && aligned(p, 16); }
bool out_ok(const void* p) { return !p || aligned(p, 16); }

}  // namespace

LLMINT8_API int64_t fp8_row_scale_pitch(int64_t rows) { return rows < 0 ? 0 : round_up(rows, 64); }

LLMINT8_API int rmsnorm_forward(const void* X, const void* residual, const void* weight, int64_t M, int64_t K, int dtype, float eps, void* H,
                                void* Y, int format, uint8_t* Yq, uint8_t* y_scale, void* stream) {
    int rc = check_norm(M, K, dtype);
    if (rc) return rc;
    if (!eps_ok(eps)) return LLMINT8_EINVAL;
    if (format != LLMINT8_CODES_NONE && format != LLMINT8_CODES_FP8_BLOCK && format != LLMINT8_CODES_MXFP4) return LLMINT8_EINVAL;
    if (M == 0 || K == 0) return LLMINT8_OK;
    const bool codes = format != LLMINT8_CODES_NONE, four = format == LLMINT8_CODES_MXFP4;
    if (!in_ok(X) || (residual && !aligned(residual, 16)) || !in_ok(weight) || !out_ok(H) || !out_ok(Y)) return LLMINT8_EINVAL;
    if (H && !residual) return LLMINT8_EINVAL;  // it would be X
    if (codes ? !in_ok(Yq) || !y_scale || !aligned(y_scale, 4) : Yq || y_scale) return LLMINT8_EINVAL;
    if (!H && !Y && !codes) return LLMINT8_OK;
    const size_t n = (size_t)M * (size_t)K * 2;
    // H may take the place of X or of the residual
    const Range r[] = {{H, n},
                       {Y, n},
                       {Yq, codes ? (size_t)M * (size_t)(four ? fp4_pitch(K) : fp8_pitch(K)) : 0},
                       {y_scale, codes ? (size_t)(four ? fp4_scale_bytes(M, K) : fp8_row_scale_bytes(M, K)) : 0},
                       {H == X ? nullptr : X, n},
                       {H == residual ? nullptr : residual, n},
                       {weight, (size_t)K * 2}};
    if (clash(r, 4, 7)) return LLMINT8_EINVAL;
    const NormPlan plan = rmsnorm_plan(M, K, format);
    if (log_call("rmsnorm_forward", M, K, 0, dtype, NAN, four ? "rmsnorm_mxfp4" : (codes ? "rmsnorm_fp8_block" : "rmsnorm")))
        fprintf(stderr, "[llmint8]   plan vectors=%d threads=%d\n", plan.vectors, plan.threads);
    return hip_status(stage("rmsnorm", [&] {
        const NormArgs a{(const uint16_t*)X, (const uint16_t*)residual, (const uint16_t*)weight, M, K, 1.0 / (double)K, eps, (uint16_t*)H, (uint16_t*)Y, format, Yq, y_scale};
        return launch_rmsnorm(dtype, a, plan, (hipStream_t)stream);
    }));
}

namespace {

struct NormBackwardLayout {
    NormBackwardPlan plan;
    size_t rows, total;
};

NormBackwardLayout backward_layout(int64_t M, int64_t K, bool dw) {
    NormBackwardLayout L{rmsnorm_backward_plan(M, K), 0, 0};
    if (!dw) return L;
    L.rows = align_up((size_t)L.plan.groups * (size_t)K * 4);
    L.total = align_up(L.rows + (L.plan.whole ? 0 : (size_t)M * 4));
    return L;
}

}  // namespace

LLMINT8_API size_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t K, int need_dw) {
    if (check_norm(M, K, LLMINT8_F16) || M == 0 || K == 0) return 0;
    return backward_layout(M, K, need_dw != 0).total;
}

LLMINT8_API int rmsnorm_backward(const void* dY, const void* H, const void* weight, const void* dH, int64_t M, int64_t K, int dtype, float eps,
                                 void* dX, void* dW, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_norm(M, K, dtype);
    if (rc) return rc;
    if (!eps_ok(eps)) return LLMINT8_EINVAL;
    if (K == 0) return LLMINT8_OK;
    hipStream_t st = (hipStream_t)stream;
    if (!out_ok(dW)) return LLMINT8_EINVAL;
    if (M == 0) {
        if (!dW) return LLMINT8_OK;
        log_call("rmsnorm_backward", M, K, 0, dtype, NAN, "empty sum");
        return hip_status(stage("fill_zero", [&] { return launch_fill_zero((float*)dW, K / 2, st); }));
    }
    if (!in_ok(dY) || !in_ok(H) || !in_ok(weight) || (dH && !aligned(dH, 16)) || !in_ok(dX)) return LLMINT8_EINVAL;
    const NormBackwardLayout L = backward_layout(M, K, dW != nullptr);
    if (L.total > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total)) return LLMINT8_EWORKSPACE;
    const size_t n = (size_t)M * (size_t)K * 2;
    const Range r[] = {{dX, n}, {dW, (size_t)K * 2}, {workspace, L.total}, {dY, n}, {H, n}, {weight, (size_t)K * 2}, {dH, n}};
    if (clash(r, 3, 7)) return LLMINT8_EINVAL;
    if (log_call("rmsnorm_backward", M, K, 0, dtype, NAN, L.plan.whole ? "rmsnorm_backward" : "rmsnorm_backward_long"))
        fprintf(stderr, "[llmint8]   plan vectors=%d threads=%d ahead=%d side=%d\n", L.plan.vectors, L.plan.row_threads, (int)L.plan.ahead,
                L.plan.whole ? L.plan.threads / L.plan.row_threads : 0);
    return hip_status(stage("rmsnorm_backward", [&] {
        uint8_t* ws = (uint8_t*)workspace;
        const NormBackwardArgs a{(const uint16_t*)dY, (const uint16_t*)H, (const uint16_t*)weight, (const uint16_t*)dH, M, K, 1.0 / (double)K, eps, (uint16_t*)dX,
                                 (uint16_t*)dW, (float*)ws, dW && !L.plan.whole ? (float*)(ws + L.rows) : nullptr};
        return launch_rmsnorm_backward(dtype, a, L.plan, st);
    }));
}
