// C-ABI entry points of the e4m3 block-scaled operators (declared and documented in
// include/llmint8.h).  Validation happens before anything is enqueued.
#include <math.h>

#include "api_common.hpp"
#include "common.hpp"
#include "fp8_common.hpp"
#include "launch.hpp"

using namespace llmint8;

namespace {

// A row of codes is a sum's operand: tiles of 256 rows are addressed with 32-bit offsets.
constexpr int64_t kMaxSum = (int64_t)1 << 22;

int check_fp8_shape(int64_t M, int64_t K, int64_t N, int dtype) {
    if (dtype != LLMINT8_F16 && dtype != LLMINT8_BF16) return LLMINT8_EINVAL;
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return LLMINT8_EINVAL;
    if (K % 16 != 0 || N % 8 != 0) return LLMINT8_EINVAL;
    if (K > kMaxSum || M > kMaxSum) return LLMINT8_ERANGE;
    if (ceil_div(M, 128) * ceil_div(N, 128) > kMaxDim) return LLMINT8_ERANGE;  // the product's grid
    return LLMINT8_OK;
}

size_t code_bytes(int64_t rows, int64_t sum) { return (size_t)rows * (size_t)fp8_pitch(sum); }
size_t scale_bytes(int64_t rows, int64_t sum) { return (size_t)rows * (size_t)fp8_scale_pitch_of(sum); }

struct Range {
    const void* p;
    size_t n;
};

// whether any of the outputs overlaps another range (outputs first, then inputs)
bool clash(const Range* r, int outputs, int all) {
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < all; ++j)
            if (overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
    return false;
}

}  // namespace

LLMINT8_API int64_t fp8_code_pitch(int64_t n) { return n < 0 ? 0 : fp8_pitch(n); }
LLMINT8_API int64_t fp8_scale_pitch(int64_t n) { return n < 0 ? 0 : fp8_scale_pitch_of(n); }

LLMINT8_API int fp8_quantize_weight_block(const void* W, int64_t K, int64_t N, int dtype, uint8_t* Wq, uint8_t* w_scale,
                                          uint8_t* WqT, uint8_t* wT_scale, void* stream) {
    int rc = check_fp8_shape(0, K, N, dtype);
    if (rc) return rc;
    if (N == 0 || K == 0) return LLMINT8_OK;
    if ((WqT != nullptr) != (wT_scale != nullptr)) return LLMINT8_EINVAL;
    if (N > kMaxSum) return LLMINT8_ERANGE;
    if (!W || !Wq || !w_scale || !aligned(W, 16) || !aligned(Wq, 16) || !aligned(w_scale, 4)) return LLMINT8_EINVAL;
    if (WqT && (!aligned(WqT, 16) || !aligned(wT_scale, 4))) return LLMINT8_EINVAL;
    const Range r[] = {{Wq, code_bytes(N, K)},
                       {w_scale, scale_bytes(ceil_div(N, 128), K)},
                       {WqT, WqT ? code_bytes(K, N) : 0},
                       {wT_scale, WqT ? scale_bytes(ceil_div(K, 128), N) : 0},
                       {W, (size_t)K * (size_t)N * 2}};
    if (clash(r, 4, 5)) return LLMINT8_EINVAL;
    log_call("fp8_quantize_weight_block", 0, K, N, dtype, NAN, WqT ? "fp8_weight_both" : "fp8_weight");
    return hip_status(stage("fp8_weight", [&] { return launch_fp8_weight(dtype, W, K, N, Wq, w_scale, WqT, wT_scale, (hipStream_t)stream); }));
}

// ---- Y = X W

namespace {

struct Fp8Layout {
    Fp8Plan plan;
    size_t xq, s_x, counters, partial, total;
};

Fp8Layout fp8_layout(int64_t M, int64_t K, int64_t N) {
    Fp8Layout L;
    L.plan = fp8_plan(M, N, ceil_div(K, 128), true, false);
    const bool fused = L.plan.kind == Fp8Plan::kFused;
    L.xq = 0;
    L.s_x = align_up(fused ? 0 : code_bytes(M, K));
    L.counters = align_up(L.s_x + (fused ? 0 : (size_t)fp8_row_scale_bytes(M, K)));
    L.partial = align_up(L.counters + (L.plan.split > 1 ? (size_t)L.plan.tiles * 4 : 0));
    L.total = align_up(L.partial + (size_t)L.plan.partial_bytes);
    return L;
}

const char* plan_name(const Fp8Plan& p) {
    switch (p.kind) {
        case Fp8Plan::kTile256: return p.split > 1 ? "fp8_tile256_split" : "fp8_tile256";
        case Fp8Plan::kTile128: return "fp8_tile128";
        case Fp8Plan::kSingle: return p.split > 1 ? "fp8_single_split" : "fp8_single";
        case Fp8Plan::kSmall: return p.split > 1 ? "fp8_small_split" : "fp8_small";
        default: return "fp8_small_fused";
    }
}

}  // namespace

LLMINT8_API size_t fp8_matmul_block_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    if (check_fp8_shape(M, K, N, LLMINT8_F16) || M == 0 || N == 0 || K == 0) return 0;
    return fp8_layout(M, K, N).total;
}

LLMINT8_API int fp8_matmul_block(const void* X, int64_t M, int64_t K, int dtype, const uint8_t* Wq,
                                 const uint8_t* w_scale, int64_t N, void* Y, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    int rc = check_fp8_shape(M, K, N, dtype);
    if (rc) return rc;
    if (M == 0 || N == 0) return LLMINT8_OK;
    if (!Y || !aligned(Y, 16)) return LLMINT8_EINVAL;
    hipStream_t st = (hipStream_t)stream;
    if (K == 0) {
        log_call("fp8_matmul_block", M, K, N, dtype, NAN, "empty sum");
        return hip_status(stage("fill_zero", [&] { return launch_fill_zero((float*)Y, M * N / 2, st); }));
    }
    if (!X || !aligned(X, 16) || !Wq || !aligned(Wq, 16) || !w_scale || !aligned(w_scale, 4)) return LLMINT8_EINVAL;
    const Fp8Layout L = fp8_layout(M, K, N);
    if (L.total > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total)) return LLMINT8_EWORKSPACE;
    const Range r[] = {{Y, (size_t)M * (size_t)N * 2},
                       {workspace, L.total},
                       {X, (size_t)M * (size_t)K * 2},
                       {Wq, code_bytes(N, K)},
                       {w_scale, scale_bytes(ceil_div(N, 128), K)}};
    if (clash(r, 2, 5)) return LLMINT8_EINVAL;
    log_call("fp8_matmul_block", M, K, N, dtype, NAN, plan_name(L.plan));
    uint8_t* ws = (uint8_t*)workspace;
    int32_t* counters = L.plan.split > 1 ? (int32_t*)(ws + L.counters) : nullptr;
    hipError_t e = hipSuccess;
    if (L.plan.kind != Fp8Plan::kFused)
        e = stage("fp8_rows", [&] {
            return launch_fp8_rows(dtype, X, M, K, ws + L.xq, ws + L.s_x, counters, counters ? L.plan.tiles : 0, st);
        });
    if (e == hipSuccess)
        e = stage("fp8_gemm", [&] {
            const Fp8GemmArgs a{ws + L.xq, Wq, M, N, fp8_pitch(K), ws + L.s_x, w_scale, fp8_scale_pitch_of(K), (uint16_t*)Y,
                                (const uint16_t*)X, K, counters, (float*)(ws + L.partial)};
            return launch_fp8_gemm(dtype, a, L.plan, st);
        });
    return hip_status(e);
}

// ---- dX = dY W^T, dW = X^T dY

namespace {

struct Fp8BackwardLayout {
    Fp8Plan dx, dw;
    size_t dyq, s_dy, dyt, s_dyt, xt, s_xt, counters, partial, total;
};

Fp8BackwardLayout fp8_backward_layout(int64_t M, int64_t K, int64_t N, bool dx, bool dw) {
    Fp8BackwardLayout L{};
    if (dx) L.dx = fp8_plan(M, K, ceil_div(N, 128), false, false);
    if (dw) L.dw = fp8_plan(K, N, ceil_div(M, 128), false, true);
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off = align_up(off + n);
        return at;
    };
    L.dyq = take(dx ? code_bytes(M, N) : 0);
    L.s_dy = take(dx ? (size_t)fp8_row_scale_bytes(M, N) : 0);
    L.dyt = take(dw ? code_bytes(N, M) : 0);
    L.s_dyt = take(dw ? (size_t)fp8_row_scale_bytes(N, M) : 0);
    L.xt = take(dw ? code_bytes(K, M) : 0);
    L.s_xt = take(dw ? (size_t)fp8_row_scale_bytes(K, M) : 0);
    // one product after the other: the partial sums share their place
    L.counters = take((L.dx.split > 1 ? (size_t)L.dx.tiles * 4 : 0) + (L.dw.split > 1 ? (size_t)L.dw.tiles * 4 : 0));
    const size_t px = (size_t)L.dx.partial_bytes, pw = (size_t)L.dw.partial_bytes;
    L.partial = take(px > pw ? px : pw);
    L.total = off;
    return L;
}

}  // namespace

LLMINT8_API size_t fp8_matmul_block_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, int need_dx, int need_dw) {
    if (check_fp8_shape(M, K, N, LLMINT8_F16) || M > kMaxSum || N > kMaxSum || M == 0 || K == 0 || N == 0) return 0;
    return fp8_backward_layout(M, K, N, need_dx != 0, need_dw != 0).total;
}

LLMINT8_API int fp8_matmul_block_backward(const void* dY, const void* X, int64_t M, int64_t K, int64_t N, int dtype,
                                          const uint8_t* WqT, const uint8_t* wT_scale, void* dX, void* dW,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_fp8_shape(M, K, N, dtype);
    if (rc) return rc;
    const bool dx = dX != nullptr, dw = dW != nullptr;
    if (M > kMaxSum || N > kMaxSum) return LLMINT8_ERANGE;
    if (!dx && !dw) return LLMINT8_OK;
    const bool out_x = dx && M > 0 && K > 0, out_w = dw && K > 0 && N > 0;
    if (!out_x && !out_w) return LLMINT8_OK;
    if ((out_x && !aligned(dX, 16)) || (out_w && !aligned(dW, 16))) return LLMINT8_EINVAL;
    const bool sum_x = out_x && N > 0, sum_w = out_w && M > 0;  // else the empty sum
    if ((sum_x || sum_w) && (!dY || !aligned(dY, 16))) return LLMINT8_EINVAL;
    if (sum_w && (!X || !aligned(X, 16))) return LLMINT8_EINVAL;
    if (sum_x && (!WqT || !aligned(WqT, 16) || !wT_scale || !aligned(wT_scale, 4))) return LLMINT8_EINVAL;
    const Fp8BackwardLayout L = fp8_backward_layout(M, K, N, sum_x, sum_w);
    if ((sum_x || sum_w) && (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total)) return LLMINT8_EWORKSPACE;
    const Range r[] = {{dX, out_x ? (size_t)M * (size_t)K * 2 : 0},
                       {dW, out_w ? (size_t)K * (size_t)N * 2 : 0},
                       {workspace, sum_x || sum_w ? L.total : 0},
                       {dY, (size_t)M * (size_t)N * 2},
                       {X, sum_w ? (size_t)M * (size_t)K * 2 : 0},
                       {WqT, sum_x ? code_bytes(K, N) : 0},
                       {wT_scale, sum_x ? scale_bytes(ceil_div(K, 128), N) : 0}};
    if (clash(r, 3, 7)) return LLMINT8_EINVAL;
    log_call("fp8_matmul_block_backward", M, K, N, dtype, NAN, dx ? (dw ? "fp8_dx_dw" : "fp8_dx") : "fp8_dw");
    hipStream_t st = (hipStream_t)stream;
    uint8_t* ws = (uint8_t*)workspace;
    int32_t* counters = (int32_t*)(ws + L.counters);
    const int64_t n_dx = L.dx.split > 1 ? L.dx.tiles : 0, n_dw = L.dw.split > 1 ? L.dw.tiles : 0;
    float* partial = (float*)(ws + L.partial);
    hipError_t e = hipSuccess;
    if (sum_w)
        e = stage("fp8_cols", [&] {
            return launch_fp8_cols(dtype, dY, X, M, N, K, ws + L.dyt, ws + L.s_dyt, sum_x ? ws + L.dyq : nullptr,
                                   sum_x ? ws + L.s_dy : nullptr, ws + L.xt, ws + L.s_xt, counters, n_dx + n_dw, st);
        });
    else if (sum_x)
        e = stage("fp8_rows", [&] { return launch_fp8_rows(dtype, dY, M, N, ws + L.dyq, ws + L.s_dy, counters, n_dx, st); });
    if (e == hipSuccess && out_x)
        e = sum_x ? stage("fp8_gemm_dx", [&] {
                        const Fp8GemmArgs a{ws + L.dyq, WqT, M, K, fp8_pitch(N), ws + L.s_dy, wT_scale, fp8_scale_pitch_of(N), (uint16_t*)dX,
                                            nullptr, 0, counters, partial};
                        return launch_fp8_gemm(dtype, a, L.dx, st);
                    })
                  : stage("fill_zero", [&] { return launch_fill_zero((float*)dX, M * K / 2, st); });
    if (e == hipSuccess && out_w)
        e = sum_w ? stage("fp8_gemm_dw", [&] {
                        const Fp8GemmArgs a{ws + L.xt, ws + L.dyt, K, N, fp8_pitch(M), ws + L.s_xt, ws + L.s_dyt, 0, (uint16_t*)dW,
                                            nullptr, 0, counters + n_dx, partial};
                        return launch_fp8_gemm(dtype, a, L.dw, st);
                    })
                  : stage("fill_zero", [&] { return launch_fill_zero((float*)dW, K * N / 2, st); });
    return hip_status(e);
}

// ---- mixture-of-experts layer for few tokens

namespace {

constexpr int64_t kMoeMaxTokens = 128, kMoeMaxExperts = 1024, kMoeMaxTopK = 16;

int check_moe(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
    if (T < 0 || H < 0 || I < 0 || E < 1 || k < 1 || k > E) return LLMINT8_EINVAL;
    if (H % 16 != 0 || I % 16 != 0) return LLMINT8_EINVAL;
    if (T > kMoeMaxTokens || E > kMoeMaxExperts || k > kMoeMaxTopK) return LLMINT8_ERANGE;
    if (H > kMaxSum || I > kMaxSum / 2 || T * k * fp8_pitch(I) >= (int64_t)1 << 30) return LLMINT8_ERANGE;
    return LLMINT8_OK;
}

const char* moe_plan_name(const Fp8MoePlan& p) {  // the form of the first launch, then of the second
    static const char* const names[3][3][2] = {
        {{"fp8_moe_light", "fp8_moe_light_split"}, {"fp8_moe_light_wide", "fp8_moe_light_wide_split"}, {"fp8_moe_light_many", "fp8_moe_light_many_split"}},
        {{"fp8_moe_wide_light", "fp8_moe_wide_light_split"}, {"fp8_moe_wide", "fp8_moe_wide_split"}, {"fp8_moe_wide_many", "fp8_moe_wide_many_split"}},
        {{"fp8_moe_many_light", "fp8_moe_many_light_split"}, {"fp8_moe_many_wide", "fp8_moe_many_wide_split"}, {"fp8_moe_many", "fp8_moe_many_split"}}};
    return names[p.up][p.down][p.parts > 1];
}

struct MoeLayout {
    Fp8MoePlan plan;
    size_t h, table, pairs, counters, partial, total;
};

MoeLayout moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
    MoeLayout L;
    L.plan = fp8_moe_plan(T, H, I, E, k);
    const size_t n = (size_t)T * (size_t)k;
    L.h = 0;
    L.table = align_up(n * (size_t)fp8_pitch(I) * 2);
    L.pairs = align_up(L.table + (1 + 3 * n) * 4);
    L.counters = align_up(L.pairs + n * 4);
    L.partial = align_up(L.counters + (L.plan.parts > 1 ? (size_t)L.plan.blocks * 4 : 0));
    L.total = align_up(L.partial + (size_t)L.plan.partial_bytes);
    return L;
}

}  // namespace

LLMINT8_API size_t fp8_moe_block_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    if (check_moe(T, H, I, E, top_k)) return 0;
    return moe_layout(T, H, I, E, top_k).total;
}

LLMINT8_API int fp8_moe_block(const void* X, int64_t T, int64_t H, int dtype, const float* logits, int64_t E,
                              int64_t top_k, int renormalize, const uint8_t* W13q, const uint8_t* w13_scale,
                              const uint8_t* W2q, const uint8_t* w2_scale, int64_t I, void* Y, int32_t* topk_ids,
                              float* topk_weights, void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != LLMINT8_F16 && dtype != LLMINT8_BF16) return LLMINT8_EINVAL;
    int rc = check_moe(T, H, I, E, top_k);
    if (rc) return rc;
    if (T == 0 || H == 0) return LLMINT8_OK;
    if (!logits || !aligned(logits, 4) || !topk_ids || !aligned(topk_ids, 4) || !topk_weights || !aligned(topk_weights, 4))
        return LLMINT8_EINVAL;
    if (!X || !aligned(X, 16) || !Y || !aligned(Y, 16)) return LLMINT8_EINVAL;
    if (I > 0 && (!W13q || !aligned(W13q, 16) || !w13_scale || !aligned(w13_scale, 4) || !W2q || !aligned(W2q, 16) ||
                  !w2_scale || !aligned(w2_scale, 4)))
        return LLMINT8_EINVAL;
    const MoeLayout L = moe_layout(T, H, I, E, top_k);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total) return LLMINT8_EWORKSPACE;
    const size_t e = (size_t)E, pairs = (size_t)T * (size_t)top_k;
    const Range r[] = {{Y, (size_t)T * (size_t)H * 2},
                       {topk_ids, pairs * 4},
                       {topk_weights, pairs * 4},
                       {workspace, L.total},
                       {X, (size_t)T * (size_t)H * 2},
                       {logits, (size_t)T * e * 4},
                       {W13q, e * code_bytes(2 * I, H)},
                       {w13_scale, e * scale_bytes(ceil_div(2 * I, 128), H)},
                       {W2q, e * code_bytes(H, I)},
                       {w2_scale, e * scale_bytes(ceil_div(H, 128), I)}};
    if (clash(r, 4, 10)) return LLMINT8_EINVAL;
    log_call("fp8_moe_block", T, H, I, dtype, NAN, moe_plan_name(L.plan));
    uint8_t* ws = (uint8_t*)workspace;
    const Fp8MoeArgs a{(const uint16_t*)X, T, H, logits, E, (int)top_k, renormalize != 0, W13q, w13_scale, W2q, w2_scale,
                       I, (uint16_t*)Y, topk_ids, topk_weights, (uint16_t*)(ws + L.h), (int32_t*)(ws + L.table),
                       (int32_t*)(ws + L.pairs), (int32_t*)(ws + L.counters), (float*)(ws + L.partial)};
    return hip_status(stage("fp8_moe", [&] { return launch_fp8_moe(dtype, a, L.plan, (hipStream_t)stream); }));
}
