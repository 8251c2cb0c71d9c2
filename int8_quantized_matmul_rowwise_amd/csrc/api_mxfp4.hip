// C-ABI entry points of the 4-bit floating point operators (declared and documented in
// include/llmint8.h).  Validation happens before anything is enqueued.
#include "api_common.hpp"
#include "launch.hpp"
#include "mxfp4_common.hpp"

using namespace llmint8;

namespace {

// Rows and sums: tiles of 256 rows of codes are addressed with 32-bit offsets.
constexpr int64_t kMaxSide = (int64_t)1 << 22;
constexpr int64_t kMaxTiles = (int64_t)1 << 24;  // workgroups of 256 threads of a launch: 2^32 threads are too many

int check_dtype(int dtype) { return dtype == LLMINT8_F16 || dtype == LLMINT8_BF16 ? LLMINT8_OK : LLMINT8_EINVAL; }

int check_product(int64_t M, int64_t K, int64_t N, int dtype) {
    if (check_dtype(dtype)) return LLMINT8_EINVAL;
    if (M < 0 || K < 0 || N < 0 || K % 16 != 0 || N % 8 != 0) return LLMINT8_EINVAL;
    if (M > kMaxSide || K > kMaxSide || N > kMaxSide) return LLMINT8_ERANGE;
    if (ceil_div(M, 32) * ceil_div(K, 256) >= kMaxTiles || ceil_div(M, 128) * ceil_div(N, 128) >= kMaxTiles) return LLMINT8_ERANGE;
    return LLMINT8_OK;
}

size_t code_bytes(int64_t rows, int64_t n) { return (size_t)rows * (size_t)fp4_pitch(n); }
size_t scale_bytes(int64_t rows, int64_t n) { return (size_t)fp4_scale_bytes(rows, n); }

bool codes_ok(const void* q, const void* s) { return q && aligned(q, 16) && s && aligned(s, 4); }

}  // namespace

LLMINT8_API int64_t fp4_code_pitch(int64_t n) { return n < 0 ? 0 : fp4_pitch(n); }
LLMINT8_API int64_t fp4_scale_pitch(int64_t n) { return n < 0 ? 0 : fp4_scale_pitch_of(n); }

LLMINT8_API int mxfp4_quantize(const void* A, int64_t R, int64_t C, int dtype, int columns, uint8_t* q, uint8_t* scale, void* stream) {
    if (check_dtype(dtype) || R < 0 || C < 0) return LLMINT8_EINVAL;
    const int64_t rows = columns ? C : R, n = columns ? R : C;
    if (n % 16 != 0 || (columns && C % 8 != 0)) return LLMINT8_EINVAL;
    if (R > kMaxSide || C > kMaxSide || ceil_div(rows, 32) * ceil_div(n, 256) >= kMaxTiles) return LLMINT8_ERANGE;
    if (R == 0 || C == 0) return LLMINT8_OK;
    if (!A || !aligned(A, 16) || !codes_ok(q, scale)) return LLMINT8_EINVAL;
    const Range r[] = {{q, code_bytes(rows, n)}, {scale, scale_bytes(rows, n)}, {A, (size_t)R * (size_t)C * 2}};
    if (clash(r, 2, 3)) return LLMINT8_EINVAL;
    log_call("mxfp4_quantize", R, C, 0, dtype, NAN, columns ? "mxfp4_columns" : "mxfp4_rows");
    hipStream_t st = (hipStream_t)stream;
    return hip_status(columns ? stage("mxfp4_columns", [&] { return launch_mxfp4_columns(dtype, A, R, C, q, scale, st); })
                              : stage("mxfp4_rows", [&] { return launch_mxfp4_rows(dtype, A, R, C, q, scale, nullptr, 0, st); }));
}

LLMINT8_API int mxfp4_dequantize(const uint8_t* q, const uint8_t* scale, int64_t R, int64_t n, int dtype, void* A, void* stream) {
    if (check_dtype(dtype) || R < 0 || n < 0 || n % 16 != 0) return LLMINT8_EINVAL;
    if (R > kMaxSide || n > kMaxSide) return LLMINT8_ERANGE;
    if (R == 0 || n == 0) return LLMINT8_OK;
    if (!A || !aligned(A, 16) || !codes_ok(q, scale)) return LLMINT8_EINVAL;
    const Range r[] = {{A, (size_t)R * (size_t)n * 2}, {q, code_bytes(R, n)}, {scale, scale_bytes(R, n)}};
    if (clash(r, 1, 3)) return LLMINT8_EINVAL;
    log_call("mxfp4_dequantize", R, n, 0, dtype, NAN, "mxfp4_values");
    return hip_status(stage("mxfp4_values", [&] { return launch_mxfp4_values(dtype, q, scale, R, n, A, (hipStream_t)stream); }));
}

// ---- Y = X W

namespace {

struct Mxfp4Layout {
    Mxfp4Plan plan;
    size_t xq, s_x, counters, partial, total;
};

Mxfp4Layout mxfp4_layout(int64_t M, int64_t K, int64_t N, bool coded) {
    Mxfp4Layout L;
    L.plan = mxfp4_plan(M, N, ceil_div(K, 256), !coded);
    const bool codes = !coded && L.plan.kind != Mxfp4Plan::kFused;
    L.xq = 0;
    L.s_x = align_up(codes ? code_bytes(M, K) : 0);
    L.counters = align_up(L.s_x + (codes ? scale_bytes(M, K) : 0));
    L.partial = align_up(L.counters + (L.plan.split > 1 ? (size_t)L.plan.tiles * 4 : 0));
    L.total = align_up(L.partial + (size_t)L.plan.partial_bytes);
    return L;
}

const char* plan_name(const Mxfp4Plan& p) {
    switch (p.kind) {
        case Mxfp4Plan::kTile256: return "mxfp4_tile256";
        case Mxfp4Plan::kTile128: return "mxfp4_tile128";
        case Mxfp4Plan::kSingle: return p.split > 1 ? "mxfp4_single_split" : "mxfp4_single";
        case Mxfp4Plan::kSmall: return p.split > 1 ? "mxfp4_small_split" : "mxfp4_small";
        default: return "mxfp4_small_fused";
    }
}

// X: 16 bits, or (coded) rows of codes with x_scale
int product(const char* name, const void* X, const uint8_t* x_scale, bool coded, int64_t M, int64_t K, int dtype, const uint8_t* Wq,
            const uint8_t* w_scale, int64_t N, void* Y, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_product(M, K, N, dtype);
    if (rc) return rc;
    if (M == 0 || N == 0) return LLMINT8_OK;
    if (!Y || !aligned(Y, 16)) return LLMINT8_EINVAL;
    hipStream_t st = (hipStream_t)stream;
    if (K == 0) {
        log_call(name, M, K, N, dtype, NAN, "empty sum");
        return hip_status(stage("fill_zero", [&] { return launch_fill_zero((float*)Y, M * N / 2, st); }));
    }
    if (!X || !aligned(X, 16) || (coded && !codes_ok(X, x_scale)) || !codes_ok(Wq, w_scale)) return LLMINT8_EINVAL;
    const Mxfp4Layout L = mxfp4_layout(M, K, N, coded);
    if (L.total > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < L.total)) return LLMINT8_EWORKSPACE;
    const Range r[] = {{Y, (size_t)M * (size_t)N * 2},
                       {workspace, L.total},
                       {X, coded ? code_bytes(M, K) : (size_t)M * (size_t)K * 2},
                       {x_scale, coded ? scale_bytes(M, K) : 0},
                       {Wq, code_bytes(N, K)},
                       {w_scale, scale_bytes(N, K)}};
    if (clash(r, 2, 6)) return LLMINT8_EINVAL;
    if (log_call(name, M, K, N, dtype, NAN, plan_name(L.plan)))
        fprintf(stderr, "[llmint8]   plan pieces=%d columns=%d parts=%d\n", (int)L.plan.pieces, (int)L.plan.columns, (int)L.plan.split);
    uint8_t* ws = (uint8_t*)workspace;
    int32_t* counters = L.plan.split > 1 ? (int32_t*)(ws + L.counters) : nullptr;
    const int64_t n_counters = counters ? L.plan.tiles : 0;
    hipError_t e = hipSuccess;
    if (coded) {
        if (counters) e = stage("fill_zero", [&] { return launch_fill_zero((float*)counters, n_counters, st); });
    } else if (L.plan.kind != Mxfp4Plan::kFused) {
        e = stage("mxfp4_rows", [&] { return launch_mxfp4_rows(dtype, X, M, K, ws + L.xq, ws + L.s_x, counters, n_counters, st); });
    }
    if (e == hipSuccess)
        e = stage("mxfp4_gemm", [&] {
            const Mxfp4GemmArgs a{coded ? (const uint8_t*)X : ws + L.xq, Wq, M, N, fp4_pitch(K), coded ? x_scale : ws + L.s_x, w_scale, 0,
                                  (uint16_t*)Y, coded ? nullptr : (const uint16_t*)X, K, counters, (float*)(ws + L.partial)};
            return launch_mxfp4_gemm(dtype, a, L.plan, st);
        });
    return hip_status(e);
}

size_t product_workspace(int64_t M, int64_t K, int64_t N, bool coded) {
    if (check_product(M, K, N, LLMINT8_F16) || M == 0 || N == 0 || K == 0) return 0;
    return mxfp4_layout(M, K, N, coded).total;
}

}  // namespace

LLMINT8_API size_t mxfp4_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N) { return product_workspace(M, K, N, false); }
LLMINT8_API size_t mxfp4_matmul_coded_workspace_bytes(int64_t M, int64_t K, int64_t N) { return product_workspace(M, K, N, true); }

LLMINT8_API int mxfp4_matmul(const void* X, int64_t M, int64_t K, int dtype, const uint8_t* Wq, const uint8_t* w_scale, int64_t N, void* Y,
                             void* workspace, size_t workspace_bytes, void* stream) {
    return product("mxfp4_matmul", X, nullptr, false, M, K, dtype, Wq, w_scale, N, Y, workspace, workspace_bytes, stream);
}

LLMINT8_API int mxfp4_matmul_coded(const uint8_t* Xq, const uint8_t* x_scale, int64_t M, int64_t K, int dtype, const uint8_t* Wq,
                                   const uint8_t* w_scale, int64_t N, void* Y, void* workspace, size_t workspace_bytes, void* stream) {
    return product("mxfp4_matmul_coded", Xq, x_scale, true, M, K, dtype, Wq, w_scale, N, Y, workspace, workspace_bytes, stream);
}
