// Host-side helpers shared by the C-ABI entry points: alignment and overlap checks, the
// per-call log, failure injection and the mapping of HIP errors.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/llmint8.h"

#define LLMINT8_API extern "C" __attribute__((visibility("default")))

namespace llmint8 {
namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

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

// ---- failure injection and logging (host layer only; both read the environment per call)
//   LLMINT8_FAULT=<stage>  dry run: nothing is enqueued; every stage the call reaches before
//                          the named one counts as done, the named one as failed, so the
//                          error path (LLMINT8_EHIP, nothing reported as done) runs on a
//                          machine without a GPU.  A call whose path does not contain the
//                          stage returns LLMINT8_OK having enqueued nothing.
//   LLMINT8_LOG=1          each call's sizes, dtype, threshold and path, and each stage, on
//                          stderr.
const char* fault_stage() {
    const char* f = getenv("LLMINT8_FAULT");
    return f && *f ? f : nullptr;
}

bool log_on() {
    const char* l = getenv("LLMINT8_LOG");
    return l && *l && strcmp(l, "0") != 0;
}

const char* dtype_name(int dt) { return dt == LLMINT8_F16 ? "fp16" : "bf16"; }

// tau: NaN where the call takes no threshold.  Returns whether the log is on.
bool log_call(const char* fn, int64_t M, int64_t K, int64_t N, int dt, float tau, const char* path) {
    if (!log_on()) return false;
    char t[32] = "";
    if (!isnan(tau)) snprintf(t, sizeof t, " threshold=%g", (double)tau);
    fprintf(stderr, "[llmint8] %s M=%lld K=%lld N=%lld dtype=%s%s path=%s%s\n", fn, (long long)M, (long long)K,
            (long long)N, dtype_name(dt), t, path, fault_stage() ? " (dry run)" : "");
    return true;
}

// Run one stage of a call: `launch` enqueues it and returns its HIP status.
template <class Launch>
hipError_t stage(const char* name, Launch&& launch) {
    const char* f = fault_stage();
    const bool fail = f && strcmp(f, name) == 0;
    if (log_on()) fprintf(stderr, "[llmint8]   stage %s%s\n", name, fail ? ": injected failure" : (f ? ": skipped" : ""));
    if (f) return fail ? hipErrorLaunchFailure : hipSuccess;
    return launch();
}

int hip_status(hipError_t e) {
    if (e == hipSuccess) return LLMINT8_OK;
    if (!fault_stage()) (void)hipGetLastError();  // consume the sticky error (an injected one has none)
    return LLMINT8_EHIP;
}

}  // namespace
}  // namespace llmint8
