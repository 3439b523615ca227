// q4_check.h -- argument checks that the entry points in q4_mx_abi.cpp and
// q4_nn_abi.cpp share: each returns Q4_OK, or stores the thread's message and
// returns the status.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/q4adamw.h"
#include "q4_internal.h"
#include "q4_mx.h"

namespace q4 {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;
constexpr int64_t kMaxElems = int64_t(1) << 34;

q4_status bad(q4_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return (q4_status)report(s, buf);
}
q4_status ok() { return (q4_status)report(Q4_OK, nullptr); }

int64_t padded(int64_t cols) { return (cols + kMxPad - 1) / kMxPad * kMxPad; }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

q4_status check_shape(const char* name, int32_t format, int64_t rows, int64_t cols) {
    if (format != Q4MX_FP4 && format != Q4MX_FP8) return bad(Q4_ERR_INVALID_ARG, "%s: unknown format %d", name, format);
    if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim)
        return bad(Q4_ERR_SHAPE, "%s: %lld x %lld outside [0, 2^31)", name, (long long)rows, (long long)cols);
    if (rows > 0 && padded(cols) >= (kMaxElems + rows - 1) / rows)
        return bad(Q4_ERR_SHAPE, "%s: %lld x %lld has 2^34 padded elements or more", name, (long long)rows,
                   (long long)cols);
    return Q4_OK;
}

q4_status check_mx_shape(const char* name, const q4mx_matrix* m) {
    if (!m) return bad(Q4_ERR_INVALID_ARG, "%s is NULL", name);
    if (m->reserved != 0) return bad(Q4_ERR_INVALID_ARG, "%s: reserved must be 0", name);
    return check_shape(name, m->format, m->rows, m->cols);
}

q4_status check_mx(const char* name, const q4mx_matrix* m) {
    q4_status s = check_mx_shape(name, m);
    if (s != Q4_OK || m->rows == 0 || m->cols == 0) return s;
    if (!m->codes || !m->scales) return bad(Q4_ERR_INVALID_ARG, "%s: codes or scales is NULL", name);
    if (((reinterpret_cast<uintptr_t>(m->codes) | reinterpret_cast<uintptr_t>(m->scales)) & 15) != 0)
        return bad(Q4_ERR_ALIGNMENT, "%s: codes and scales must be 16-byte aligned", name);
    return Q4_OK;
}

q4_status check_dense(const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
    if (dtype != Q4MX_F32 && dtype != Q4MX_BF16) return bad(Q4_ERR_INVALID_ARG, "%s: unknown dtype %d", name, dtype);
    if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim)
        return bad(Q4_ERR_SHAPE, "%s: %lld x %lld outside [0, 2^31)", name, (long long)rows, (long long)cols);
    if (rows == 0 || cols == 0) return Q4_OK;
    if (ld < cols || ld >= kMaxDim)
        return bad(Q4_ERR_SHAPE, "%s: row stride %lld outside [%lld, 2^31)", name, (long long)ld, (long long)cols);
    if (!p) return bad(Q4_ERR_INVALID_ARG, "%s is NULL", name);
    const uintptr_t unit = dtype == Q4MX_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(p) % unit) return bad(Q4_ERR_ALIGNMENT, "%s is not aligned to its element", name);
    return Q4_OK;
}

MxMat mat(const q4mx_matrix* m) {
    if (!m) return MxMat{};
    return MxMat{m->codes, m->scales, m->rows, m->cols, padded(m->cols) / kMxPad, m->format};
}

q4_status launched(hipError_t e, const char* what) {
    return e == hipSuccess ? ok() : bad(Q4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

q4_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (need == 0) return Q4_OK;
    if (!ws) return bad(Q4_ERR_WORKSPACE, "workspace is NULL, the call needs %zu bytes", need);
    if (reinterpret_cast<uintptr_t>(ws) & 15) return bad(Q4_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
    if (ws_bytes < need) return bad(Q4_ERR_WORKSPACE, "workspace has %zu bytes, the call needs %zu", ws_bytes, need);
    return Q4_OK;
}

#define Q4_TRY(x)                        \
    do {                                 \
        const q4_status s_ = (x);        \
        if (s_ != Q4_OK) return s_;      \
    } while (0)

q4_status device() {
    int dev = 0;
    return (q4_status)current_device(&dev);
}

q4_status check_result(int64_t rows, int64_t cols) {
    if (rows > 0 && cols > 0 && rows >= (int64_t(1) << 38) / cols)
        return bad(Q4_ERR_SHAPE, "a result of %lld x %lld has 2^38 elements or more", (long long)rows, (long long)cols);
    return Q4_OK;
}

}  // namespace
}  // namespace q4
