// q4_mx_abi.cpp -- host side of the microscaled linear layer's entry points
// (include/q4adamw.h): every call checks its arguments first and enqueues
// nothing when it returns an error.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/q4adamw.h"
#include "q4_internal.h"
#include "q4_mx.h"

using namespace q4;

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

// x's codes and scales in a workspace, when a BF16 x is quantized on the way.
struct Quantized {
    size_t codes, scales;
    size_t bytes() const { return codes + scales; }
};
Quantized quantized(int64_t tokens, int64_t cols) {
    return Quantized{round256((size_t)(tokens * padded(cols))), round256((size_t)(tokens * padded(cols) / 32))};
}

// The same product's workspace: those, then the product's own.
MxMat quantized_at(uint8_t* p, const Quantized& q, int64_t tokens, int64_t cols) {
    return MxMat{p, p ? p + q.codes : nullptr, tokens, cols, padded(cols) / kMxPad, Q4MX_FP8};
}
size_t bf16_workspace(int64_t tokens, const q4mx_matrix* w) {
    if (tokens <= Q4MX_FEW_TOKENS) return 0;
    const Quantized q = quantized(tokens, w->cols);
    return q.bytes() + linear_workspace(quantized_at(nullptr, q, tokens, w->cols), mat(w));
}

// Workspace of a gradient product, in front of the product's own: the copy of a dy whose rows are not aligned.
size_t copy_bytes(const uint16_t* dy, int64_t lddy, int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0 || !dense_needs_copy(Dense{const_cast<uint16_t*>(dy), lddy, Q4MX_BF16}, rows, cols))
        return 0;
    return round256(dense_copy_bytes(rows, cols));
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

// The products address a tile's rows with 32-bit byte offsets from its first.
constexpr int64_t kMaxWidth = int64_t(1) << 23;
q4_status check_width(const char* name, int64_t n) {
    if (n >= kMaxWidth) return bad(Q4_ERR_SHAPE, "%s is %lld, a product takes less than 2^23", name, (long long)n);
    return Q4_OK;
}

q4_status check_result(int64_t rows, int64_t cols) {
    if (rows > 0 && cols > 0 && rows >= (int64_t(1) << 38) / cols)
        return bad(Q4_ERR_SHAPE, "a result of %lld x %lld has 2^38 elements or more", (long long)rows, (long long)cols);
    return Q4_OK;
}

q4_status check_weight(const q4mx_matrix* w) {
    Q4_TRY(check_mx("w", w));
    if (w->format != Q4MX_FP4) return bad(Q4_ERR_CONFLICT, "w must be in Q4MX_FP4");
    return check_width("w->cols", w->cols);
}

}  // namespace

extern "C" {

q4_status q4mx_matrix_bytes(int32_t format, int64_t rows, int64_t cols, size_t* codes, size_t* scales) {
    if (!codes || !scales) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    Q4_TRY(check_shape("matrix", format, rows, cols));
    const size_t n = (size_t)(rows * padded(cols));
    *codes = format == Q4MX_FP4 ? n / 2 : n;
    *scales = n / 32;
    return ok();
}

q4_status q4mx_quantize(const void* src, int32_t dtype, int64_t ld, int32_t transpose, const q4mx_matrix* out,
                        void* stream) {
    Q4_TRY(check_mx("out", out));
    if (transpose != 0 && transpose != 1) return bad(Q4_ERR_INVALID_ARG, "transpose must be 0 or 1");
    Q4_TRY(check_dense("src", src, dtype, transpose ? out->cols : out->rows, transpose ? out->rows : out->cols, ld));
    if (out->rows == 0 || out->cols == 0) return ok();
    Q4_TRY(device());
    return launched(launch_mx_quantize(Dense{const_cast<void*>(src), ld, dtype}, transpose != 0, mat(out),
                                       reinterpret_cast<hipStream_t>(stream)),
                    "quantize launch");
}

q4_status q4mx_dequantize(const q4mx_matrix* a, void* dst, int32_t dtype, int64_t ld, void* stream) {
    Q4_TRY(check_mx("a", a));
    Q4_TRY(check_dense("dst", dst, dtype, a->rows, a->cols, ld));
    if (a->rows == 0 || a->cols == 0) return ok();
    Q4_TRY(device());
    return launched(launch_mx_dequantize(mat(a), Dense{dst, ld, dtype}, reinterpret_cast<hipStream_t>(stream)),
                    "dequantize launch");
}

q4_status q4mx_linear_workspace_bytes(const q4mx_matrix* x, const q4mx_matrix* w, size_t* bytes) {
    if (!bytes) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    Q4_TRY(check_mx_shape("x", x));
    Q4_TRY(check_mx_shape("w", w));
    *bytes = linear_workspace(mat(x), mat(w));
    return ok();
}

q4_status q4mx_linear(const q4mx_matrix* x, const q4mx_matrix* w, void* y, int32_t dtype, int64_t ldy, void* ws,
                      size_t ws_bytes, void* stream) {
    Q4_TRY(check_mx("x", x));
    Q4_TRY(check_weight(w));
    if (x->cols != w->cols)
        return bad(Q4_ERR_SHAPE, "x has %lld columns, w has %lld", (long long)x->cols, (long long)w->cols);
    Q4_TRY(check_dense("y", y, dtype, x->rows, w->rows, ldy));
    Q4_TRY(check_result(x->rows, w->rows));
    if (x->rows == 0 || w->rows == 0) return ok();
    size_t need = 0;
    Q4_TRY(q4mx_linear_workspace_bytes(x, w, &need));
    Q4_TRY(check_ws(ws, ws_bytes, need));
    Q4_TRY(device());
    return launched(launch_linear(mat(x), mat(w), Dense{y, ldy, dtype}, ws, reinterpret_cast<hipStream_t>(stream)),
                    "linear launch");
}

q4_status q4mx_linear_bf16_workspace_bytes(int64_t tokens, const q4mx_matrix* w, size_t* bytes) {
    if (!bytes) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    Q4_TRY(check_mx_shape("w", w));
    Q4_TRY(check_shape("x", Q4MX_FP8, tokens, w->cols));
    *bytes = bf16_workspace(tokens, w);
    return ok();
}

q4_status q4mx_linear_bf16(const uint16_t* x, int64_t ldx, int64_t tokens, const q4mx_matrix* w, void* y,
                           int32_t dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    Q4_TRY(check_weight(w));
    Q4_TRY(check_shape("x", Q4MX_FP8, tokens, w->cols));
    Q4_TRY(check_dense("x", x, Q4MX_BF16, tokens, w->cols, ldx));
    Q4_TRY(check_dense("y", y, dtype, tokens, w->rows, ldy));
    Q4_TRY(check_result(tokens, w->rows));
    if (tokens == 0 || w->rows == 0) return ok();
    Q4_TRY(check_width("ldx", tokens > 1 && w->cols > 0 ? ldx : 0));
    const Quantized q = quantized(tokens, w->cols);
    Q4_TRY(check_ws(ws, ws_bytes, bf16_workspace(tokens, w)));
    Q4_TRY(device());
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (tokens <= Q4MX_FEW_TOKENS)
        return launched(launch_linear_few(Dense{const_cast<uint16_t*>(x), ldx, Q4MX_BF16}, tokens, mat(w),
                                          Dense{y, ldy, dtype}, st),
                        "linear launch");
    uint8_t* p = static_cast<uint8_t*>(ws);
    const MxMat xq = quantized_at(p, q, tokens, w->cols);
    if (w->cols > 0) {
        const hipError_t e =
            launch_mx_quantize(Dense{const_cast<uint16_t*>(x), ldx, Q4MX_BF16}, false, xq, st);
        if (e != hipSuccess) return launched(e, "quantize launch");
    }
    return launched(launch_linear(xq, mat(w), Dense{y, ldy, dtype}, p + q.bytes(), st), "linear launch");
}

q4_status q4mx_dgrad_workspace_bytes(const uint16_t* dy, int64_t lddy, int64_t tokens, const q4mx_matrix* w,
                                     size_t* bytes) {
    if (!bytes) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    Q4_TRY(check_mx_shape("w", w));
    Q4_TRY(check_dense("dy", dy, Q4MX_BF16, tokens, w->rows, lddy));
    *bytes = copy_bytes(dy, lddy, tokens, w->rows) + grad_workspace(mat(w), tokens);
    return ok();
}

q4_status q4mx_dgrad(const uint16_t* dy, int64_t lddy, int64_t tokens, const q4mx_matrix* w, void* dx, int32_t dtype,
                     int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
    Q4_TRY(check_weight(w));
    Q4_TRY(check_dense("dy", dy, Q4MX_BF16, tokens, w->rows, lddy));
    Q4_TRY(check_width("lddy", tokens > 0 && w->rows > 0 ? lddy : 0));
    Q4_TRY(check_dense("dx", dx, dtype, tokens, w->cols, lddx));
    Q4_TRY(check_result(tokens, w->cols));
    if (tokens == 0 || w->cols == 0) return ok();
    size_t need = 0;
    Q4_TRY(q4mx_dgrad_workspace_bytes(dy, lddy, tokens, w, &need));
    Q4_TRY(check_ws(ws, ws_bytes, need));
    Q4_TRY(device());
    return launched(launch_dgrad(Dense{const_cast<uint16_t*>(dy), lddy, Q4MX_BF16}, tokens, mat(w),
                                 Dense{dx, lddx, dtype}, ws,
                                 static_cast<char*>(ws) + copy_bytes(dy, lddy, tokens, w->rows), reinterpret_cast<hipStream_t>(stream)),
                    "dgrad launch");
}

q4_status q4mx_wgrad_workspace_bytes(const uint16_t* dy, int64_t lddy, int64_t n, const q4mx_matrix* x,
                                     int32_t flags, size_t* bytes) {
    if (!bytes) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    if (flags & ~(Q4MX_WGRAD_TRANSPOSED | Q4MX_WGRAD_ADD)) return bad(Q4_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    Q4_TRY(check_mx_shape("x", x));
    Q4_TRY(check_dense("dy", dy, Q4MX_BF16, x->rows, n, lddy));
    *bytes = copy_bytes(dy, lddy, x->rows, n) + grad_workspace(mat(x), n);
    return ok();
}

q4_status q4mx_wgrad(const uint16_t* dy, int64_t lddy, int64_t n, const q4mx_matrix* x, void* dw, int32_t dtype,
                     int64_t lddw, int32_t flags, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    Q4_TRY(check_mx("x", x));
    Q4_TRY(check_width("x->cols", x->cols));
    Q4_TRY(check_width("lddy", x->rows > 0 && n > 0 ? lddy : 0));
    Q4_TRY(q4mx_wgrad_workspace_bytes(dy, lddy, n, x, flags, &need));
    const bool t = (flags & Q4MX_WGRAD_TRANSPOSED) != 0;
    Q4_TRY(check_dense("dw", dw, dtype, t ? x->cols : n, t ? n : x->cols, lddw));
    Q4_TRY(check_result(n, x->cols));
    if (n == 0 || x->cols == 0) return ok();
    Q4_TRY(check_ws(ws, ws_bytes, need));
    Q4_TRY(device());
    return launched(launch_wgrad(Dense{const_cast<uint16_t*>(dy), lddy, Q4MX_BF16}, n, mat(x), Dense{dw, lddw, dtype},
                                 t, (flags & Q4MX_WGRAD_ADD) != 0, ws, static_cast<char*>(ws) + copy_bytes(dy, lddy, x->rows, n),
                                 reinterpret_cast<hipStream_t>(stream)),
                    "wgrad launch");
}

}  // extern "C"

namespace {

q4_status check_act(int32_t act) {
    if (act < Q4MX_GELU || act > Q4MX_SWIGLU) return bad(Q4_ERR_INVALID_ARG, "unknown activation %d", act);
    return Q4_OK;
}

// An MX operand of an activation call: rows x cols, in FP8 unless `any`.
q4_status check_act_mx(const char* name, const q4mx_matrix* m, int64_t rows, int64_t cols, bool any) {
    Q4_TRY(check_mx(name, m));
    if (m->rows != rows || m->cols != cols)
        return bad(Q4_ERR_SHAPE, "%s is %lld x %lld, expected %lld x %lld", name, (long long)m->rows,
                   (long long)m->cols, (long long)rows, (long long)cols);
    if (!any && m->format != Q4MX_FP8) return bad(Q4_ERR_CONFLICT, "%s must be in Q4MX_FP8", name);
    return Q4_OK;
}

}  // namespace

extern "C" {

q4_status q4mx_act_forward(int32_t act, const uint16_t* x, int64_t ldx, const uint16_t* up, int64_t ldup,
                           int64_t rows, int64_t cols, uint16_t* y, int64_t ldy, const q4mx_matrix* y_mx,
                           const q4mx_matrix* kept_x, const q4mx_matrix* kept_up, void* stream) {
    Q4_TRY(check_act(act));
    Q4_TRY(check_shape("x", Q4MX_FP8, rows, cols));
    const bool two = act == Q4MX_SWIGLU;
    if (!two && (up || kept_up)) return bad(Q4_ERR_CONFLICT, "only Q4MX_SWIGLU takes up and kept_up");
    if (y_mx) Q4_TRY(check_act_mx("y_mx", y_mx, rows, cols, true));
    if (kept_x) Q4_TRY(check_act_mx("kept_x", kept_x, rows, cols, false));
    if (kept_up) Q4_TRY(check_act_mx("kept_up", kept_up, rows, cols, false));
    Q4_TRY(check_dense("x", x, Q4MX_BF16, rows, cols, ldx));
    if (two) Q4_TRY(check_dense("up", up, Q4MX_BF16, rows, cols, ldup));
    if (y) Q4_TRY(check_dense("y", y, Q4MX_BF16, rows, cols, ldy));
    if (rows == 0 || cols == 0) return ok();
    if (!y && !y_mx && !kept_x && !kept_up) return bad(Q4_ERR_INVALID_ARG, "no output is given");
    Q4_TRY(device());
    return launched(launch_act_forward(act, Dense{const_cast<uint16_t*>(x), ldx, Q4MX_BF16},
                                       Dense{const_cast<uint16_t*>(two ? up : nullptr), ldup, Q4MX_BF16}, rows, cols,
                                       Dense{y, ldy, Q4MX_BF16}, mat(y_mx), mat(kept_x), mat(kept_up),
                                       reinterpret_cast<hipStream_t>(stream)),
                    "activation launch");
}

q4_status q4mx_act_backward(int32_t act, const q4mx_matrix* kept_x, const q4mx_matrix* kept_up, const uint16_t* dy,
                            int64_t lddy, uint16_t* dx, int64_t lddx, uint16_t* dup, int64_t lddup, void* stream) {
    Q4_TRY(check_act(act));
    if (!kept_x) return bad(Q4_ERR_INVALID_ARG, "kept_x is NULL");
    const int64_t rows = kept_x->rows, cols = kept_x->cols;
    Q4_TRY(check_act_mx("kept_x", kept_x, rows, cols, false));
    const bool two = act == Q4MX_SWIGLU;
    if (!two && (kept_up || dup)) return bad(Q4_ERR_CONFLICT, "only Q4MX_SWIGLU takes kept_up and dup");
    if (two) Q4_TRY(check_act_mx("kept_up", kept_up, rows, cols, false));
    Q4_TRY(check_dense("dy", dy, Q4MX_BF16, rows, cols, lddy));
    Q4_TRY(check_dense("dx", dx, Q4MX_BF16, rows, cols, lddx));
    if (two) Q4_TRY(check_dense("dup", dup, Q4MX_BF16, rows, cols, lddup));
    if (dx == dy && lddx != lddy) return bad(Q4_ERR_SHAPE, "dx in place of dy must have its row stride");
    if (rows == 0 || cols == 0) return ok();
    Q4_TRY(device());
    return launched(launch_act_backward(act, mat(kept_x), mat(kept_up), Dense{const_cast<uint16_t*>(dy), lddy, Q4MX_BF16},
                                        Dense{dx, lddx, Q4MX_BF16}, Dense{two ? dup : nullptr, lddup, Q4MX_BF16},
                                        reinterpret_cast<hipStream_t>(stream)),
                    "activation gradient launch");
}

}  // extern "C"
