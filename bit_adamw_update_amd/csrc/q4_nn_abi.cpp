// q4_nn_abi.cpp -- host side of the entry points of embedding, head norms and
// dropout (include/q4adamw.h): every call checks its arguments first and
// enqueues nothing when it returns an error.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "../../include/q4adamw.h"
#include "q4_check.h"
#include "q4_nn.h"

using namespace q4;

namespace {

q4_status check_ints(const char* name, const void* p, int32_t type, int64_t n) {
    if (type != Q4NN_I32 && type != Q4NN_I64) return bad(Q4_ERR_INVALID_ARG, "%s: unknown integer type %d", name, type);
    if (n < 0 || n >= kMaxDim) return bad(Q4_ERR_SHAPE, "%s: %lld entries, outside [0, 2^31)", name, (long long)n);
    if (n == 0) return Q4_OK;
    if (!p) return bad(Q4_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % (type == Q4NN_I32 ? 4 : 8))
        return bad(Q4_ERR_ALIGNMENT, "%s is not aligned to its element", name);
    return Q4_OK;
}

q4_status check_scale(float scale) {
    if (!std::isfinite(scale)) return bad(Q4_ERR_INVALID_ARG, "scale is not finite");
    return Q4_OK;
}

q4_status check_flags(int32_t flags) {
    if (flags & ~Q4NN_ADD) return bad(Q4_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    return Q4_OK;
}

Dense dense(const void* p, int64_t ld, int dtype) { return Dense{const_cast<void*>(p), ld, dtype}; }

// The results of an embedding, shared by its two forms.
q4_status check_lookup(const void* ids, int32_t id_type, int64_t tokens, int64_t cols, float scale, const void* out,
                       int32_t out_dtype, int64_t ldo) {
    Q4_TRY(check_ints("ids", ids, id_type, tokens));
    Q4_TRY(check_scale(scale));
    Q4_TRY(check_dense("out", out, out_dtype, tokens, cols, ldo));
    return check_result(tokens, cols);
}

// One [batches][tokens][heads][dim] operand.
q4_status check_heads(const char* name, const q4nn_heads* v, const q4nn_rope* r, int32_t heads, bool written) {
    if (!v) return bad(Q4_ERR_INVALID_ARG, "%s is NULL", name);
    if (r->batches * r->tokens * heads == 0) return Q4_OK;
    if (!v->p) return bad(Q4_ERR_INVALID_ARG, "%s.p is NULL", name);
    if (reinterpret_cast<uintptr_t>(v->p) & 1) return bad(Q4_ERR_ALIGNMENT, "%s is not aligned to its element", name);
    int64_t stride[3] = {v->batch, v->token, v->head}, count[3] = {r->batches, r->tokens, heads};
    __int128 last = r->dim;
    for (int i = 0; i < 3; ++i) {
        if (stride[i] < 0 || stride[i] >= int64_t(1) << 40)
            return bad(Q4_ERR_SHAPE, "%s: stride %lld outside [0, 2^40)", name, (long long)stride[i]);
        last += (__int128)stride[i] * (count[i] - 1);
    }
    if (last >= int64_t(1) << 50) return bad(Q4_ERR_SHAPE, "%s: spans 2^50 elements or more", name);
    if (!written) return Q4_OK;
    // no two elements of a result in one place: from the smallest stride on, each steps past what the others span
    int64_t span = r->dim;
    for (int n = 0; n < 3; ++n) {
        int least = -1;
        for (int i = 0; i < 3; ++i)
            if (count[i] > 1 && (least < 0 || stride[i] < stride[least])) least = i;
        if (least < 0) break;
        if (stride[least] < span) return bad(Q4_ERR_SHAPE, "%s: elements overlap", name);
        span += stride[least] * (count[least] - 1);
        count[least] = 1;
    }
    return Q4_OK;
}

// Whether a in place of b would be read as another element than it is written;
// the stride of a single entry means nothing.
bool shifted(const q4nn_heads* a, const q4nn_heads* b, const q4nn_rope* r, int32_t heads) {
    return a->p == b->p && r->batches * r->tokens * heads > 0 &&
           ((r->batches > 1 && a->batch != b->batch) || (r->tokens > 1 && a->token != b->token) ||
            (heads > 1 && a->head != b->head));
}

// Whether an operand of q and one of k begin in one place.
bool one_place(const q4nn_heads* q, const q4nn_heads* k, const q4nn_rope* r) {
    return q->p == k->p && r->batches * r->tokens > 0 && r->q_heads > 0 && r->k_heads > 0;
}

q4_status check_rope(const q4nn_rope* r) {
    if (!r) return bad(Q4_ERR_INVALID_ARG, "r is NULL");
    if (r->batches < 0 || r->tokens < 0 || r->batches >= kMaxDim || r->tokens >= kMaxDim ||
        r->batches * r->tokens >= kMaxDim)
        return bad(Q4_ERR_SHAPE, "%lld batches of %lld tokens are outside [0, 2^31)", (long long)r->batches,
                   (long long)r->tokens);
    if (r->q_heads < 0 || r->q_heads > 4096 || r->k_heads < 0 || r->k_heads > 4096)
        return bad(Q4_ERR_SHAPE, "%d and %d heads, outside [0, 4096]", r->q_heads, r->k_heads);
    if (r->dim < 2 || r->dim > 1024 || r->dim % 2)
        return bad(Q4_ERR_SHAPE, "dim %d is not even or outside [2, 1024]", r->dim);
    if (r->rotary < 0 || r->rotary > r->dim || r->rotary % 2)
        return bad(Q4_ERR_SHAPE, "rotary %d is not even or outside [0, %d]", r->rotary, r->dim);
    if (r->interleaved != 0 && r->interleaved != 1) return bad(Q4_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(r->eps >= FLT_MIN && r->eps <= FLT_MAX))
        return bad(Q4_ERR_INVALID_ARG, "eps must be a normal positive number");
    if (r->gain_dtype != Q4MX_F32 && r->gain_dtype != Q4MX_BF16)
        return bad(Q4_ERR_INVALID_ARG, "gains: unknown dtype %d", r->gain_dtype);
    Q4_TRY(check_ints("positions", r->positions, r->position_type, r->batches * r->tokens));
    if (r->position_batch < 0 || r->position_batch >= kMaxDim || r->position_token < 0 || r->position_token >= kMaxDim)
        return bad(Q4_ERR_SHAPE, "positions: a stride is outside [0, 2^31)");
    const uintptr_t unit = r->gain_dtype == Q4MX_F32 ? 4 : 2;
    if (r->q_heads > 0 && !r->q_gain) return bad(Q4_ERR_INVALID_ARG, "q_gain is NULL");
    if (r->k_heads > 0 && !r->k_gain) return bad(Q4_ERR_INVALID_ARG, "k_gain is NULL");
    if ((reinterpret_cast<uintptr_t>(r->q_gain) | reinterpret_cast<uintptr_t>(r->k_gain)) % unit)
        return bad(Q4_ERR_ALIGNMENT, "a gain is not aligned to its element");
    if (r->rotary > 0 && !r->frequencies) return bad(Q4_ERR_INVALID_ARG, "frequencies is NULL");
    if (reinterpret_cast<uintptr_t>(r->frequencies) % 8)
        return bad(Q4_ERR_ALIGNMENT, "frequencies is not aligned to its element");
    return check_result(r->batches * r->tokens, (int64_t)(r->q_heads > r->k_heads ? r->q_heads : r->k_heads) * r->dim);
}

bool empty(const q4nn_rope* r) { return r->batches == 0 || r->tokens == 0 || r->q_heads + r->k_heads == 0; }

}  // namespace

extern "C" {

q4_status q4nn_embedding(const void* ids, int32_t id_type, int64_t tokens, const void* table, int32_t dtype,
                         int64_t rows, int64_t cols, int64_t ld, float scale, void* out, int32_t out_dtype, int64_t ldo,
                         void* stream) {
    Q4_TRY(check_dense("table", table, dtype, rows, cols, ld));
    Q4_TRY(check_lookup(ids, id_type, tokens, cols, scale, out, out_dtype, ldo));
    if (tokens == 0 || cols == 0) return ok();
    if (rows > 0 && out == table) return bad(Q4_ERR_CONFLICT, "out is in the place of the table");
    Q4_TRY(device());
    return launched(launch_embedding(Ids{ids, tokens, id_type}, dense(table, ld, dtype), MxMat{}, rows, cols, scale,
                                     dense(out, ldo, out_dtype), reinterpret_cast<hipStream_t>(stream)),
                    "embedding launch");
}

q4_status q4nn_embedding_mx(const void* ids, int32_t id_type, int64_t tokens, const q4mx_matrix* table, float scale,
                            void* out, int32_t out_dtype, int64_t ldo, void* stream) {
    Q4_TRY(check_mx("table", table));
    Q4_TRY(check_lookup(ids, id_type, tokens, table->cols, scale, out, out_dtype, ldo));
    if (tokens == 0 || table->cols == 0) return ok();
    if (table->rows > 0 && (out == table->codes || out == table->scales))
        return bad(Q4_ERR_CONFLICT, "out is in the place of the table");
    Q4_TRY(device());
    return launched(launch_embedding(Ids{ids, tokens, id_type}, Dense{}, mat(table), table->rows, table->cols, scale,
                                     dense(out, ldo, out_dtype), reinterpret_cast<hipStream_t>(stream)),
                    "embedding launch");
}

q4_status q4nn_embedding_grad_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    if (tokens < 0 || rows < 0 || cols < 0 || tokens >= kMaxDim || rows >= kMaxDim || cols >= kMaxDim)
        return bad(Q4_ERR_SHAPE, "%lld tokens, %lld x %lld rows: outside [0, 2^31)", (long long)tokens, (long long)rows,
                   (long long)cols);
    Q4_TRY(check_result(tokens, cols));
    *bytes = rows == 0 || cols == 0 ? 0 : embedding_grad_workspace(tokens, cols);
    return ok();
}

q4_status q4nn_embedding_grad(const void* ids, int32_t id_type, int64_t tokens, const uint16_t* dy, int64_t lddy,
                              float scale, int64_t rows, int64_t cols, void* grad, int32_t dtype, int64_t ldg,
                              int32_t flags, void* ws, size_t ws_bytes, void* stream) {
    Q4_TRY(check_flags(flags));
    Q4_TRY(check_ints("ids", ids, id_type, tokens));
    Q4_TRY(check_scale(scale));
    Q4_TRY(check_dense("dy", dy, Q4MX_BF16, tokens, cols, lddy));
    Q4_TRY(check_dense("grad", grad, dtype, rows, cols, ldg));
    Q4_TRY(check_result(rows, cols));
    size_t need = 0;
    Q4_TRY(q4nn_embedding_grad_workspace_bytes(tokens, rows, cols, &need));
    const bool add = (flags & Q4NN_ADD) != 0;
    if (rows == 0 || cols == 0 || (add && tokens == 0)) return ok();
    Q4_TRY(check_ws(ws, ws_bytes, need));
    if (tokens > 0 && grad == dy) return bad(Q4_ERR_CONFLICT, "grad is in the place of dy, which is read after it is written");
    Q4_TRY(device());
    return launched(launch_embedding_grad(Ids{ids, tokens, id_type}, dense(dy, lddy, Q4MX_BF16), scale, rows, cols,
                                          dense(grad, ldg, dtype), add, ws, reinterpret_cast<hipStream_t>(stream)),
                    "embedding gradient launch");
}

q4_status q4nn_head_norm_rope(const q4nn_rope* r, const q4nn_heads* q, const q4nn_heads* k, const q4nn_heads* q_out,
                              const q4nn_heads* k_out, void* stream) {
    Q4_TRY(check_rope(r));
    Q4_TRY(check_heads("q", q, r, r->q_heads, false));
    Q4_TRY(check_heads("k", k, r, r->k_heads, false));
    Q4_TRY(check_heads("q_out", q_out, r, r->q_heads, true));
    Q4_TRY(check_heads("k_out", k_out, r, r->k_heads, true));
    if (shifted(q_out, q, r, r->q_heads) || shifted(k_out, k, r, r->k_heads))
        return bad(Q4_ERR_SHAPE, "an output in place of its input must have its strides");
    if (one_place(q_out, k_out, r)) return bad(Q4_ERR_CONFLICT, "q_out and k_out are one buffer");
    if (one_place(q_out, k, r) || one_place(q, k_out, r))
        return bad(Q4_ERR_CONFLICT, "an output is in the place of the other tensor's input");
    if (empty(r)) return ok();
    Q4_TRY(device());
    return launched(launch_head_norm_rope(*r, *q, *k, *q_out, *k_out, reinterpret_cast<hipStream_t>(stream)),
                    "head norm launch");
}

q4_status q4nn_head_norm_rope_backward_workspace_bytes(const q4nn_rope* r, size_t* bytes) {
    if (!bytes) return bad(Q4_ERR_INVALID_ARG, "output is NULL");
    Q4_TRY(check_rope(r));
    *bytes = empty(r) ? 0 : head_norm_rope_workspace(*r);
    return ok();
}

q4_status q4nn_head_norm_rope_backward(const q4nn_rope* r, const q4nn_heads* q, const q4nn_heads* k,
                                       const q4nn_heads* dq, const q4nn_heads* dk, const q4nn_heads* dq_in,
                                       const q4nn_heads* dk_in, void* dq_gain, void* dk_gain, int32_t dtype,
                                       int32_t flags, void* ws, size_t ws_bytes, void* stream) {
    Q4_TRY(check_flags(flags));
    size_t need = 0;
    Q4_TRY(q4nn_head_norm_rope_backward_workspace_bytes(r, &need));
    Q4_TRY(check_heads("q", q, r, r->q_heads, false));
    Q4_TRY(check_heads("k", k, r, r->k_heads, false));
    Q4_TRY(check_heads("dq", dq, r, r->q_heads, false));
    Q4_TRY(check_heads("dk", dk, r, r->k_heads, false));
    Q4_TRY(check_heads("dq_in", dq_in, r, r->q_heads, true));
    Q4_TRY(check_heads("dk_in", dk_in, r, r->k_heads, true));
    if (shifted(dq_in, dq, r, r->q_heads) || shifted(dq_in, q, r, r->q_heads) || shifted(dk_in, dk, r, r->k_heads) ||
        shifted(dk_in, k, r, r->k_heads))
        return bad(Q4_ERR_SHAPE, "a gradient in place of the result's or of the input must have its strides");
    if (one_place(dq_in, dk_in, r)) return bad(Q4_ERR_CONFLICT, "dq_in and dk_in are one buffer");
    if (one_place(dq_in, dk, r) || one_place(dq, dk_in, r) || one_place(dq_in, k, r) || one_place(q, dk_in, r))
        return bad(Q4_ERR_CONFLICT, "a gradient is in the place of the other tensor's operand");
    Q4_TRY(check_dense("dq_gain", dq_gain, dtype, 1, r->dim, r->dim));
    Q4_TRY(check_dense("dk_gain", dk_gain, dtype, 1, r->dim, r->dim));
    if (dq_gain == dk_gain) return bad(Q4_ERR_CONFLICT, "dq_gain and dk_gain are one buffer: add them up afterwards");
    const bool add = (flags & Q4NN_ADD) != 0;
    if (add && empty(r)) return ok();
    Q4_TRY(check_ws(ws, ws_bytes, need));
    Q4_TRY(device());
    return launched(launch_head_norm_rope_backward(*r, *q, *k, *dq, *dk, *dq_in, *dk_in, dq_gain, dk_gain, dtype, add,
                                                   ws, reinterpret_cast<hipStream_t>(stream)),
                    "head norm gradient launch");
}

q4_status q4nn_dropout(double p, uint64_t seed, uint64_t step, const uint64_t* step_at, uint32_t layer, int64_t offset,
                       const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t rows, int64_t cols,
                       void* out, int64_t ldo, int32_t dtype, void* stream) {
    if (!(p >= 0.0 && p <= 1.0)) return bad(Q4_ERR_INVALID_ARG, "p is outside [0, 1]");
    if (reinterpret_cast<uintptr_t>(step_at) & 7) return bad(Q4_ERR_ALIGNMENT, "step_at is not 8-byte aligned");
    Q4_TRY(check_dense("x", x, dtype, rows, cols, ldx));
    if (residual) Q4_TRY(check_dense("residual", residual, dtype, rows, cols, ldr));
    Q4_TRY(check_dense("out", out, dtype, rows, cols, ldo));
    constexpr int64_t kDraws = int64_t(1) << 35;  // 8 elements to a counter of 32 bits
    if (offset < 0 || offset % 8) return bad(Q4_ERR_SHAPE, "offset %lld is not a multiple of 8", (long long)offset);
    if (offset > kDraws || (rows > 0 && cols > 0 && rows > (kDraws - offset) / cols))
        return bad(Q4_ERR_SHAPE, "offset + rows * cols is more than 2^35");
    if ((out == x && rows > 1 && ldo != ldx) || (residual && out == residual && rows > 1 && ldo != ldr))
        return bad(Q4_ERR_SHAPE, "out in place of an operand must have its row stride");
    if (rows == 0 || cols == 0) return ok();
    Q4_TRY(device());
    Drop d;
    d.key0 = (uint32_t)seed, d.key1 = (uint32_t)(seed >> 32), d.step = (uint32_t)step, d.layer = layer;
    d.step_at = step_at;
    d.first = (uint32_t)(offset / 8);
    d.below = (uint32_t)std::nearbyint(p * 65536.0);
    d.scale = d.below < 65536u ? (float)(65536.0 / (65536.0 - d.below)) : 0.0f;
    return launched(launch_dropout(d, dense(x, ldx, dtype), dense(residual, ldr, dtype), rows, cols,
                                   dense(out, ldo, dtype), reinterpret_cast<hipStream_t>(stream)),
                    "dropout launch");
}

}  // extern "C"
