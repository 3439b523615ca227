// q4_nn.h -- shared by the host entry points (q4_nn_abi.cpp) and the kernels
// (q4_nn_embed.hip, q4_nn_heads.hip, q4_nn_dropout.hip) of embedding, head
// norms and dropout.  Not part of the public C ABI.
#pragma once

#include "q4_mx.h"

namespace q4 {

// Token numbers in device memory.
struct Ids {
    const void* p;
    int64_t n;
    int type;  // q4nn_int
};

hipError_t launch_embedding(const Ids& ids, const Dense& table, const MxMat& mx, int64_t rows, int64_t cols,
                            float scale, const Dense& out, hipStream_t st);  // mx: if its codes are not NULL
size_t embedding_grad_workspace(int64_t tokens, int64_t cols);
hipError_t launch_embedding_grad(const Ids& ids, const Dense& dy, float scale, int64_t rows, int64_t cols,
                                 const Dense& grad, bool add, void* ws, hipStream_t st);

size_t head_norm_rope_workspace(const q4nn_rope& r);
hipError_t launch_head_norm_rope(const q4nn_rope& r, const q4nn_heads& q, const q4nn_heads& k, const q4nn_heads& qo,
                                 const q4nn_heads& ko, hipStream_t st);
// gq, gk: the gains' gradients (dtype), added to if add.
hipError_t launch_head_norm_rope_backward(const q4nn_rope& r, const q4nn_heads& q, const q4nn_heads& k,
                                          const q4nn_heads& dq, const q4nn_heads& dk, const q4nn_heads& dq_in,
                                          const q4nn_heads& dk_in, void* gq, void* gk, int dtype, bool add, void* ws,
                                          hipStream_t st);

// What dropout draws from, and what it does with a kept element.
struct Drop {
    uint32_t key0, key1, step, layer;
    const uint64_t* step_at;  // device, or NULL
    uint32_t first;           // offset / 8
    uint32_t below;           // dropped if the 16 bits are below this
    float scale;
};
hipError_t launch_dropout(const Drop& d, const Dense& x, const Dense& residual, int64_t rows, int64_t cols,
                          const Dense& out, hipStream_t st);

}  // namespace q4
