// q4_mx.h -- shared by the host entry points (q4_mx_abi.cpp) and the kernels
// (q4_mx_elem.hip, q4_mx_gemm.hip) of the microscaled linear layer.  Not
// part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/q4adamw.h"

namespace q4 {

constexpr int64_t kMxPad = 128;  // columns of a row are padded to this many

// An MX matrix as the kernels see it.
struct MxMat {
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows, cols;
    int64_t slices;  // P / 128
    int fmt;         // q4mx_format
};

// A dense row-major matrix: element (r, c) at p[r * ld + c].
struct Dense {
    void* p;
    int64_t ld;
    int dtype;  // q4mx_dtype
};

// The grid of n work-groups of up to 512 threads.  A launch takes fewer than
// 2^32 threads along a dimension (it refuses 2^32 and drops what is above), so
// groups past 2^22 go into rows; the last row may have more than n groups.
inline dim3 grid_of(int64_t n) {
    constexpr int64_t kRow = int64_t(1) << 22;
    return n <= kRow ? dim3((unsigned)n) : dim3((unsigned)kRow, (unsigned)((n + kRow - 1) / kRow));
}

hipError_t launch_mx_quantize(const Dense& src, bool transpose, const MxMat& out, hipStream_t st);
hipError_t launch_mx_dequantize(const MxMat& a, const Dense& dst, hipStream_t st);
// y, y_mx, kx, ku: absent where their pointer (codes) is NULL.
hipError_t launch_act_forward(int act, const Dense& x, const Dense& up, int64_t rows, int64_t cols, const Dense& y,
                              const MxMat& y_mx, const MxMat& kx, const MxMat& ku, hipStream_t st);
hipError_t launch_act_backward(int act, const MxMat& kx, const MxMat& ku, const Dense& dy, const Dense& dx,
                               const Dense& dup, hipStream_t st);

// Whether dy (rows x cols) must be copied into 16-byte aligned rows of whole
// 8-element pieces first, and the bytes of that copy.
bool dense_needs_copy(const Dense& d, int64_t rows, int64_t cols);
size_t dense_copy_bytes(int64_t rows, int64_t cols);

// Workspaces of the products: the sums of tiles that are split along the sum.
size_t linear_workspace(const MxMat& x, const MxMat& w);
size_t grad_workspace(const MxMat& m, int64_t width);  // m: w (width: tokens) or x (width: n)

// The three products.  add: the result is added to what out holds.  copy: room
// for the copy of dy, if it needs one.
hipError_t launch_linear_few(const Dense& x, int64_t tokens, const MxMat& w, const Dense& y, hipStream_t st);  // BF16 x
hipError_t launch_linear(const MxMat& x, const MxMat& w, const Dense& y, void* ws, hipStream_t st);
hipError_t launch_dgrad(const Dense& dy, int64_t tokens, const MxMat& w, const Dense& dx, void* copy, void* ws,
                        hipStream_t st);
hipError_t launch_wgrad(const Dense& dy, int64_t n, const MxMat& x, const Dense& dw, bool transposed, bool add,
                        void* copy, void* ws, hipStream_t st);

}  // namespace q4
