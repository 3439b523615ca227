// q4_nn_dropout.hip -- dropout whose mask is drawn anew wherever it is needed
// (gfx950).
//
// y = keep ? x / (1 - p) : 0, plus a residual.  One Philox4x32-10 call gives
// 128 bits, 16 to an element, so a lane takes 8 consecutive elements: one
// 16-byte BF16 access each way.  p on a grid of 2^-16 is what 16 bits give
// (the scale uses that p, so the expectation is exact); 32 bits to an element
// would double the generator's work, which takes half of the VALU's time now.
// Memory bounds it: 8192 x 2560 in BF16 15 us, 84 MB at 5.6 TB/s, with a residual
// 21 us, 126 MB at 6.0.  Rows with a gap between them: 25 where rows that follow
// each other take 24 (from memory alone), in FP32 47 and 44.
#include "q4_exact.h"
#include "q4_mx_dev.h"
#include "q4_nn.h"

namespace q4 {
namespace {

constexpr uint32_t kDropStream = 2;  // Philox counter word: 0 and 1 are the optimizer's

// Element i of the row-major matrix is at row i / cols, column i % cols.
// FLAT: rows follow each other without a gap in every operand, so i itself is
// the offset.  Otherwise a run of 8 elements may cross a row's end.
template <bool BF16, bool FLAT>
__global__ __launch_bounds__(256) void k_dropout(Drop d, const void* x, int64_t ldx, const void* res, int64_t ldr,
                                                  void* out, int64_t ldo, int64_t n, int64_t cols) {
    const int64_t g = (int64_t)group_index() * 256 + threadIdx.x, i = g * 8;
    if (i >= n) return;
    const uint32_t step = d.step_at ? (uint32_t)*d.step_at : d.step;
    const PhiloxFixed f = philox_fixed(step, d.layer, d.key0, d.key1);
    const uint4 w = philox_from(d.first + (uint32_t)g, kDropStream, f, d.key0, d.key1);
    const uint32_t bits[4] = {w.x, w.y, w.z, w.w};
    float v[8], r[8];
    int64_t row = 0, col = i;
    if (!FLAT) row = i / cols, col = i - row * cols;
    const bool whole = FLAT || col + 8 <= cols;
    const int64_t left = n - i < 8 ? n - i : 8;
    if (whole) {
        load8<BF16>(x, row * ldx + col, left, v);
        if (res) load8<BF16>(res, row * ldr + col, left, r);
    } else {
        int64_t rr = row, cc = col;
        for (int k = 0; k < 8; ++k) {
            v[k] = k < left ? load1<BF16>(x, rr * ldx + cc) : 0.0f;
            r[k] = res && k < left ? load1<BF16>(res, rr * ldr + cc) : 0.0f;
            if (++cc == cols) cc = 0, ++rr;
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const bool drop = ((bits[k / 2] >> (16 * (k & 1))) & 0xFFFFu) < d.below;
        // chosen, not multiplied: a dropped NaN is 0 too
        v[k] = drop ? 0.0f : v[k] * d.scale;
        if (res) v[k] += r[k];
    }
    if (whole) {
        store8<BF16>(out, row * ldo + col, left, v);
    } else {
        for (int k = 0; k < 8; ++k) {
            if (k < left) {
                if (BF16) static_cast<uint16_t*>(out)[row * ldo + col] = bf16_bits(v[k]);
                else static_cast<float*>(out)[row * ldo + col] = v[k];
            }
            if (++col == cols) col = 0, ++row;
        }
    }
}

}  // namespace

hipError_t launch_dropout(const Drop& d, const Dense& x, const Dense& residual, int64_t rows, int64_t cols,
                          const Dense& out, hipStream_t st) {
    const int64_t n = rows * cols;
    const dim3 g = grid_of((n + 2047) / 2048), b(256);
    const bool flat = rows == 1 || (x.ld == cols && out.ld == cols && (!residual.p || residual.ld == cols));
#define Q4_DROP(BF, F) \
    k_dropout<BF, F><<<g, b, 0, st>>>(d, x.p, x.ld, residual.p, residual.ld, out.p, out.ld, n, cols)
    if (x.dtype == Q4MX_BF16 && flat) Q4_DROP(true, true);
    else if (x.dtype == Q4MX_BF16) Q4_DROP(true, false);
    else if (flat) Q4_DROP(false, true);
    else Q4_DROP(false, false);
#undef Q4_DROP
    return hipGetLastError();
}

}  // namespace q4
