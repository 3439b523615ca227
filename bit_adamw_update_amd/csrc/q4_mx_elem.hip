// q4_mx_elem.hip -- quantization to and from the microscaled formats, and
// the activation functions that keep their input in 8 bits (gfx950).
//
// All of it streams memory: a few conversions per element, so HBM bounds it
// (checkpoint and restore of 8192 x 5632: 49 us, 280 MB at 5.7 TB/s; swiglu
// forward, backward and restore there: 172 us, 839 MB at 4.9 TB/s; a large
// copy 5.2).
// The conversions are the hardware's (v_cvt_scalef32_*): they divide or
// multiply by the block's power of two and round to nearest even in one
// instruction, exactly the format's definition.

#include "q4_mx.h"
#include "q4_mx_dev.h"

namespace q4 {
namespace {

// ---- row-wise tiles ---------------------------------------------------------
// A work-group takes 32 rows x 128 columns in two passes: lane s of a 16-lane
// row on columns 8s .. 8s+7, so a block of 32 is a quad of lanes, and a
// 128-column slice of a row is read as whole 256-byte (BF16) or 512-byte
// (FP32) runs; the 32 rows' scales of a slice are one 128-byte line.  The
// passes follow each other: both rows loaded first cost registers and are
// slower (swiglu 8192 x 5632 forward, backward and restore: 187 us against
// 172; 16 rows to a work-group: 177).
constexpr int kTileRows = 32;

struct Lane {
    int64_t row;
    int64_t col;  // first of the lane's 8 columns
};

__device__ __forceinline__ Lane lane_of(int64_t slices, int pass) {
    const uint32_t id = group_index(), rt = id / (uint32_t)slices, slice = id - rt * (uint32_t)slices;
    return Lane{(int64_t)rt * kTileRows + pass * 16 + (threadIdx.x >> 4), (int64_t)slice * 128 + (threadIdx.x & 15) * 8};
}

template <bool BF16> __global__ __launch_bounds__(256) void k_mx_quantize(const void* src, int64_t ld, MxMat out) {
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const Lane l = lane_of(out.slices, pass);
        if (l.row >= out.rows) return;
        float v[8];
        load8<BF16>(src, l.row * ld + l.col, out.cols - l.col, v);
        store_mx8(out, l.row, l.col, v);
    }
}

// The quantized transpose: blocks run along the source's rows.  A work-group
// takes 128 source rows x 64 source columns: lane c of wave b holds the 32
// rows of block b in column c (one block in registers, no exchange), reads 64
// consecutive elements a row, and the four blocks of a column leave together
// through shared memory as one run of a result row.  2560 x 10240 FP32 masters
// to E2M1: 19 us, 119 MB at 6.2 TB/s (part of it from the last-level cache).
template <bool BF16, int FMT>
__global__ __launch_bounds__(256) void k_mx_quantize_t(const void* src, int64_t ld, MxMat out, int64_t ctiles) {
    constexpr int kBytes = FMT == Q4MX_FP4 ? 16 : 32;  // codes of a block
    __shared__ __attribute__((aligned(16))) uint8_t lds[64][4 * kBytes + 16];
    __shared__ __attribute__((aligned(4))) uint8_t lds_scale[64][4];
    const uint32_t id = group_index(), st = id / (uint32_t)ctiles;
    const int64_t slice = st, c0 = (int64_t)(id - st * (uint32_t)ctiles) * 64;
    if (slice >= out.slices) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = slice * 128 + wave * 32, c = c0 + lane;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = (c < out.rows && r0 + i < out.cols) ? load1<BF16>(src, (r0 + i) * ld + c) : 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint32_t e = scale_byte<FMT>(top);
    const float s = scale_of(e);
    uint32_t w[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i)
        w[i] = e == 255 ? 0u : FMT == Q4MX_FP4 ? enc4x8(v + 8 * i, s) : enc8x4(v + 4 * i, s);
    uint32_t* dst = reinterpret_cast<uint32_t*>(&lds[lane][wave * kBytes]);
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) dst[i] = w[i];
    lds_scale[lane][wave] = (uint8_t)(r0 < out.cols ? e : 0);
    __syncthreads();
    constexpr int kPieces = kBytes * 4 / 16;  // 16-byte pieces of a column's run
    const int64_t pitch = out.slices * (FMT == Q4MX_FP4 ? 64 : 128);
    for (int i = threadIdx.x; i < 64 * kPieces; i += 256) {
        const int col = i / kPieces, piece = i % kPieces;
        if (c0 + col < out.rows)
            *reinterpret_cast<uint4*>(out.codes + (c0 + col) * pitch + slice * (4 * kBytes) + piece * 16) =
                *reinterpret_cast<const uint4*>(&lds[col][piece * 16]);
    }
    if (threadIdx.x < 64 && c0 + threadIdx.x < out.rows)
        *reinterpret_cast<uint32_t*>(out.scales + (slice * out.rows + c0 + threadIdx.x) * 4) =
            *reinterpret_cast<const uint32_t*>(lds_scale[threadIdx.x]);
}

template <bool BF16> __global__ __launch_bounds__(256) void k_mx_dequantize(MxMat a, void* dst, int64_t ld) {
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const Lane l = lane_of(a.slices, pass);
        if (l.row >= a.rows || l.col >= a.cols) return;
        float v[8];
        load_mx8(a, l.row, l.col, v);
        store8<BF16>(dst, l.row * ld + l.col, a.cols - l.col, v);
    }
}

// ---- activation functions ---------------------------------------------------
// 8192 x 5632, forward and backward: SwiGLU 73 and 76 us, GELU (tanh) 41 and 45
// (memory); GELU (erf) 71 and 83 (arithmetic: erfcf and an exponential).
//
// f(x) and f'(x).  With s = 1 / (1 + e^-t): x s for the gated unit (t = x) and
// for the tanh form, since 0.5 (1 + tanh u) = 1 / (1 + e^-2u).
struct ActValue {
    float f, d;
};

// 2^t for t <= 0, subnormal results included (the hardware's 2^t has none).
__device__ __forceinline__ float exp2_neg(float t) {
    const bool small = t < -126.0f;
    return __builtin_amdgcn_exp2f(small ? t + 64.0f : t) * (small ? 5.421010862427522e-20f : 1.0f);
}

// 1 / (1 + e^-t), by e^-|t|, which does not overflow: for t < -88, where e^-t
// would, the result is still a number that BF16 holds.
__device__ __forceinline__ float sigmoid(float t) {
    const float e = exp2_neg(-1.4426950408889634f * __builtin_fabsf(t));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    return t < 0.0f ? e * r : r;
}

template <int ACT> __device__ __forceinline__ ActValue act_value(float x) {
    if (ACT == Q4MX_SWIGLU) {
        const float s = sigmoid(x);
        return {x * s, s * __builtin_fmaf(x, 1.0f - s, 1.0f)};
    }
    if (ACT == Q4MX_GELU) {
        // 2u = 2 sqrt(2/pi) (x + 0.044715 x^3); f' = s + x s (1 - s) (2u)'.
        // Past |x| = 16, |2u| > 300: s is 0 or 1 and f' is s, so x is held there
        // (a NaN is not) and its powers stay finite.
        const float a = 1.5957691216057308f, b = 0.07135481627260f;
        const float c = x > 16.0f ? 16.0f : x < -16.0f ? -16.0f : x, c2 = c * c;
        const float s = sigmoid(c * __builtin_fmaf(b, c2, a));
        return {x * s, s * __builtin_fmaf(c * (1.0f - s), __builtin_fmaf(3.0f * b, c2, a), 1.0f)};
    }
    // 0.5 erfc(-x / sqrt 2) keeps the small values of negative x
    const float p = 0.5f * erfcf(-0.7071067811865476f * x);
    const float n = 0.3989422804014327f * exp2_neg(-0.7213475204444817f * x * x);
    return {x * p, __builtin_fmaf(x, n, p)};
}

template <int ACT>
__global__ __launch_bounds__(256) void k_act_forward(const void* x, int64_t ldx, const void* up, int64_t ldup,
                                                      int64_t rows, int64_t cols, int64_t slices, void* y, int64_t ldy,
                                                      MxMat ymx, MxMat kx, MxMat ku) {
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const Lane l = lane_of(slices, pass);
        if (l.row >= rows) return;
        const int64_t left = cols - l.col;
        float v[8], u[8], r[8];
        load8<true>(x, l.row * ldx + l.col, left, v);
        if (ACT == Q4MX_SWIGLU) load8<true>(up, l.row * ldup + l.col, left, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = act_value<ACT>(v[i]).f;
            if (ACT == Q4MX_SWIGLU) r[i] *= u[i];
            r[i] = round_bf16(r[i]);
        }
        if (y && left > 0) store8<true>(y, l.row * ldy + l.col, left, r);
        if (ymx.codes) store_mx8(ymx, l.row, l.col, r);
        if (kx.codes) store_mx8(kx, l.row, l.col, v);
        if (ACT == Q4MX_SWIGLU && ku.codes) store_mx8(ku, l.row, l.col, u);
    }
}

template <int ACT>
__global__ __launch_bounds__(256) void k_act_backward(MxMat kx, MxMat ku, const void* dy, int64_t lddy, void* dx,
                                                       int64_t lddx, void* dup, int64_t lddup) {
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const Lane l = lane_of(kx.slices, pass);
        const int64_t left = kx.cols - l.col;
        if (l.row >= kx.rows || left <= 0) return;
        float g[8], v[8], u[8], a[8], b[8];
        load8<true>(dy, l.row * lddy + l.col, left, g);
        load_mx8(kx, l.row, l.col, v);
        if (ACT == Q4MX_SWIGLU) load_mx8(ku, l.row, l.col, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const ActValue t = act_value<ACT>(v[i]);
            a[i] = ACT == Q4MX_SWIGLU ? g[i] * u[i] * t.d : g[i] * t.d;
            b[i] = g[i] * t.f;
        }
        store8<true>(dx, l.row * lddx + l.col, left, a);
        if (ACT == Q4MX_SWIGLU) store8<true>(dup, l.row * lddup + l.col, left, b);
    }
}

int64_t row_tiles(int64_t rows, int64_t slices) { return (rows + kTileRows - 1) / kTileRows * slices; }

}  // namespace

hipError_t launch_mx_quantize(const Dense& src, bool transpose, const MxMat& out, hipStream_t st) {
    const bool bf = src.dtype == Q4MX_BF16;
    if (transpose) {
        const int64_t ctiles = (out.rows + 63) / 64;
        const dim3 g = grid_of(ctiles * out.slices), b(256);
        if (bf && out.fmt == Q4MX_FP4) k_mx_quantize_t<true, Q4MX_FP4><<<g, b, 0, st>>>(src.p, src.ld, out, ctiles);
        else if (bf) k_mx_quantize_t<true, Q4MX_FP8><<<g, b, 0, st>>>(src.p, src.ld, out, ctiles);
        else if (out.fmt == Q4MX_FP4) k_mx_quantize_t<false, Q4MX_FP4><<<g, b, 0, st>>>(src.p, src.ld, out, ctiles);
        else k_mx_quantize_t<false, Q4MX_FP8><<<g, b, 0, st>>>(src.p, src.ld, out, ctiles);
        return hipGetLastError();
    }
    const dim3 g = grid_of(row_tiles(out.rows, out.slices)), b(256);
    if (bf) k_mx_quantize<true><<<g, b, 0, st>>>(src.p, src.ld, out);
    else k_mx_quantize<false><<<g, b, 0, st>>>(src.p, src.ld, out);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxMat& a, const Dense& dst, hipStream_t st) {
    const dim3 g = grid_of(row_tiles(a.rows, a.slices)), b(256);
    if (dst.dtype == Q4MX_BF16) k_mx_dequantize<true><<<g, b, 0, st>>>(a, dst.p, dst.ld);
    else k_mx_dequantize<false><<<g, b, 0, st>>>(a, dst.p, dst.ld);
    return hipGetLastError();
}

hipError_t launch_act_forward(int act, const Dense& x, const Dense& up, int64_t rows, int64_t cols, const Dense& y,
                              const MxMat& y_mx, const MxMat& kx, const MxMat& ku, hipStream_t st) {
    const int64_t slices = (cols + kMxPad - 1) / kMxPad;
    const dim3 g = grid_of(row_tiles(rows, slices)), b(256);
#define Q4_ACT_FWD(A) \
    k_act_forward<A><<<g, b, 0, st>>>(x.p, x.ld, up.p, up.ld, rows, cols, slices, y.p, y.ld, y_mx, kx, ku)
    if (act == Q4MX_GELU) Q4_ACT_FWD(Q4MX_GELU);
    else if (act == Q4MX_GELU_ERF) Q4_ACT_FWD(Q4MX_GELU_ERF);
    else Q4_ACT_FWD(Q4MX_SWIGLU);
#undef Q4_ACT_FWD
    return hipGetLastError();
}

hipError_t launch_act_backward(int act, const MxMat& kx, const MxMat& ku, const Dense& dy, const Dense& dx,
                               const Dense& dup, hipStream_t st) {
    const dim3 g = grid_of(row_tiles(kx.rows, kx.slices)), b(256);
#define Q4_ACT_BWD(A) k_act_backward<A><<<g, b, 0, st>>>(kx, ku, dy.p, dy.ld, dx.p, dx.ld, dup.p, dup.ld)
    if (act == Q4MX_GELU) Q4_ACT_BWD(Q4MX_GELU);
    else if (act == Q4MX_GELU_ERF) Q4_ACT_BWD(Q4MX_GELU_ERF);
    else Q4_ACT_BWD(Q4MX_SWIGLU);
#undef Q4_ACT_BWD
    return hipGetLastError();
}

}  // namespace q4
