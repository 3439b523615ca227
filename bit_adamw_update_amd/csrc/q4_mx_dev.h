// q4_mx_dev.h -- device primitives of the microscaled formats: a block's
// scale, the conversions between codes and FP32, and 8-element accesses of
// dense and MX matrices.
#pragma once

#include "q4_mx.h"

namespace q4 {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

// The work-group's number in a grid_of grid.
__device__ __forceinline__ uint32_t group_index() { return blockIdx.y * gridDim.x + blockIdx.x; }

// 2^(e-127): the FP32 with that biased exponent, subnormal for e = 0.  For e
// = 255 the bits are those of an infinity; the conversions read the exponent
// field alone and give NaN.
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(max(e << 23, 0x00400000u)); }

// The scale byte of a block whose largest magnitude has the bits `top`: the
// smallest e >= 0 with |x| 2^(127-e) <= 6 = 1.5 2^2 (E2M1) or 448 = 1.75 2^8
// (E4M3).  NaN and infinite inputs have the largest bits.
template <int FMT> __device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    constexpr int kExp = FMT == Q4MX_FP4 ? 2 : 8;
    constexpr uint32_t kMan = FMT == Q4MX_FP4 ? 0x400000u : 0x600000u;
    if (top >= 0x7F800000u) return 255;
    const int e = (int)(top >> 23) - kExp + ((top & 0x7FFFFFu) > kMan ? 1 : 0);
    return e < 0 ? 0 : (uint32_t)e;
}

// 8 values to 8 E2M1 codes, 4 values to 4 E4M3 codes.
__device__ __forceinline__ uint32_t enc4x8(const float* v, float s) {
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}
__device__ __forceinline__ uint32_t enc8x4(const float* v, float s) {
    union {
        s16x2 h;
        uint32_t u;
    } w;
    w.u = 0;
    w.h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w.h, v[0], v[1], s, false);
    w.h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w.h, v[2], v[3], s, true);
    return w.u;
}

__device__ __forceinline__ void dec4x8(uint32_t w, float s, float* v) {
    f32x2 t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    v[0] = t[0], v[1] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    v[2] = t[0], v[3] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
    v[4] = t[0], v[5] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    v[6] = t[0], v[7] = t[1];
}
__device__ __forceinline__ void dec8x4(uint32_t w, float s, float* v) {
    f32x2 t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false);
    v[0] = t[0], v[1] = t[1];
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
    v[2] = t[0], v[3] = t[1];
}

// FP32 to BF16, to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float x) {
    union {
        __bf16 b;
        uint16_t u;
    } t;
    t.b = (__bf16)x;
    return t.u;
}
__device__ __forceinline__ float bf16_value(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float round_bf16(float x) { return bf16_value(bf16_bits(x)); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return (uint32_t)bf16_bits(lo) | ((uint32_t)bf16_bits(hi) << 16);
}

template <bool BF16> __device__ __forceinline__ float load1(const void* p, int64_t i) {
    return BF16 ? bf16_value(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Vectors at any element's alignment: the memory path takes them whole.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// 8 elements from index i, of which the first `left` exist (the others read
// as 0).
template <bool BF16> __device__ __forceinline__ void load8(const void* p, int64_t i, int64_t left, float* v) {
    if (left >= 8) {
        if (BF16) {
            const u32x4_any q = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = bf16_value(q[k] & 0xFFFFu);
                v[2 * k + 1] = __uint_as_float(q[k] & 0xFFFF0000u);
            }
        } else {
            const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
            const f32x4_any a = q[0], b = q[1];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = a[k], v[4 + k] = b[k];
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < left ? load1<BF16>(p, i + k) : 0.0f;
}

template <bool BF16> __device__ __forceinline__ void store8(void* p, int64_t i, int64_t left, const float* v) {
    if (left >= 8) {
        if (BF16) {
            *reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(p) + i) =
                u32x4_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
        } else {
            f32x4_any* q = reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + i);
            q[0] = f32x4_any{v[0], v[1], v[2], v[3]};
            q[1] = f32x4_any{v[4], v[5], v[6], v[7]};
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) {
            if (BF16) static_cast<uint16_t*>(p)[i + k] = bf16_bits(v[k]);
            else static_cast<float*>(p)[i + k] = v[k];
        }
}

// Maximum over a quad of lanes (4 consecutive lanes: one block of 32).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// The codes of 8 values in columns col .. col+7 of a row (values past the
// last column are 0), and the block's scale.  The four lanes of a quad hold
// one block and call together.
template <int FMT> __device__ __forceinline__ void store_mx8_as(const MxMat& m, int64_t row, int64_t col, const float* v) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    const uint32_t e = scale_byte<FMT>(quad_max(top));
    const float s = scale_of(e);
    if (FMT == Q4MX_FP4) {
        *reinterpret_cast<uint32_t*>(m.codes + row * (m.slices * 64) + col / 2) = e == 255 ? 0u : enc4x8(v, s);
    } else {
        *reinterpret_cast<uint2*>(m.codes + row * (m.slices * 128) + col) =
            e == 255 ? make_uint2(0, 0) : make_uint2(enc8x4(v, s), enc8x4(v + 4, s));
    }
    if ((threadIdx.x & 3) == 0) m.scales[((col >> 7) * m.rows + row) * 4 + ((col >> 5) & 3)] = (uint8_t)e;
}
__device__ __forceinline__ void store_mx8(const MxMat& m, int64_t row, int64_t col, const float* v) {
    if (m.fmt == Q4MX_FP4) store_mx8_as<Q4MX_FP4>(m, row, col, v);
    else store_mx8_as<Q4MX_FP8>(m, row, col, v);
}

__device__ __forceinline__ void load_mx8(const MxMat& m, int64_t row, int64_t col, float* v) {
    const float s = scale_of(m.scales[((col >> 7) * m.rows + row) * 4 + ((col >> 5) & 3)]);
    if (m.fmt == Q4MX_FP4) {
        dec4x8(*reinterpret_cast<const uint32_t*>(m.codes + row * (m.slices * 64) + col / 2), s, v);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(m.codes + row * (m.slices * 128) + col);
        dec8x4(w.x, s, v);
        dec8x4(w.y, s, v + 4);
    }
}

}  // namespace
}  // namespace q4
