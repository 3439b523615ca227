// q4_mx_gemm.hip -- the three products of the microscaled linear layer
// (gfx950).
//
// Every code value is exact in BF16 (E2M1 has one fraction bit, E4M3 three,
// and scales are powers of two), so all three products are sums of BF16
// products in FP32 on the matrix cores.

#include "q4_mx.h"
#include "q4_mx_dev.h"

namespace q4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// An operand: element (row, k) of `rows` x `depth`.
struct Operand {
    const void* p;  // dense BF16
    MxMat mx;       // or codes (p == NULL)
    int64_t rows, depth;
    int64_t sr, sk;  // dense strides
    bool turned;     // MX: row is the MX column
};

__device__ __forceinline__ uint16_t element(const Operand& a, int64_t row, int64_t k) {
    if (row >= a.rows || k >= a.depth) return 0;
    if (a.p) return static_cast<const uint16_t*>(a.p)[row * a.sr + k * a.sk];
    const int64_t r = a.turned ? k : row, c = a.turned ? row : k;
    const float s = scale_of(a.mx.scales[((c >> 7) * a.mx.rows + r) * 4 + ((c >> 5) & 3)]);
    float v[8];
    if (a.mx.fmt == Q4MX_FP4) {
        dec4x8(a.mx.codes[r * a.mx.slices * 64 + c / 2], s, v);
        return bf16_bits(v[c & 1]);
    }
    dec8x4(a.mx.codes[r * a.mx.slices * 128 + c], s, v);
    return bf16_bits(v[0]);
}

struct Result {
    void* p;
    int64_t sm, sn;  // element (m, n) at p[m * sm + n * sn]
    int dtype;
    bool add;
};

// 64 x 64 results per work-group of four wavefronts, 32 deep per step.
__global__ __launch_bounds__(256) void k_mx_product(Operand a, Operand b, Result out, int64_t ntiles) {
    __shared__ __attribute__((aligned(16))) uint16_t la[64][40], lb[64][40];
    const int64_t m0 = blockIdx.x / ntiles * 64, n0 = blockIdx.x % ntiles * 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sr = threadIdx.x >> 2, sk = (threadIdx.x & 3) * 8;
    f32x4 acc[4] = {};
    for (int64_t k0 = 0; k0 < a.depth; k0 += 32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            la[sr][sk + j] = element(a, m0 + sr, k0 + sk + j);
            lb[sr][sk + j] = element(b, n0 + sr, k0 + sk + j);
        }
        __syncthreads();
        const bf16x8 x = *reinterpret_cast<const bf16x8*>(&la[wave * 16 + (lane & 15)][(lane >> 4) * 8]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 y = *reinterpret_cast<const bf16x8*>(&lb[j * 16 + (lane & 15)][(lane >> 4) * 8]);
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, acc[j], 0, 0, 0);
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + wave * 16 + (lane >> 4) * 4 + i, n = n0 + j * 16 + (lane & 15);
            if (m >= a.rows || n >= b.rows) continue;
            const int64_t at = m * out.sm + n * out.sn;
            float v = acc[j][i];
            if (out.dtype == Q4MX_BF16) {
                uint16_t* p = static_cast<uint16_t*>(out.p) + at;
                if (out.add) v += bf16_value(*p);
                *p = bf16_bits(v);
            } else {
                float* p = static_cast<float*>(out.p) + at;
                if (out.add) v += *p;
                *p = v;
            }
        }
}

hipError_t product(const Operand& a, const Operand& b, const Result& out, hipStream_t st) {
    const int64_t mt = (a.rows + 63) / 64, nt = (b.rows + 63) / 64;
    k_mx_product<<<dim3((unsigned)(mt * nt)), dim3(256), 0, st>>>(a, b, out, nt);
    return hipGetLastError();
}

Operand dense(const Dense& d, int64_t rows, int64_t depth, bool turned) {
    return Operand{d.p, MxMat{}, rows, depth, turned ? 1 : d.ld, turned ? d.ld : 1, false};
}
Operand codes(const MxMat& m, bool turned) {
    return Operand{nullptr, m, turned ? m.cols : m.rows, turned ? m.rows : m.cols, 0, 0, turned};
}

}  // namespace

hipError_t launch_linear(const MxMat& x, const MxMat& w, const Dense& y, hipStream_t st) {
    return product(codes(x, false), codes(w, false), Result{y.p, y.ld, 1, y.dtype, false}, st);
}

hipError_t launch_dgrad(const Dense& dy, int64_t tokens, const MxMat& w, const Dense& dx, hipStream_t st) {
    return product(dense(dy, tokens, w.rows, false), codes(w, true), Result{dx.p, dx.ld, 1, dx.dtype, false}, st);
}

hipError_t launch_wgrad(const Dense& dy, int64_t n, const MxMat& x, const Dense& dw, bool transposed, bool add,
                        hipStream_t st) {
    return product(dense(dy, n, x.rows, true), codes(x, true),
                   Result{dw.p, transposed ? 1 : dw.ld, transposed ? dw.ld : 1, dw.dtype, add}, st);
}

}  // namespace q4
