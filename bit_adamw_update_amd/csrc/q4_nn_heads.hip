// q4_nn_heads.hip -- the norm of queries and keys over each head and their
// rotation by position, in one pass, and its gradients (gfx950).
//
// A row is one head of one token: dim elements, consecutive.  Memory bounds
// both directions (4 bytes an element forward, 6 backward), so a row is read
// once, held in registers by a few lanes, and written once: its sums are
// exchanged between those lanes without shared memory.  The unit of work is a
// pair of elements that turn together; a lane takes VEC neighbouring pairs in
// two vectors (the halves' (i, i + rotary/2), or 2 VEC neighbours when pairs
// are interleaved), so the rotation needs no exchange.  Elements past `rotary`
// pair up the same way, with the angle 0.
//
// The angles of a token are those of all its heads, and FP64: a work-group
// forms the cosines and sines of its tokens once, in shared memory.
#include "q4_mx_dev.h"
#include "q4_nn.h"

namespace q4 {
namespace {

constexpr int kTokens = 16, kAngles = 2048;  // most tokens and angles of a work-group
constexpr int kMaxGroups = 1024;             // of a backward pass: each leaves one sum of the gains' gradients

struct HeadsArgs {
    q4nn_heads v[6];  // q, k, dq, dk, q_out, k_out (backward: dq_in, dk_in)
    const void *positions, *gain[2];
    const double* frequencies;
    int64_t position_batch, position_token, total, per_batch, blocks;
    int heads[2];
    uint32_t magic[2];  // ceil(2^32 / heads)
    int dim, half, pairs, log_lanes, tokens;
    bool positions_wide, gain_bf16;
    float eps, inv_dim;
    float* part;  // [work-groups][2][dim]
};

// Cosine and sine of `a` radians.  FP64 brings the angle to a quarter turn and
// its remainder within +-1/8 turn, which FP32 holds to half a step; there the
// Taylor polynomials to x^9 and x^10 are off by less than 2^-29.
__device__ __forceinline__ float2 cos_sin(double a) {
    const double quarters = a * 0.63661977236758134308;  // 2 / pi
    const double q = __builtin_rint(quarters);
    // the remainder in radians: a multiply-add keeps what the product alone loses of a far angle
    const double r = __builtin_fma(q, -1.57079632679489661923, a);
    const float x = (float)__builtin_fma(q, -6.123233995736766036e-17, r), z = x * x;
    float s = __builtin_fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    s = __builtin_fmaf(z, s, 8.3333333e-3f);
    s = __builtin_fmaf(z, s, -0.16666667f);
    s = __builtin_fmaf(x * z, s, x);
    float c = __builtin_fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    c = __builtin_fmaf(z, c, -1.3888889e-3f);
    c = __builtin_fmaf(z, c, 4.1666667e-2f);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.0f);
    const int n = (int)(q - 4.0 * __builtin_floor(q * 0.25));  // q mod 4
    const float cc = (n & 1) ? s : c, ss = (n & 1) ? c : s;
    return make_float2((n == 1 || n == 2) ? -cc : cc, n >= 2 ? -ss : ss);
}

// Sum over the 2^log_lanes neighbouring lanes of a row.
__device__ __forceinline__ float row_sum(float x, int log_lanes) {
#define Q4_ADD_DPP(ctrl) \
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, 0xF, 0xF, true))
    if (log_lanes > 0) Q4_ADD_DPP(0xB1);   // lanes 1 0 3 2
    if (log_lanes > 1) Q4_ADD_DPP(0x4E);   // lanes 2 3 0 1
    if (log_lanes > 2) Q4_ADD_DPP(0x141);  // the other quad of 8
    if (log_lanes > 3) Q4_ADD_DPP(0x140);  // the other 8 of 16
#undef Q4_ADD_DPP
    if (log_lanes > 4) x += __shfl_xor(x, 16);
    if (log_lanes > 5) x += __shfl_xor(x, 32);
    return x;
}

// VEC elements of a dense BF16 or FP32 run.
template <int VEC, bool BF16> __device__ __forceinline__ void load_vec(const void* p, int64_t i, float* v) {
    if (VEC == 8) {
        load8<BF16>(p, i, 8, v);
    } else if (VEC == 4 && BF16) {
        const u32x2_any q = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(p) + i);
        v[0] = bf16_value(q[0] & 0xFFFFu), v[1] = __uint_as_float(q[0] & 0xFFFF0000u);
        v[2] = bf16_value(q[1] & 0xFFFFu), v[3] = __uint_as_float(q[1] & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = load1<BF16>(p, i + k);
    }
}
template <int VEC> __device__ __forceinline__ void store_vec(uint16_t* p, int64_t i, const float* v) {
    if (VEC == 8) {
        store8<true>(p, i, 8, v);
    } else if (VEC == 4) {
        *reinterpret_cast<u32x2_any*>(p + i) = u32x2_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) p[i + k] = bf16_bits(v[k]);
    }
}

// Where a lane's VEC pairs from pair u on lie: two vectors at e[0] and e[1].
// INTER: pairs are neighbours.  Else the halves of the rotary part, behind it
// the halves of the rest.
template <int VEC, bool INTER> struct Place {
    int e[2];
    __device__ __forceinline__ Place(const HeadsArgs& a, int u) {
        if (INTER) e[0] = 2 * u, e[1] = 2 * u + VEC;
        else if (u < a.half) e[0] = u, e[1] = u + a.half;
        else e[0] = u + a.half, e[1] = u + a.pairs;
    }
};
// The pairs' first and second elements of two vectors, and back.
template <int VEC, bool INTER> __device__ __forceinline__ void split_pairs(const float* v, float* p, float* s) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) p[k] = v[INTER ? 2 * k : k], s[k] = v[INTER ? 2 * k + 1 : VEC + k];
}
template <int VEC, bool INTER> __device__ __forceinline__ void join_pairs(const float* p, const float* s, float* v) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[INTER ? 2 * k : k] = p[k], v[INTER ? 2 * k + 1 : VEC + k] = s[k];
}

// The rows of `which` (0: q, 1: k) of a work-group's tokens; K vectors of
// pairs to a lane.  acc: the gain's gradient, pairs' first elements and second.
template <int VEC, int K, bool INTER, bool BACK>
__device__ __forceinline__ void rows_of(const HeadsArgs& a, int which, int tokens, const float2* angles,
                                        const int64_t (*at)[6], float (*acc)[2 * VEC]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lanes = 1 << a.log_lanes;
    const int sub = lane & (lanes - 1), per_wave = 64 >> a.log_lanes;
    const int heads = a.heads[which], rows = tokens * heads;
    if (rows == 0) return;
    const q4nn_heads &in = a.v[which], &grad = a.v[2 + which], &out = a.v[4 + which];
    float gp[K][VEC], gs[K][VEC];
#pragma unroll
    for (int c = 0; c < K; ++c) {
        const int u = (c * lanes + sub) * VEC;
        if (u >= a.pairs) break;
        const Place<VEC, INTER> e(a, u);
        float v[2 * VEC];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (a.gain_bf16) load_vec<VEC, true>(a.gain[which], e.e[h], v + h * VEC);
            else load_vec<VEC, false>(a.gain[which], e.e[h], v + h * VEC);
        }
        split_pairs<VEC, INTER>(v, gp[c], gs[c]);
    }
    // q's rows go to the first waves first, k's to the last
    for (int r = (which ? 3 - wave : wave) * per_wave + (lane >> a.log_lanes); r < rows; r += 4 * per_wave) {
        // r / heads: the reciprocal is less than heads 2^-32 of itself too large, and r < 16 * 4096: r heads < 2^32
        const int tok = heads == 1 ? r : (int)__umulhi((uint32_t)r, a.magic[which]), head = r - tok * heads;
        const uint16_t* x = in.p + at[tok][which] + head * in.head;
        const uint16_t* dy = BACK ? grad.p + at[tok][2 + which] + head * grad.head : nullptr;
        uint16_t* y = out.p + at[tok][4 + which] + head * out.head;
        float xp[K][VEC], xs[K][VEC], dp[K][VEC], ds[K][VEC], sum = 0.0f;
#pragma unroll
        for (int c = 0; c < K; ++c) {
            const int u = (c * lanes + sub) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) xp[c][k] = xs[c][k] = dp[c][k] = ds[c][k] = 0.0f;
            if (u >= a.pairs) continue;
            const Place<VEC, INTER> e(a, u);
            float v[2 * VEC];
            load_vec<VEC, true>(x, e.e[0], v);
            load_vec<VEC, true>(x, e.e[1], v + VEC);
            split_pairs<VEC, INTER>(v, xp[c], xs[c]);
            if (BACK) {
                load_vec<VEC, true>(dy, e.e[0], v);
                load_vec<VEC, true>(dy, e.e[1], v + VEC);
                split_pairs<VEC, INTER>(v, dp[c], ds[c]);
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum = __builtin_fmaf(xp[c][k], xp[c][k], __builtin_fmaf(xs[c][k], xs[c][k], sum));
        }
        const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(sum, a.log_lanes), a.inv_dim, a.eps));
        float along = 0.0f;
#pragma unroll
        for (int c = 0; c < K; ++c) {
            const int u = (c * lanes + sub) * VEC;
            if (u >= a.pairs) continue;
            const float2* t = angles + tok * a.pairs + u;
            float p[VEC], s[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float2 w = t[k];
                xp[c][k] *= inv, xs[c][k] *= inv;  // n
                if (!BACK) {
                    const float yp = xp[c][k] * gp[c][k], ys = xs[c][k] * gs[c][k];
                    p[k] = __builtin_fmaf(yp, w.x, -(ys * w.y));
                    s[k] = __builtin_fmaf(ys, w.x, yp * w.y);
                } else {
                    const float up = __builtin_fmaf(dp[c][k], w.x, ds[c][k] * w.y);  // turned back
                    const float us = __builtin_fmaf(ds[c][k], w.x, -(dp[c][k] * w.y));
                    acc[c][k] = __builtin_fmaf(up, xp[c][k], acc[c][k]);
                    acc[c][VEC + k] = __builtin_fmaf(us, xs[c][k], acc[c][VEC + k]);
                    dp[c][k] = up * gp[c][k], ds[c][k] = us * gs[c][k];
                    along = __builtin_fmaf(dp[c][k], xp[c][k], __builtin_fmaf(ds[c][k], xs[c][k], along));
                }
            }
            if (!BACK) {
                const Place<VEC, INTER> e(a, u);
                float v[2 * VEC];
                join_pairs<VEC, INTER>(p, s, v);
                store_vec<VEC>(y, e.e[0], v);
                store_vec<VEC>(y, e.e[1], v + VEC);
            }
        }
        if (!BACK) continue;
        const float mean = row_sum(along, a.log_lanes) * a.inv_dim;
#pragma unroll
        for (int c = 0; c < K; ++c) {
            const int u = (c * lanes + sub) * VEC;
            if (u >= a.pairs) continue;
            float p[VEC], s[VEC], v[2 * VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                p[k] = inv * __builtin_fmaf(-xp[c][k], mean, dp[c][k]);
                s[k] = inv * __builtin_fmaf(-xs[c][k], mean, ds[c][k]);
            }
            const Place<VEC, INTER> e(a, u);
            join_pairs<VEC, INTER>(p, s, v);
            store_vec<VEC>(y, e.e[0], v);
            store_vec<VEC>(y, e.e[1], v + VEC);
        }
    }
}

template <int VEC, int K, bool INTER, bool BACK> __global__ __launch_bounds__(256) void k_heads(HeadsArgs a) {
    __shared__ float2 angles[kAngles];
    __shared__ int64_t at[kTokens][6];
    __shared__ double position[kTokens];
    float acc[2][K][2 * VEC];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int c = 0; c < K; ++c)
#pragma unroll
            for (int k = 0; k < 2 * VEC; ++k) acc[w][c][k] = 0.0f;
    for (int64_t block = group_index(); block < a.blocks; block += (int64_t)gridDim.x * gridDim.y) {
        const int64_t first = block * a.tokens;
        const int tokens = (int)(a.total - first < a.tokens ? a.total - first : a.tokens);
        if (BACK) __syncthreads();  // the block before is done with the angles
        if ((int)threadIdx.x < tokens) {
            const int64_t n = first + threadIdx.x, b = a.total == a.per_batch ? 0 : n / a.per_batch, t = n - b * a.per_batch;
#pragma unroll
            for (int i = 0; i < 6; ++i) at[threadIdx.x][i] = b * a.v[i].batch + t * a.v[i].token;
            const int64_t i = b * a.position_batch + t * a.position_token;
            position[threadIdx.x] = a.positions_wide ? (double)static_cast<const int64_t*>(a.positions)[i]
                                                     : (double)static_cast<const int32_t*>(a.positions)[i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < tokens * a.pairs; i += 256) {
            const int tok = i / a.pairs, u = i - tok * a.pairs;
            angles[i] = u < a.half ? cos_sin(position[tok] * a.frequencies[u]) : make_float2(1.0f, 0.0f);
        }
        __syncthreads();
        rows_of<VEC, K, INTER, BACK>(a, 0, tokens, angles, at, acc[0]);
        rows_of<VEC, K, INTER, BACK>(a, 1, tokens, angles, at, acc[1]);
        if (!BACK) return;
    }
    if (!BACK) return;
    // the work-group's sums: over the rows of a wave, then over the waves
    float* lds = reinterpret_cast<float*>(angles);  // [4][dim]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lanes = 1 << a.log_lanes;
    float* part = a.part + (int64_t)group_index() * 2 * a.dim;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < K; ++c) {
            const int u = (c * lanes + (lane & (lanes - 1))) * VEC;
#pragma unroll
            for (int k = 0; k < 2 * VEC; ++k)
                for (int m = lanes; m < 64; m *= 2) acc[w][c][k] += __shfl_xor(acc[w][c][k], m);
            if (u >= a.pairs || lane >= lanes) continue;
            const Place<VEC, INTER> e(a, u);
            float v[2 * VEC];
            join_pairs<VEC, INTER>(acc[w][c], acc[w][c] + VEC, v);
#pragma unroll
            for (int k = 0; k < VEC; ++k) lds[wave * a.dim + e.e[0] + k] = v[k], lds[wave * a.dim + e.e[1] + k] = v[VEC + k];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.dim; i += 256)
            part[w * a.dim + i] = (lds[i] + lds[a.dim + i]) + (lds[2 * a.dim + i] + lds[3 * a.dim + i]);
    }
}

// The gains' gradients from the work-groups' sums: 16 of the 2 dim columns to a
// work-group, a 64th of the sums to a thread.
template <bool BF16, bool ADD>
__global__ __launch_bounds__(1024) void k_gain_grads(const float* part, int64_t groups, int dim, void* gq, void* gk) {
    __shared__ float lds[64][17];
    const int i = blockIdx.x * 16 + (threadIdx.x & 15), slice = threadIdx.x >> 4;
    float sum = 0.0f;
    if (i < 2 * dim)
        for (int64_t g = slice; g < groups; g += 64) sum += part[g * 2 * dim + i];
    lds[slice][threadIdx.x & 15] = sum;
    for (int s = 32; s > 0; s /= 2) {
        __syncthreads();
        if (slice < s) lds[slice][threadIdx.x & 15] += lds[slice + s][threadIdx.x & 15];
    }
    if (slice != 0 || i >= 2 * dim) return;
    sum = lds[0][threadIdx.x];
    void* p = i < dim ? gq : gk;
    const int at = i < dim ? i : i - dim;
    if (ADD) sum += load1<BF16>(p, at);
    if (BF16) static_cast<uint16_t*>(p)[at] = bf16_bits(sum);
    else static_cast<float*>(p)[at] = sum;
}

// Pairs to a lane and lanes to a row: 8 (or 4) pairs where both the rotary
// part and the rest are made of whole vectors, else single ones.
struct Shape {
    int vec, log_lanes, tokens;
};
Shape shape_of(const q4nn_rope& r) {
    const int pairs = r.dim / 2, half = r.rotary / 2;
    Shape s = {1, 0, 1};
    for (int v : {8, 4})
        if (s.vec == 1 && pairs % v == 0 && (r.interleaved || half % v == 0) && pairs <= 64 * v) s.vec = v;
    while ((1 << s.log_lanes) * s.vec < pairs && s.log_lanes < 6) ++s.log_lanes;
    // tokens to a work-group: until its four waves are full of rows of q and of k, while many work-groups are left
    const int rows = 4 * (64 >> s.log_lanes);
    int heads = r.q_heads < r.k_heads ? r.q_heads : r.k_heads;
    if (heads == 0) heads = r.q_heads + r.k_heads;
    const int64_t total = r.batches * r.tokens;
    while (s.tokens < kTokens && s.tokens * heads < rows && 2 * s.tokens * pairs <= kAngles &&
           total / (2 * s.tokens) >= 1024)
        s.tokens *= 2;
    return s;
}

HeadsArgs args_of(const q4nn_rope& r, const Shape& s) {
    HeadsArgs a = {};
    a.positions = r.positions, a.gain[0] = r.q_gain, a.gain[1] = r.k_gain, a.frequencies = r.frequencies;
    a.position_batch = r.position_batch, a.position_token = r.position_token;
    a.per_batch = r.tokens, a.total = r.batches * r.tokens, a.blocks = (a.total + s.tokens - 1) / s.tokens;
    a.heads[0] = r.q_heads, a.heads[1] = r.k_heads;
    for (int i = 0; i < 2; ++i)
        if (a.heads[i] > 1) a.magic[i] = (uint32_t)(((uint64_t(1) << 32) + a.heads[i] - 1) / a.heads[i]);
    a.dim = r.dim, a.half = r.rotary / 2, a.pairs = r.dim / 2, a.log_lanes = s.log_lanes, a.tokens = s.tokens;
    a.positions_wide = r.position_type == Q4NN_I64, a.gain_bf16 = r.gain_dtype == Q4MX_BF16;
    a.eps = r.eps, a.inv_dim = 1.0f / (float)r.dim;
    return a;
}

template <bool BACK> void launch_rows(const q4nn_rope& r, const Shape& s, const HeadsArgs& a, int64_t groups, hipStream_t st) {
    const dim3 g = grid_of(groups), b(256);
#define Q4_HEADS(V, K) \
    (r.interleaved ? k_heads<V, K, true, BACK><<<g, b, 0, st>>>(a) : k_heads<V, K, false, BACK><<<g, b, 0, st>>>(a))
    if (s.vec == 8) Q4_HEADS(8, 1);
    else if (s.vec == 4) Q4_HEADS(4, 1);
    else if (a.pairs <= 64) Q4_HEADS(1, 1);
    else Q4_HEADS(1, 8);
#undef Q4_HEADS
}

int64_t groups_of(const HeadsArgs& a) { return a.blocks < kMaxGroups ? a.blocks : kMaxGroups; }

}  // namespace

size_t head_norm_rope_workspace(const q4nn_rope& r) {
    return (size_t)groups_of(args_of(r, shape_of(r))) * 2 * r.dim * sizeof(float);
}

hipError_t launch_head_norm_rope(const q4nn_rope& r, const q4nn_heads& q, const q4nn_heads& k, const q4nn_heads& qo,
                                 const q4nn_heads& ko, hipStream_t st) {
    const Shape s = shape_of(r);
    HeadsArgs a = args_of(r, s);
    a.v[0] = q, a.v[1] = k, a.v[4] = qo, a.v[5] = ko;
    launch_rows<false>(r, s, a, a.blocks, st);
    return hipGetLastError();
}

hipError_t launch_head_norm_rope_backward(const q4nn_rope& r, const q4nn_heads& q, const q4nn_heads& k,
                                          const q4nn_heads& dq, const q4nn_heads& dk, const q4nn_heads& dq_in,
                                          const q4nn_heads& dk_in, void* gq, void* gk, int dtype, bool add, void* ws,
                                          hipStream_t st) {
    const Shape s = shape_of(r);
    HeadsArgs a = args_of(r, s);
    a.v[0] = q, a.v[1] = k, a.v[2] = dq, a.v[3] = dk, a.v[4] = dq_in, a.v[5] = dk_in;
    a.part = static_cast<float*>(ws);
    const bool some = a.total > 0 && r.q_heads + r.k_heads > 0;
    const int64_t groups = some ? groups_of(a) : 0;
    if (some) launch_rows<true>(r, s, a, groups, st);
    const dim3 g((unsigned)((2 * r.dim + 15) / 16)), b(1024);
    if (dtype == Q4MX_BF16 && add) k_gain_grads<true, true><<<g, b, 0, st>>>(a.part, groups, r.dim, gq, gk);
    else if (dtype == Q4MX_BF16) k_gain_grads<true, false><<<g, b, 0, st>>>(a.part, groups, r.dim, gq, gk);
    else if (add) k_gain_grads<false, true><<<g, b, 0, st>>>(a.part, groups, r.dim, gq, gk);
    else k_gain_grads<false, false><<<g, b, 0, st>>>(a.part, groups, r.dim, gq, gk);
    return hipGetLastError();
}

}  // namespace q4
