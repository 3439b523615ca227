// q4_nn_heads.hip -- the norm of queries and keys over each head and their
// rotation by position, in one pass, and its gradients (gfx950).
//
// A row is one head of one token: dim elements, consecutive.  Memory bounds
// both directions, 4 bytes an element forward, 6 backward (8192 tokens x 24 heads
// of 128: 21 us, 101 MB at 4.8 TB/s, and 31 us, 151 MB at 4.9, with 4 us for the
// gains' gradients; 16001 x 64 heads of 80 forward: 66 us, 328 MB at 5.0).  So a
// row is read once, held in registers by a few lanes, and written once: its sums are
// exchanged between those lanes without shared memory.  The unit of work is a
// pair of elements that turn together; a lane takes VEC neighbouring pairs in
// two vectors (the halves' (i, i + rotary/2), or 2 VEC neighbours when pairs
// are interleaved), so the rotation needs no exchange.  Elements past `rotary`
// pair up the same way, with the angle 0.
//
// A work-group takes some tokens' rows of q, or of k.  The angles of a token
// are those of all its rows, and FP64: a work-group forms the cosines and sines
// of its tokens once, in shared memory, while its first rows are being loaded.
// Arithmetic is not far behind memory (an instruction is 4 cycles of a wave), so
// a lane steps from row to row by additions, and rows whose lanes are no power
// of two (5 for a head of 80) are packed without idle lanes.
#include "q4_mx_dev.h"
#include "q4_nn.h"

namespace q4 {
namespace {

constexpr int kTokens = 64, kAngles = 2048;  // most tokens and angles of a work-group
constexpr int kGroups = 1000;                // of a backward pass the chip holds at once: 4 to a compute unit, a few to spare

// One of q and k.
struct Tensor {
    q4nn_heads in, grad, out;  // grad: backward only
    const void* gain;
    int64_t batch_groups, groups;  // work-groups of a batch, and all
    int heads, tokens;             // tokens: of a work-group
    float* part;                   // [groups][dim]: sums of the gain's gradient
};
struct HeadsArgs {
    Tensor t[2];
    const void* positions;
    const double* frequencies;
    int64_t position_batch, position_token, per_batch;  // per_batch: tokens
    int dim, half, pairs, lanes, log_pairs;  // lanes: of a row; 2^log_pairs >= pairs, or 256
    bool positions_wide, gain_bf16;
    float eps, inv_dim;
};

// Cosine and sine of `a` radians.  FP64 brings the angle to a quarter turn and
// its remainder within +-1/8 turn, which FP32 holds to half a step; there the
// Taylor polynomials to x^9 and x^10 are off by less than 2^-29.  From 2^40 on
// the number of quarters is itself rounded, more than half a quarter from 2^52
// on, so the remainder is reduced once more: 2^72 quarters leave up to 2^20, and
// pi/2 in two parts, off by 2^-109, still gives them to 2^-33.  That holds every
// 64-bit position at frequencies up to 2^9; from 2^72 on the angle is NaN.
__device__ __forceinline__ float2 cos_sin(double a) {
    constexpr double kQuarters = 0.63661977236758134308;  // 2 / pi
    const double q = __builtin_rint(a * kQuarters);
    // the remainder in radians: a multiply-add keeps what the product alone loses of a far angle
    const auto less = [](double x, double quarters) {
        return __builtin_fma(quarters, -6.123233995736766036e-17, __builtin_fma(quarters, -1.57079632679489661923, x));
    };
    double r = less(a, q);
    int n = (int)(q - 4.0 * __builtin_floor(q * 0.25));  // q mod 4
    if (__builtin_fabs(a) >= 0x1p40) {
        const double more = __builtin_rint(r * kQuarters);
        r = __builtin_fabs(a) < 0x1p72 ? less(r, more) : __builtin_nan("");
        n = (n + (int)more) & 3;
    }
    const float x = (float)r, z = x * x;
    float s = __builtin_fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    s = __builtin_fmaf(z, s, 8.3333333e-3f);
    s = __builtin_fmaf(z, s, -0.16666667f);
    s = __builtin_fmaf(x * z, s, x);
    float c = __builtin_fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    c = __builtin_fmaf(z, c, -1.3888889e-3f);
    c = __builtin_fmaf(z, c, 4.1666667e-2f);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.0f);
    const float cc = (n & 1) ? s : c, ss = (n & 1) ? c : s;
    return make_float2((n == 1 || n == 2) ? -cc : cc, n >= 2 ? -ss : ss);
}

// Sum over the neighbouring lanes of a row, of which lane `first` is the
// first: the same in each of them.
__device__ __forceinline__ float row_sum(float x, int lanes, int first) {
    if ((lanes & (lanes - 1)) != 0) {
        float sum = 0.0f;
        for (int k = 0; k < lanes; ++k)
            sum += __int_as_float(__builtin_amdgcn_ds_bpermute((first + k) * 4, __float_as_int(x)));
        return sum;
    }
#define Q4_ADD_DPP(ctrl) \
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, 0xF, 0xF, true))
    if (lanes > 1) Q4_ADD_DPP(0xB1);   // lanes 1 0 3 2
    if (lanes > 2) Q4_ADD_DPP(0x4E);   // lanes 2 3 0 1
    if (lanes > 4) Q4_ADD_DPP(0x141);  // the other quad of 8
    if (lanes > 8) Q4_ADD_DPP(0x140);  // the other 8 of 16
#undef Q4_ADD_DPP
    if (lanes > 16) x += __shfl_xor(x, 16);
    if (lanes > 32) x += __shfl_xor(x, 32);
    return x;
}

// Two FP32 as BF16 in a word, to nearest even.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    union {
        bf16x2 b;
        uint32_t u;
    } t;
    t.b = __builtin_convertvector((f32x2{lo, hi}), bf16x2);
    return t.u;
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

// A lane's pairs of a row as they lie in memory: VEC words, the two vectors one
// behind the other.
template <int VEC> struct Words {
    uint32_t w[VEC];
};
template <int VEC> __device__ __forceinline__ Words<VEC> load_words(const uint16_t* p, const int* e) {
    Words<VEC> r;
    if (VEC == 8) {
        const u32x4_any a = *reinterpret_cast<const u32x4_any*>(p + e[0]), b = *reinterpret_cast<const u32x4_any*>(p + e[1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[k] = a[k], r.w[(4 + k) % VEC] = b[k];
    } else if (VEC == 4) {
        const u32x2_any a = *reinterpret_cast<const u32x2_any*>(p + e[0]), b = *reinterpret_cast<const u32x2_any*>(p + e[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) r.w[k] = a[k], r.w[(2 + k) % VEC] = b[k];
    } else {
        r.w[0] = (uint32_t)p[e[0]] | (uint32_t)p[e[1]] << 16;
    }
    return r;
}
template <int VEC> __device__ __forceinline__ void store_words(uint16_t* p, const int* e, const Words<VEC>& r) {
    if (VEC == 8) {
        *reinterpret_cast<u32x4_any*>(p + e[0]) = u32x4_any{r.w[0], r.w[1 % VEC], r.w[2 % VEC], r.w[3 % VEC]};
        *reinterpret_cast<u32x4_any*>(p + e[1]) = u32x4_any{r.w[4 % VEC], r.w[5 % VEC], r.w[6 % VEC], r.w[7 % VEC]};
    } else if (VEC == 4) {
        *reinterpret_cast<u32x2_any*>(p + e[0]) = u32x2_any{r.w[0], r.w[1 % VEC]};
        *reinterpret_cast<u32x2_any*>(p + e[1]) = u32x2_any{r.w[2 % VEC], r.w[3 % VEC]};
    } else {
        p[e[0]] = (uint16_t)r.w[0], p[e[1]] = (uint16_t)(r.w[0] >> 16);
    }
}
// The pairs' first and second elements, and back.
template <int VEC, bool INTER> __device__ __forceinline__ void split_pairs(const Words<VEC>& r, float* p, float* s) {
    const auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
    const auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        if (INTER || VEC == 1) {
            p[k] = lo(r.w[k]), s[k] = hi(r.w[k]);
        } else {
            p[k] = k & 1 ? hi(r.w[k / 2]) : lo(r.w[k / 2]);
            s[k] = k & 1 ? hi(r.w[VEC / 2 + k / 2]) : lo(r.w[VEC / 2 + k / 2]);
        }
    }
}
template <int VEC, bool INTER> __device__ __forceinline__ Words<VEC> join_pairs(const float* p, const float* s) {
    Words<VEC> r;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        if (INTER || VEC == 1) r.w[k] = pack2(p[k], s[k]);
        else if (k < VEC / 2) r.w[k] = pack2(p[2 * k], p[(2 * k + 1) % VEC]);
        else r.w[k] = pack2(s[2 * k - VEC], s[(2 * k + 1) % VEC]);
    }
    return r;
}

// K vectors of pairs to a lane (one, but for heads of odd sizes above 128).
template <int VEC, int K, bool INTER, bool BACK>
__global__ __launch_bounds__(256, K == 1 ? 4 : 1) void k_heads(HeadsArgs a) {
    // angles [tokens][K][VEC][lanes] (of pair (c lanes + sub) VEC + k: lanes read neighbours); backward, after
    // that: sums of the gain's gradient [4 waves][dim]
    extern __shared__ float4 shared[];
    float2* const angles = reinterpret_cast<float2*>(shared);
    int64_t group = group_index();
    const bool second = group >= a.t[0].groups;
    const Tensor& w = a.t[second];
    if (second) group -= a.t[0].groups;
    if (group >= w.groups) return;
    const int64_t b = group / w.batch_groups, t0 = (group - b * w.batch_groups) * w.tokens;
    const int tokens = (int)(a.per_batch - t0 < w.tokens ? a.per_batch - t0 : w.tokens);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per_wave = 64 / a.lanes, mine = lane / a.lanes, sub = lane - mine * a.lanes, stride = 4 * per_wave;
    const int token_size = K * VEC * a.lanes, rows = tokens * w.heads;

    // A lane's rows are `stride` apart: that many heads on, or a token and some less.
    int row = mine < per_wave ? wave * per_wave + mine : rows;
    const int step_tokens = stride / w.heads, step_heads = stride - step_tokens * w.heads;
    const int start = row < rows ? row : 0;  // a lane without a row computes on the first, and stores nothing
    int tok = start / w.heads, head = start - tok * w.heads;
    const auto first_of = [&](const q4nn_heads& v) { return v.p + (b * v.batch + (t0 + tok) * v.token + head * v.head); };
    const uint16_t *x_at = first_of(w.in), *dy_at = BACK ? first_of(w.grad) : nullptr;
    uint16_t* y_at = first_of(w.out);
    const auto step_of = [&](const q4nn_heads& v) { return step_tokens * v.token + step_heads * v.head; };
    const auto wrap_of = [&](const q4nn_heads& v) { return v.token - w.heads * v.head; };
    const int64_t x_step = step_of(w.in), y_step = step_of(w.out), dy_step = BACK ? step_of(w.grad) : 0;
    const int64_t x_past = x_step + wrap_of(w.in), y_past = y_step + wrap_of(w.out);
    const int64_t dy_past = BACK ? dy_step + wrap_of(w.grad) : 0;

    Words<VEC> x[K] = {}, dy[K] = {};  // zeros stay where a lane's pairs are past the row's
    const auto load = [&] {
#pragma unroll
        for (int c = 0; c < K; ++c) {
            const int u = (c * a.lanes + sub) * VEC;
            if (u >= a.pairs) continue;
            const Place<VEC, INTER> e(a, u);
            x[c] = load_words<VEC>(x_at, e.e);
            if (BACK) dy[c] = load_words<VEC>(dy_at, e.e);
        }
    };
    load();
    float gp[K][VEC], gs[K][VEC];
#pragma unroll
    for (int c = 0; c < K; ++c) {
        const int u = (c * a.lanes + sub) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) gp[c][k] = gs[c][k] = 0.0f;
        if (u >= a.pairs) continue;
        const Place<VEC, INTER> e(a, u);
        if (a.gain_bf16) {
            split_pairs<VEC, INTER>(load_words<VEC>(static_cast<const uint16_t*>(w.gain), e.e), gp[c], gs[c]);
        } else {
            const float* g = static_cast<const float*>(w.gain);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                gp[c][k] = INTER ? (2 * k < VEC ? g[e.e[0] + 2 * k] : g[e.e[1] + 2 * k - VEC]) : g[e.e[0] + k];
                gs[c][k] = INTER ? (2 * k + 1 < VEC ? g[e.e[0] + 2 * k + 1] : g[e.e[1] + 2 * k + 1 - VEC]) : g[e.e[1] + k];
            }
        }
    }
    // a thread forms the angles of one pair (or every 256th) for every so many tokens
    for (int u = threadIdx.x & ((1 << a.log_pairs) - 1); u < K * VEC * a.lanes; u += 256) {
        const int cl = u / VEC, c = K == 1 ? 0 : cl / a.lanes;
        const int at = (c * VEC + u % VEC) * a.lanes + cl - c * a.lanes;
        const double frequency = u < a.half ? a.frequencies[u] : 0.0;
        for (int t = threadIdx.x >> a.log_pairs; t < tokens; t += 256 >> a.log_pairs) {
            const int64_t p = b * a.position_batch + (t0 + t) * a.position_token;
            const double position = a.positions_wide ? (double)static_cast<const int64_t*>(a.positions)[p]
                                                     : (double)static_cast<const int32_t*>(a.positions)[p];
            angles[t * token_size + at] = u < a.half ? cos_sin(position * frequency) : make_float2(1.0f, 0.0f);
        }
    }
    __syncthreads();

    float acc[K][2 * VEC];  // of the gain's gradient: pairs' first elements and second
#pragma unroll
    for (int c = 0; c < K; ++c)
#pragma unroll
        for (int k = 0; k < 2 * VEC; ++k) acc[c][k] = 0.0f;
    const float2* turns = angles + tok * token_size + sub;
    while (row < rows) {
        float xp[K][VEC], xs[K][VEC], dp[K][VEC], ds[K][VEC], sum = 0.0f;
#pragma unroll
        for (int c = 0; c < K; ++c) {
            split_pairs<VEC, INTER>(x[c], xp[c], xs[c]);
            if (BACK) split_pairs<VEC, INTER>(dy[c], dp[c], ds[c]);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                sum = __builtin_fmaf(xp[c][k], xp[c][k], __builtin_fmaf(xs[c][k], xs[c][k], sum));
        }
        const float inv =
            __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(sum, a.lanes, lane - sub), a.inv_dim, a.eps));
        float along = 0.0f;
#pragma unroll
        for (int c = 0; c < K; ++c) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float2 t = turns[(c * VEC + k) * a.lanes];
                xp[c][k] *= inv, xs[c][k] *= inv;  // n
                if (!BACK) {
                    const float yp = xp[c][k] * gp[c][k], ys = xs[c][k] * gs[c][k];
                    xp[c][k] = __builtin_fmaf(yp, t.x, -(ys * t.y));
                    xs[c][k] = __builtin_fmaf(ys, t.x, yp * t.y);
                } else {
                    const float up = __builtin_fmaf(dp[c][k], t.x, ds[c][k] * t.y);  // turned back
                    const float us = __builtin_fmaf(ds[c][k], t.x, -(dp[c][k] * t.y));
                    acc[c][k] = __builtin_fmaf(up, xp[c][k], acc[c][k]);
                    acc[c][VEC + k] = __builtin_fmaf(us, xs[c][k], acc[c][VEC + k]);
                    dp[c][k] = up * gp[c][k], ds[c][k] = us * gs[c][k];
                    along = __builtin_fmaf(dp[c][k], xp[c][k], __builtin_fmaf(ds[c][k], xs[c][k], along));
                }
            }
        }
        if (BACK) {
            const float mean = row_sum(along, a.lanes, lane - sub) * a.inv_dim;
#pragma unroll
            for (int c = 0; c < K; ++c)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    xp[c][k] = inv * __builtin_fmaf(-xp[c][k], mean, dp[c][k]);
                    xs[c][k] = inv * __builtin_fmaf(-xs[c][k], mean, ds[c][k]);
                }
        }
        uint16_t* const y = y_at;
        // the next row
        row += stride, head += step_heads;
        const bool past = head >= w.heads;
        head -= past ? w.heads : 0;
        turns += (step_tokens + (past ? 1 : 0)) * token_size;
        x_at += past ? x_past : x_step, y_at += past ? y_past : y_step;
        if (BACK) dy_at += past ? dy_past : dy_step;
        if (row < rows) load();
#pragma unroll
        for (int c = 0; c < K; ++c) {
            const int u = (c * a.lanes + sub) * VEC;
            if (u >= a.pairs) continue;
            store_words<VEC>(y, Place<VEC, INTER>(a, u).e, join_pairs<VEC, INTER>(xp[c], xs[c]));
        }
    }
    if (!BACK) return;

    // the sums over a wave's rows, then over the waves
    float* const sums = reinterpret_cast<float*>(angles + w.tokens * token_size);
    if ((a.lanes & (a.lanes - 1)) == 0) {
        for (int m = a.lanes; m < 64; m *= 2)
#pragma unroll
            for (int c = 0; c < K; ++c)
#pragma unroll
                for (int k = 0; k < 2 * VEC; ++k) acc[c][k] += __shfl_xor(acc[c][k], m);
    } else {
        float own[K][2 * VEC];
#pragma unroll
        for (int c = 0; c < K; ++c)
#pragma unroll
            for (int k = 0; k < 2 * VEC; ++k) own[c][k] = acc[c][k];
        for (int m = 1; m < per_wave; ++m)
#pragma unroll
            for (int c = 0; c < K; ++c)
#pragma unroll
                for (int k = 0; k < 2 * VEC; ++k)
                    acc[c][k] += __int_as_float(
                        __builtin_amdgcn_ds_bpermute((sub + m * a.lanes) * 4, __float_as_int(own[c][k])));
    }
#pragma unroll
    for (int c = 0; c < K; ++c) {
        const int u = (c * a.lanes + sub) * VEC;
        if (u >= a.pairs || lane >= a.lanes) continue;
        const Place<VEC, INTER> e(a, u);
#pragma unroll
        for (int k = 0; k < 2 * VEC; ++k) {
            const int p = k < VEC ? k : k - VEC;  // pair u + p
            sums[wave * a.dim + (INTER ? 2 * (u + p) + (k >= VEC) : e.e[k >= VEC] + p)] = acc[c][k];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.dim; i += 256)
        w.part[group * a.dim + i] = (sums[i] + sums[a.dim + i]) + (sums[2 * a.dim + i] + sums[3 * a.dim + i]);
}

// The gains' gradients from the work-groups' sums: 16 columns of q's or k's to a
// work-group, a 64th of the sums to a thread.
struct GainSums {
    const float* part[2];
    int64_t groups[2];
    void* grad[2];
};
template <bool BF16, bool ADD> __global__ __launch_bounds__(1024) void k_gain_grads(GainSums a, int dim) {
    __shared__ float lds[64][17];
    const int blocks = (dim + 15) / 16, w = (int)blockIdx.x >= blocks;
    const int col = threadIdx.x & 15, i = ((int)blockIdx.x - w * blocks) * 16 + col, slice = threadIdx.x >> 4;
    float sum = 0.0f;
    if (i < dim) {
#pragma unroll 8
        for (int64_t g = slice; g < a.groups[w]; g += 64) sum += a.part[w][g * dim + i];
    }
    lds[slice][col] = sum;
    for (int s = 32; s > 0; s /= 2) {
        __syncthreads();
        if (slice < s) lds[slice][col] += lds[slice + s][col];
    }
    if (slice != 0 || i >= dim) return;
    sum = lds[0][col];
    if (ADD) sum += load1<BF16>(a.grad[w], i);
    if (BF16) static_cast<uint16_t*>(a.grad[w])[i] = bf16_bits(sum);
    else static_cast<float*>(a.grad[w])[i] = sum;
}

// The call with its tokens in as few batches as their strides allow: one where
// the batches follow each other, or have a token each.
q4nn_rope flat_batches(const q4nn_rope& r, q4nn_heads* const* v, int n) {
    q4nn_rope f = r;
    bool follow = r.position_batch == r.tokens * r.position_token;
    for (int i = 0; i < n; ++i) follow = follow && v[i]->batch == r.tokens * v[i]->token;
    if (r.batches <= 1 || (!follow && r.tokens > 1)) return f;
    if (r.tokens == 1) {
        for (int i = 0; i < n; ++i) v[i]->token = v[i]->batch;
        f.position_token = r.position_batch;
    }
    f.tokens = r.batches * r.tokens, f.batches = 1;
    return f;
}

// Pairs to a lane and lanes to a row: 8 (or 4) pairs where both the rotary
// part and the rest are made of whole vectors, else single ones, in accesses of 2
// bytes (8192 tokens x 24 heads of 72, forward and backward: 18 + 24 us, with 36
// elements rotated 50 + 57).  Rows of up to 16 lanes lie side by side as they are
// where a wave takes more of them so (heads of 80: 12 in place of 8, and 66 us in
// place of 73 for a prompt of 16001 tokens x 64 heads), else padded to a power of
// two.
struct Shape {
    int vec, lanes;
};
Shape shape_of(const q4nn_rope& r) {
    const int pairs = r.dim / 2, half = r.rotary / 2;
    Shape s = {1, 1};
    for (int v : {8, 4})
        if (s.vec == 1 && pairs % v == 0 && (r.interleaved || half % v == 0) && pairs <= 64 * v) s.vec = v;
    while (s.lanes * s.vec < pairs && s.lanes < 64) s.lanes *= 2;
    const int tight = pairs / s.vec;
    if (tight <= 16 && 64 / tight > 64 / s.lanes) s.lanes = tight;
    return s;
}

// Angles of a token in shared memory: a lane's whole vectors of them.
int angles_of(const q4nn_rope& r, const Shape& s) { return s.vec * s.lanes * (s.vec == 1 && r.dim > 128 ? 8 : 1); }

// Tokens to a work-group, `heads` rows each: forward two steps of its waves,
// while there are work-groups for all compute units; backward as many rows as
// leave the work-groups that the chip holds at once, since each ends in a sum
// over its waves.
int tokens_of(const q4nn_rope& r, const Shape& s, int heads, bool back) {
    const int64_t step = 4 * (64 / s.lanes), rows = r.batches * r.tokens * (r.q_heads + r.k_heads);
    int64_t tokens = 1;
    if (heads > 0 && back) tokens = (rows / kGroups + heads) / heads;
    else if (heads > 0) tokens = (rows / kGroups < step ? rows / kGroups : rows / kGroups < 2 * step ? step : 2 * step) / heads;
    if (tokens > kTokens) tokens = kTokens;
    if (tokens > kAngles / angles_of(r, s)) tokens = kAngles / angles_of(r, s);
    return tokens < 1 ? 1 : (int)tokens;
}

HeadsArgs args_of(const q4nn_rope& r, const Shape& s, bool back) {
    HeadsArgs a = {};
    a.positions = r.positions, a.frequencies = r.frequencies;
    a.position_batch = r.position_batch, a.position_token = r.position_token;
    a.per_batch = r.tokens;
    for (int i = 0; i < 2; ++i) {
        Tensor& t = a.t[i];
        t.heads = i ? r.k_heads : r.q_heads, t.gain = i ? r.k_gain : r.q_gain;
        t.tokens = tokens_of(r, s, t.heads, back);
        t.batch_groups = (r.tokens + t.tokens - 1) / t.tokens;
        t.groups = t.heads > 0 ? r.batches * t.batch_groups : 0;
    }
    a.dim = r.dim, a.half = r.rotary / 2, a.pairs = r.dim / 2, a.lanes = s.lanes;
    while (a.log_pairs < 8 && (1 << a.log_pairs) < angles_of(r, s)) ++a.log_pairs;
    a.positions_wide = r.position_type == Q4NN_I64, a.gain_bf16 = r.gain_dtype == Q4MX_BF16;
    a.eps = r.eps, a.inv_dim = 1.0f / (float)r.dim;
    return a;
}

template <bool BACK> void launch_rows(const q4nn_rope& r, const Shape& s, const HeadsArgs& a, hipStream_t st) {
    const dim3 g = grid_of(a.t[0].groups + a.t[1].groups), b(256);
    const int tokens = a.t[0].tokens > a.t[1].tokens ? a.t[0].tokens : a.t[1].tokens;
    const size_t lds = (BACK ? 4 * sizeof(float) * a.dim : 0) + sizeof(float2) * tokens * angles_of(r, s);
#define Q4_HEADS(V, K)                                               \
    (r.interleaved ? k_heads<V, K, true, BACK><<<g, b, lds, st>>>(a) \
                   : k_heads<V, K, false, BACK><<<g, b, lds, st>>>(a))
    if (s.vec == 8) Q4_HEADS(8, 1);
    else if (s.vec == 4) Q4_HEADS(4, 1);
    else if (a.pairs <= 64) Q4_HEADS(1, 1);
    else Q4_HEADS(1, 8);
#undef Q4_HEADS
}

}  // namespace

// The most work-groups that any strides lead to.
size_t head_norm_rope_workspace(const q4nn_rope& r) {
    const Shape s = shape_of(r);
    q4nn_rope flat = r;
    flat.tokens = r.batches * r.tokens, flat.batches = 1;
    const HeadsArgs a = args_of(r, s, true), f = args_of(flat, s, true);
    const int64_t q = a.t[0].groups > f.t[0].groups ? a.t[0].groups : f.t[0].groups;
    const int64_t k = a.t[1].groups > f.t[1].groups ? a.t[1].groups : f.t[1].groups;
    return (size_t)(q + k) * r.dim * sizeof(float);
}

hipError_t launch_head_norm_rope(const q4nn_rope& rope, const q4nn_heads& q, const q4nn_heads& k, const q4nn_heads& qo,
                                 const q4nn_heads& ko, hipStream_t st) {
    q4nn_heads v[4] = {q, k, qo, ko}, *const at[4] = {v, v + 1, v + 2, v + 3};
    const q4nn_rope r = flat_batches(rope, at, 4);
    const Shape s = shape_of(r);
    HeadsArgs a = args_of(r, s, false);
    for (int i = 0; i < 2; ++i) a.t[i].in = v[i], a.t[i].out = v[2 + i];
    launch_rows<false>(r, s, a, st);
    return hipGetLastError();
}

hipError_t launch_head_norm_rope_backward(const q4nn_rope& rope, const q4nn_heads& q, const q4nn_heads& k,
                                          const q4nn_heads& dq, const q4nn_heads& dk, const q4nn_heads& dq_in,
                                          const q4nn_heads& dk_in, void* gq, void* gk, int dtype, bool add, void* ws,
                                          hipStream_t st) {
    q4nn_heads v[6] = {q, k, dq, dk, dq_in, dk_in}, *const at[6] = {v, v + 1, v + 2, v + 3, v + 4, v + 5};
    const q4nn_rope r = flat_batches(rope, at, 6);
    GainSums g = {};
    g.grad[0] = gq, g.grad[1] = gk;
    if (r.batches * r.tokens > 0 && r.q_heads + r.k_heads > 0) {
        const Shape s = shape_of(r);
        HeadsArgs a = args_of(r, s, true);
        float* part = static_cast<float*>(ws);
        for (int i = 0; i < 2; ++i) {
            Tensor& t = a.t[i];
            t.in = v[i], t.grad = v[2 + i], t.out = v[4 + i], t.part = part;
            g.part[i] = part, g.groups[i] = t.groups;
            part += t.groups * r.dim;
        }
        launch_rows<true>(r, s, a, st);
    }
    const dim3 n((unsigned)(2 * ((r.dim + 15) / 16))), b(1024);
    if (dtype == Q4MX_BF16 && add) k_gain_grads<true, true><<<n, b, 0, st>>>(g, r.dim);
    else if (dtype == Q4MX_BF16) k_gain_grads<true, false><<<n, b, 0, st>>>(g, r.dim);
    else if (add) k_gain_grads<false, true><<<n, b, 0, st>>>(g, r.dim);
    else k_gain_grads<false, false><<<n, b, 0, st>>>(g, r.dim);
    return hipGetLastError();
}

}  // namespace q4
