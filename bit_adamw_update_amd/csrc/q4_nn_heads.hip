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
// forms the cosines and sines of its tokens once, in shared memory.  Its four
// waves then walk the rows, q's first; the loads of a wave's next rows are on
// their way while it computes, those of its first ones while the angles are
// formed.
#include "q4_mx_dev.h"
#include "q4_nn.h"

namespace q4 {
namespace {

constexpr int kTokens = 32, kAngles = 2048;  // most tokens and angles of a work-group
constexpr int kMaxGroups = 1024;             // of a backward pass: each leaves one sum of the gains' gradients

struct HeadsArgs {
    q4nn_heads v[6];  // q, k, dq, dk, q_out, k_out (backward: dq_in, dk_in)
    const void *positions, *gain[2];
    const double* frequencies;
    int64_t position_batch, position_token;
    int64_t per_batch, batch_blocks, blocks;  // tokens and work-groups' parts of a batch, and all parts
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
        if (INTER || VEC == 1) r.w[k] = bf16_pair(p[k], s[k]);
        else if (k < VEC / 2) r.w[k] = bf16_pair(p[2 * k], p[(2 * k + 1) % VEC]);
        else r.w[k] = bf16_pair(s[2 * k - VEC], s[(2 * k + 1) % VEC]);
    }
    return r;
}

// K vectors of pairs to a lane (one, but for heads of odd sizes above 128).
template <int VEC, int K, bool INTER, bool BACK>
__global__ __launch_bounds__(256, K == 1 ? 4 : 1) void k_heads(HeadsArgs a) {
    extern __shared__ float4 shared[];
    // gains [2][dim], backward: sums [4 waves][2][dim]; angles
    float* gains = reinterpret_cast<float*>(shared);
    float* sums = gains + 2 * a.dim;
    float2* angles = reinterpret_cast<float2*>(sums + (BACK ? 8 * a.dim : 0));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lanes = 1 << a.log_lanes;
    const int sub = lane & (lanes - 1), mine = lane >> a.log_lanes, per_wave = 64 >> a.log_lanes;
    for (int i = threadIdx.x; i < 2 * a.dim; i += 256) {
        const int w = i >= a.dim, at = i - (w ? a.dim : 0);
        gains[i] = a.heads[w] == 0 ? 0.0f : a.gain_bf16 ? load1<true>(a.gain[w], at) : load1<false>(a.gain[w], at);
    }
    if (BACK)
        for (int i = threadIdx.x; i < 8 * a.dim; i += 256) sums[i] = 0.0f;

    for (int64_t block = group_index(); block < a.blocks; block += (int64_t)gridDim.x * gridDim.y) {
        const int64_t b = block / a.batch_blocks, t0 = (block - b * a.batch_blocks) * a.tokens;
        const int tokens = (int)(a.per_batch - t0 < a.tokens ? a.per_batch - t0 : a.tokens);
        const int rows_q = tokens * a.heads[0], rows_k = tokens * a.heads[1];
        const int steps_q = (rows_q + 4 * per_wave - 1) / (4 * per_wave);
        const int steps = steps_q + (rows_k + 4 * per_wave - 1) / (4 * per_wave);
        // Step i of a wave: its rows' tensor, and this lane's row.  q's rows go to the first waves first, k's to the last.
        const auto row_of = [&](int i) {
            return i < steps_q ? (i * 4 + wave) * per_wave + mine : ((i - steps_q) * 4 + 3 - wave) * per_wave + mine;
        };
        // r / heads: the reciprocal is less than heads 2^-32 of itself too large, and r < 32 * 4096 + 256, heads <= 4096
        const auto token_of = [&](int r, int w) {
            return a.heads[w] == 1 ? r : (int)__umulhi((uint32_t)r, a.magic[w]);
        };
        const auto place_of = [&](const q4nn_heads& v, int tok, int head) {
            return v.p + (b * v.batch + t0 * v.token) + (tok * v.token + head * v.head);
        };
        struct Loaded {
            Words<VEC> x[K], dy[BACK ? K : 1];
        };
        const auto load_step = [&](int i) {
            Loaded l = {};
            const int w = i < steps_q ? 0 : 1, r = row_of(i);
            if (r < (w ? rows_k : rows_q)) {
                const int tok = token_of(r, w), head = r - tok * a.heads[w];
                const uint16_t* x = place_of(a.v[w], tok, head);
                const uint16_t* dy = BACK ? place_of(a.v[2 + w], tok, head) : nullptr;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    const int u = (c * lanes + sub) * VEC;
                    if (u >= a.pairs) continue;
                    const Place<VEC, INTER> e(a, u);
                    l.x[c] = load_words<VEC>(x, e.e);
                    if (BACK) l.dy[c] = load_words<VEC>(dy, e.e);
                }
            }
            return l;
        };
        Loaded now = load_step(0);
        __syncthreads();  // the block before is done with the angles
        for (int i = threadIdx.x; i < tokens * a.pairs; i += 256) {
            const int tok = i / a.pairs, u = i - tok * a.pairs;
            float2 w = make_float2(1.0f, 0.0f);
            if (u < a.half) {
                const int64_t at = b * a.position_batch + (t0 + tok) * a.position_token;
                const double position = a.positions_wide ? (double)static_cast<const int64_t*>(a.positions)[at]
                                                         : (double)static_cast<const int32_t*>(a.positions)[at];
                w = cos_sin(position * a.frequencies[u]);
            }
            angles[i] = w;
        }
        __syncthreads();
        float acc[K][2 * VEC];  // of the gain's gradient: pairs' first elements and second
#pragma unroll
        for (int c = 0; c < K; ++c)
#pragma unroll
            for (int k = 0; k < 2 * VEC; ++k) acc[c][k] = 0.0f;
        for (int i = 0; i < steps; ++i) {
            const int w = i < steps_q ? 0 : 1, r = row_of(i);
            Loaded next;
            if (i + 1 < steps) next = load_step(i + 1);
            if (r < (w ? rows_k : rows_q)) {
                const int tok = token_of(r, w), head = r - tok * a.heads[w];
                float xp[K][VEC], xs[K][VEC], dp[K][VEC], ds[K][VEC], sum = 0.0f;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    split_pairs<VEC, INTER>(now.x[c], xp[c], xs[c]);  // zeros past the row
                    if (BACK) split_pairs<VEC, INTER>(now.dy[c], dp[c], ds[c]);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        sum = __builtin_fmaf(xp[c][k], xp[c][k], __builtin_fmaf(xs[c][k], xs[c][k], sum));
                }
                const float inv =
                    __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum(sum, a.log_lanes), a.inv_dim, a.eps));
                uint16_t* y = place_of(a.v[4 + w], tok, head);
                float along = 0.0f;
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    const int u = (c * lanes + sub) * VEC;
                    if (u >= a.pairs) continue;
                    const Place<VEC, INTER> e(a, u);
                    const float2* turn = angles + tok * a.pairs + u;
                    const float *g0 = gains + w * a.dim + e.e[0], *g1 = gains + w * a.dim + e.e[1];
                    float p[VEC], s[VEC];
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const float2 t = turn[k];
                        const float gp = INTER && VEC > 1 ? (2 * k < VEC ? g0[2 * k] : g1[2 * k - VEC]) : g0[k];
                        const float gs = INTER && VEC > 1 ? (2 * k < VEC ? g0[2 * k + 1] : g1[2 * k + 1 - VEC]) : g1[k];
                        xp[c][k] *= inv, xs[c][k] *= inv;  // n
                        if (!BACK) {
                            const float yp = xp[c][k] * gp, ys = xs[c][k] * gs;
                            p[k] = __builtin_fmaf(yp, t.x, -(ys * t.y));
                            s[k] = __builtin_fmaf(ys, t.x, yp * t.y);
                        } else {
                            const float up = __builtin_fmaf(dp[c][k], t.x, ds[c][k] * t.y);  // turned back
                            const float us = __builtin_fmaf(ds[c][k], t.x, -(dp[c][k] * t.y));
                            acc[c][k] = __builtin_fmaf(up, xp[c][k], acc[c][k]);
                            acc[c][VEC + k] = __builtin_fmaf(us, xs[c][k], acc[c][VEC + k]);
                            dp[c][k] = up * gp, ds[c][k] = us * gs;
                            along = __builtin_fmaf(dp[c][k], xp[c][k], __builtin_fmaf(ds[c][k], xs[c][k], along));
                        }
                    }
                    if (!BACK) store_words<VEC>(y, e.e, join_pairs<VEC, INTER>(p, s));
                }
                if (BACK) {
                    const float mean = row_sum(along, a.log_lanes) * a.inv_dim;
#pragma unroll
                    for (int c = 0; c < K; ++c) {
                        const int u = (c * lanes + sub) * VEC;
                        if (u >= a.pairs) continue;
                        float p[VEC], s[VEC];
#pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            p[k] = inv * __builtin_fmaf(-xp[c][k], mean, dp[c][k]);
                            s[k] = inv * __builtin_fmaf(-xs[c][k], mean, ds[c][k]);
                        }
                        store_words<VEC>(y, Place<VEC, INTER>(a, u).e, join_pairs<VEC, INTER>(p, s));
                    }
                }
            }
            if (BACK && (i + 1 == steps_q || i + 1 == steps)) {
                // all of a tensor's rows: the sums over the wave's rows, added to the wave's own
#pragma unroll
                for (int c = 0; c < K; ++c) {
                    const int u = (c * lanes + sub) * VEC;
#pragma unroll
                    for (int k = 0; k < 2 * VEC; ++k)
                        for (int m = lanes; m < 64; m *= 2) acc[c][k] += __shfl_xor(acc[c][k], m);
                    if (u < a.pairs && lane < lanes) {
                        const Place<VEC, INTER> e(a, u);
                        float *p0 = sums + (wave * 2 + w) * a.dim + e.e[0], *p1 = sums + (wave * 2 + w) * a.dim + e.e[1];
#pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            // INTER: elements 2k and 2k + 1 of the two vectors
                            if (INTER && VEC > 1) {
                                (2 * k < VEC ? p0[2 * k] : p1[2 * k - VEC]) += acc[c][k];
                                (2 * k < VEC ? p0[2 * k + 1] : p1[2 * k + 1 - VEC]) += acc[c][VEC + k];
                            } else {
                                p0[k] += acc[c][k], p1[k] += acc[c][VEC + k];
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2 * VEC; ++k) acc[c][k] = 0.0f;
                }
            }
            now = next;
        }
        if (!BACK) return;
    }
    if (!BACK) return;
    __syncthreads();
    float* part = a.part + (int64_t)group_index() * 2 * a.dim;
    for (int i = threadIdx.x; i < 2 * a.dim; i += 256)
        part[i] = (sums[i] + sums[2 * a.dim + i]) + (sums[4 * a.dim + i] + sums[6 * a.dim + i]);
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
// part and the rest are made of whole vectors, else single ones.
struct Shape {
    int vec, log_lanes;
};
Shape shape_of(const q4nn_rope& r) {
    const int pairs = r.dim / 2, half = r.rotary / 2;
    Shape s = {1, 0};
    for (int v : {8, 4})
        if (s.vec == 1 && pairs % v == 0 && (r.interleaved || half % v == 0) && pairs <= 64 * v) s.vec = v;
    while ((1 << s.log_lanes) * s.vec < pairs && s.log_lanes < 6) ++s.log_lanes;
    return s;
}

// Tokens to a work-group's part.  Forward: until its four waves are full of
// rows of q and of k, while many work-groups are left.  Backward: as many as
// leave the parts that the chip holds at once.
int tokens_of(const q4nn_rope& r, const Shape& s, bool back) {
    const int rows = 4 * (64 >> s.log_lanes), pairs = r.dim / 2;
    int heads = r.q_heads < r.k_heads ? r.q_heads : r.k_heads, tokens = 1;
    if (heads == 0) heads = r.q_heads + r.k_heads;
    while (2 * tokens <= kTokens && 2 * tokens * pairs <= kAngles &&
           (back ? r.batches * ((r.tokens + tokens - 1) / tokens) > kMaxGroups
                 : tokens * heads < rows && r.batches * (r.tokens / (2 * tokens)) >= 1024))
        tokens *= 2;
    return tokens;
}

HeadsArgs args_of(const q4nn_rope& r, const Shape& s, bool back) {
    HeadsArgs a = {};
    a.positions = r.positions, a.gain[0] = r.q_gain, a.gain[1] = r.k_gain, a.frequencies = r.frequencies;
    a.position_batch = r.position_batch, a.position_token = r.position_token;
    a.tokens = tokens_of(r, s, back);
    a.per_batch = r.tokens, a.batch_blocks = (r.tokens + a.tokens - 1) / a.tokens, a.blocks = r.batches * a.batch_blocks;
    a.heads[0] = r.q_heads, a.heads[1] = r.k_heads;
    for (int i = 0; i < 2; ++i)
        if (a.heads[i] > 1) a.magic[i] = (uint32_t)(((uint64_t(1) << 32) + a.heads[i] - 1) / a.heads[i]);
    a.dim = r.dim, a.half = r.rotary / 2, a.pairs = r.dim / 2, a.log_lanes = s.log_lanes;
    a.positions_wide = r.position_type == Q4NN_I64, a.gain_bf16 = r.gain_dtype == Q4MX_BF16;
    a.eps = r.eps, a.inv_dim = 1.0f / (float)r.dim;
    return a;
}

template <bool BACK> void launch_rows(const q4nn_rope& r, const Shape& s, const HeadsArgs& a, int64_t groups, hipStream_t st) {
    const dim3 g = grid_of(groups), b(256);
    const size_t lds = (size_t)(BACK ? 10 : 2) * a.dim * sizeof(float) + (size_t)a.tokens * a.pairs * sizeof(float2);
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
    const int64_t total = r.batches * r.tokens;
    return (size_t)(total < kMaxGroups ? total : kMaxGroups) * 2 * r.dim * sizeof(float);
}

hipError_t launch_head_norm_rope(const q4nn_rope& rope, const q4nn_heads& q, const q4nn_heads& k, const q4nn_heads& qo,
                                 const q4nn_heads& ko, hipStream_t st) {
    q4nn_heads v[4] = {q, k, qo, ko}, *const at[4] = {v, v + 1, v + 2, v + 3};
    const q4nn_rope r = flat_batches(rope, at, 4);
    const Shape s = shape_of(r);
    HeadsArgs a = args_of(r, s, false);
    a.v[0] = v[0], a.v[1] = v[1], a.v[4] = v[2], a.v[5] = v[3];
    launch_rows<false>(r, s, a, a.blocks, st);
    return hipGetLastError();
}

hipError_t launch_head_norm_rope_backward(const q4nn_rope& rope, const q4nn_heads& q, const q4nn_heads& k,
                                          const q4nn_heads& dq, const q4nn_heads& dk, const q4nn_heads& dq_in,
                                          const q4nn_heads& dk_in, void* gq, void* gk, int dtype, bool add, void* ws,
                                          hipStream_t st) {
    q4nn_heads v[6] = {q, k, dq, dk, dq_in, dk_in}, *const at[6] = {v, v + 1, v + 2, v + 3, v + 4, v + 5};
    const q4nn_rope r = flat_batches(rope, at, 6);
    int64_t groups = 0;
    float* part = static_cast<float*>(ws);
    if (r.batches * r.tokens > 0 && r.q_heads + r.k_heads > 0) {
        const Shape s = shape_of(r);
        HeadsArgs a = args_of(r, s, true);
        for (int i = 0; i < 6; ++i) a.v[i] = v[i];
        a.part = part;
        groups = a.blocks < kMaxGroups ? a.blocks : kMaxGroups;
        launch_rows<true>(r, s, a, groups, st);
    }
    const dim3 g((unsigned)((2 * r.dim + 15) / 16)), b(1024);
    if (dtype == Q4MX_BF16 && add) k_gain_grads<true, true><<<g, b, 0, st>>>(part, groups, r.dim, gq, gk);
    else if (dtype == Q4MX_BF16) k_gain_grads<true, false><<<g, b, 0, st>>>(part, groups, r.dim, gq, gk);
    else if (add) k_gain_grads<false, true><<<g, b, 0, st>>>(part, groups, r.dim, gq, gk);
    else k_gain_grads<false, false><<<g, b, 0, st>>>(part, groups, r.dim, gq, gk);
    return hipGetLastError();
}

}  // namespace q4
