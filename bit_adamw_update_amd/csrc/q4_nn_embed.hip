// q4_nn_embed.hip -- rows of an embedding table and the table's gradient
// (gfx950).
#include "q4_mx_dev.h"
#include "q4_nn.h"

namespace q4 {
namespace {

__device__ __forceinline__ int64_t load_id(const Ids& ids, int64_t t) {
    return ids.type == Q4NN_I32 ? static_cast<const int32_t*>(ids.p)[t] : static_cast<const int64_t*>(ids.p)[t];
}

// ---- lookup -----------------------------------------------------------------
// Rows gathered and scaled: memory.  A lane takes 8 columns of a token; lanes
// follow the row-major order of the result, so odd widths leave none idle
// but at a row's end.
enum TableKind { TABLE_F32, TABLE_BF16, TABLE_MX };

template <int KIND, bool OUT_BF16>
__global__ __launch_bounds__(256) void k_embedding(Ids ids, Dense table, MxMat mx, int64_t rows, int64_t cols,
                                                    uint32_t chunks, float scale, Dense out) {
    const int64_t first = (int64_t)group_index() * 256;
    const int64_t t0 = first / chunks;
    const uint32_t at = (uint32_t)(first - t0 * chunks) + threadIdx.x, dt = at / chunks;
    const int64_t t = t0 + dt, col = (int64_t)(at - dt * chunks) * 8, left = cols - col;
    if (t >= ids.n) return;
    const int64_t id = load_id(ids, t);
    float v[8];
    if (id >= 0 && id < rows) {
        if (KIND == TABLE_MX) load_mx8(mx, id, col, v);
        else load8<KIND == TABLE_BF16>(table.p, id * table.ld + col, left, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= scale;
    } else {
        // padding, or a number that names no row, which has to show
        const float none = id < 0 ? 0.0f : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = none;
    }
    store8<OUT_BF16>(out.p, t * out.ld + col, left, v);
}

// ---- the table's gradient -----------------------------------------------------
// grad[v] = scale * the sum of dy[t] over the tokens with id v.  The tokens are
// sorted by (id, position), so that a row's gradients lie together and are
// summed in one order:
//   1. tiles of 1024 tokens are sorted in shared memory, and the gradient is
//      filled with zeros by the work-groups behind them: the sort is over long
//      before the fill of a large vocabulary's table is;
//   2. up to 16 sorted runs at a time are merged: an element's place is its
//      place in its own run plus the number of smaller ones in each other;
//   3. pieces of 32 sorted tokens are summed, a wave to 512 columns of a piece.
//      A row that lies within a piece is finished; one that crosses a piece's
//      end leaves FP32 sums in the workspace;
//   4. those are joined, in the order of the pieces.
// Keys are (id << 32) | position; a token that counts for no row has the id
// kNone and lies behind all others.
constexpr int kSortTile = 1024, kMergeRuns = 16, kPiece = 32, kSlab = 512, kJoinCols = 256, kJoinPieces = 16;
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr int64_t kFillBytes = 64 << 10;  // zeros of a work-group

__device__ __forceinline__ uint32_t id_of(uint64_t key) { return (uint32_t)(key >> 32); }

// Zeros into part `block` of grad (rows x cols elements of `unit` bytes).
struct Fill {
    void* p;
    int64_t rows, row_bytes, pitch;  // one row if the rows follow each other
    int64_t row_blocks;              // parts of a row
    int64_t blocks;
};
__device__ __forceinline__ void fill_zero(const Fill& f, int64_t block) {
    if (block >= f.blocks) return;
    const int64_t row = block / f.row_blocks, from = (block - row * f.row_blocks) * kFillBytes;
    const int64_t size = f.row_bytes - from < kFillBytes ? f.row_bytes - from : kFillBytes;
    char* p = static_cast<char*>(f.p) + row * f.pitch + from;
    for (int64_t i = threadIdx.x * 16; i < size; i += 256 * 16) {
        if (size - i >= 16) {
            *reinterpret_cast<u32x4_any*>(p + i) = u32x4_any{0, 0, 0, 0};
        } else {
            for (int64_t k = i; k < size; k += 2) *reinterpret_cast<uint16_t*>(p + k) = 0;
        }
    }
}

__global__ __launch_bounds__(256) void k_sort_tiles(Ids ids, int64_t rows, uint64_t* keys, int64_t tiles, Fill fill) {
    __shared__ uint64_t lds[kSortTile];
    const int64_t tile = group_index();
    if (tile >= tiles) return fill_zero(fill, tile - tiles);
    const int64_t first = tile * kSortTile;
#pragma unroll
    for (int j = 0; j < kSortTile / 256; ++j) {
        const int64_t t = first + j * 256 + threadIdx.x;
        uint64_t key = ~uint64_t(0);
        if (t < ids.n) {
            const int64_t id = load_id(ids, t);
            key = (uint64_t)(id >= 0 && id < rows ? (uint32_t)id : kNone) << 32 | (uint32_t)t;
        }
        lds[j * 256 + threadIdx.x] = key;
    }
    // bitonic: blocks of `size` alternate in direction
    for (int size = 2; size <= kSortTile; size *= 2)
        for (int step = size / 2; step > 0; step /= 2) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kSortTile / 512; ++j) {
                const int i = j * 256 + threadIdx.x, lo = 2 * i - (i & (step - 1)), hi = lo + step;
                const uint64_t a = lds[lo], b = lds[hi];
                if ((a > b) == ((lo & size) == 0)) lds[lo] = b, lds[hi] = a;
            }
        }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortTile / 256; ++j) {
        const int64_t t = first + j * 256 + threadIdx.x;
        if (t < ids.n) keys[t] = lds[j * 256 + threadIdx.x];
    }
}

// Runs of `run` keys, the last one shorter: each kMergeRuns neighbours become one.
__global__ __launch_bounds__(256) void k_merge_runs(const uint64_t* src, uint64_t* dst, int64_t n, int64_t run) {
    const int64_t i = (int64_t)group_index() * 256 + threadIdx.x;
    if (i >= n) return;
    const uint64_t key = src[i];
    const int64_t group = i / (run * kMergeRuns) * (run * kMergeRuns);
    int64_t place = i;
    for (int r = 0; r < kMergeRuns; ++r) {
        const int64_t begin = group + r * run;
        if (begin >= n) break;
        const int64_t end = begin + run < n ? begin + run : n;
        if (i >= begin && i < end) continue;
        int64_t lo = begin, hi = end;  // the first of this run that is larger (no two are equal)
        while (lo < hi) {
            const int64_t mid = lo + (hi - lo) / 2;
            if (src[mid] < key) lo = mid + 1;
            else hi = mid;
        }
        place += begin < i ? lo - end : lo - begin;  // those of a run before it that are larger move behind it
    }
    dst[place] = key;
}

// scale * sum into 8 columns of a row, or added to what is there; the first
// `left` of them exist.
template <bool BF16, bool ADD, int N>
__device__ __forceinline__ void store_grad(const Dense& grad, int64_t row, int64_t col, int64_t left, float scale,
                                           const float* sum) {
    const int64_t at = row * grad.ld + col;
    float v[8] = {};
    if (ADD) {
        if (N == 8) load8<BF16>(grad.p, at, left, v);
        else
            for (int k = 0; k < N; ++k) v[k] = k < left ? load1<BF16>(grad.p, at + k) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = ADD ? __builtin_fmaf(scale, sum[k], v[k]) : scale * sum[k];
    store8<BF16>(grad.p, at, left < N ? left : N, v);
}

struct GradArgs {
    const uint64_t* keys;
    int64_t n, pieces, slabs;
    const uint16_t* dy;
    int64_t lddy, cols, part_ld;
    float* part;  // [pieces][2][part_ld]: a row that the piece begins with and does not finish, and one that it ends with
    float scale;
    Dense grad;
};

template <bool BF16, bool ADD> __global__ __launch_bounds__(256) void k_grad_pieces(GradArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)group_index() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t piece = unit / a.slabs;
    if (piece >= a.pieces) return;
    const int64_t col = (unit - piece * a.slabs) * kSlab + lane * 8, left = a.cols - col;
    const int64_t begin = piece * kPiece;
    const int count = (int)(a.n - begin < kPiece ? a.n - begin : kPiece);
    const uint64_t key = lane < count ? a.keys[begin + lane] : ~uint64_t(0);
    const uint32_t id = id_of(key), token = (uint32_t)key;
    const uint32_t before = begin > 0 ? id_of(a.keys[begin - 1]) : kNone;
    const uint32_t behind = begin + count < a.n ? id_of(a.keys[begin + count]) : kNone;
    float sum[8] = {};
    uint32_t current = (uint32_t)__builtin_amdgcn_readlane((int)id, 0);
    int from = 0;
    auto finish = [&](int to) {
        const bool begun = from == 0 && before == current, goes_on = to == count && behind == current;
        if (left <= 0) return;
        if (!begun && !goes_on) {
            store_grad<BF16, ADD, 8>(a.grad, current, col, left, a.scale, sum);
        } else {
            float4* p = reinterpret_cast<float4*>(a.part + (piece * 2 + (from == 0 ? 0 : 1)) * a.part_ld + col);
            p[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            p[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
        }
    };
    for (int i = 0; i < count; i += 8) {
        float v[8][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // past the piece: its last token once more, not added
            const int at = i + j < count ? i + j : count - 1;
            const int64_t t = (uint32_t)__builtin_amdgcn_readlane((int)token, at);
            if (left > 0) load8<true>(a.dy, t * a.lddy + col, left, v[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (i + j >= count) break;
            const uint32_t now = (uint32_t)__builtin_amdgcn_readlane((int)id, i + j);
            if (now != current) {
                finish(i + j);
                current = now, from = i + j;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
            }
            if (now == kNone) return;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += v[j][k];
        }
    }
    finish(count);
}

// The rows that begin in one of 16 pieces and go on past its end: a wave adds
// every fourth of a row's sums, 4 columns to a lane, and the four waves' sums
// are added in order.
template <bool BF16, bool ADD> __global__ __launch_bounds__(256) void k_grad_join(GradArgs a, int64_t col_groups) {
    __shared__ float4 lds[4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t block = group_index(), pg = block / col_groups;
    const int64_t col = (block - pg * col_groups) * kJoinCols + lane * 4, left = a.cols - col;
    const int64_t mine = pg * kJoinPieces + lane;
    uint32_t last = kNone;
    bool owner = false, whole = false;
    if (lane < kJoinPieces && mine < a.pieces - 1) {
        const int64_t begin = mine * kPiece, end = begin + kPiece;  // not the last piece: it is full, and nothing follows that
        last = id_of(a.keys[end - 1]);
        const bool goes_on = last != kNone && id_of(a.keys[end]) == last;
        whole = id_of(a.keys[begin]) == last;
        owner = goes_on && !(whole && begin > 0 && id_of(a.keys[begin - 1]) == last);
    }
    uint64_t todo = __builtin_amdgcn_ballot_w64(owner);
    const uint64_t whole_mask = __builtin_amdgcn_ballot_w64(whole);
    while (todo) {
        const int at = __builtin_ctzll(todo);
        todo &= todo - 1;
        const uint32_t id = (uint32_t)__builtin_amdgcn_readlane((int)last, at);
        const int64_t piece = pg * kJoinPieces + at;
        // the pieces behind it that begin with this row
        int64_t more = 0;
        for (;;) {
            const int64_t q = piece + 1 + more + lane;
            const uint64_t other = __builtin_amdgcn_ballot_w64(!(q < a.pieces && id_of(a.keys[q * kPiece]) == id));
            if (other) {
                more += __builtin_ctzll(other);
                break;
            }
            more += 64;
        }
        float sum[4] = {};
        if (left > 0) {
            const float* own = a.part + (piece * 2 + ((whole_mask >> at) & 1 ? 0 : 1)) * a.part_ld + col;
            const float* next = a.part + (piece + 1) * 2 * a.part_ld + col;
            for (int64_t k = wave; k <= more; k += 4) {
                const float4 v = *reinterpret_cast<const float4*>(k == 0 ? own : next + (k - 1) * 2 * a.part_ld);
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
            }
        }
        __syncthreads();
        lds[wave][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        if (wave == 0 && left > 0) {
            for (int w = 1; w < 4; ++w) {
                const float4 v = lds[w][lane];
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
            }
            store_grad<BF16, ADD, 4>(a.grad, id, col, left, a.scale, sum);
        }
    }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t parts_of(int64_t n, int64_t part) { return (n + part - 1) / part; }

template <bool BF16, bool ADD> void launch_sums(const GradArgs& a, hipStream_t st) {
    k_grad_pieces<BF16, ADD><<<grid_of(parts_of(a.pieces * a.slabs, 4)), dim3(256), 0, st>>>(a);
    if (a.pieces > 1) {
        const int64_t cg = parts_of(a.cols, kJoinCols);
        k_grad_join<BF16, ADD><<<grid_of(parts_of(a.pieces - 1, kJoinPieces) * cg), dim3(256), 0, st>>>(a, cg);
    }
}

}  // namespace

hipError_t launch_embedding(const Ids& ids, const Dense& table, const MxMat& mx, int64_t rows, int64_t cols,
                            float scale, const Dense& out, hipStream_t st) {
    const uint32_t chunks = (uint32_t)parts_of(cols, 8);
    const dim3 g = grid_of(parts_of(ids.n * chunks, 256)), b(256);
    const bool bf = out.dtype == Q4MX_BF16;
#define Q4_EMBED(K, O) k_embedding<K, O><<<g, b, 0, st>>>(ids, table, mx, rows, cols, chunks, scale, out)
    if (mx.codes || rows == 0) {
        if (bf) Q4_EMBED(TABLE_MX, true);
        else Q4_EMBED(TABLE_MX, false);
    } else if (table.dtype == Q4MX_BF16) {
        if (bf) Q4_EMBED(TABLE_BF16, true);
        else Q4_EMBED(TABLE_BF16, false);
    } else {
        if (bf) Q4_EMBED(TABLE_F32, true);
        else Q4_EMBED(TABLE_F32, false);
    }
#undef Q4_EMBED
    return hipGetLastError();
}

size_t embedding_grad_workspace(int64_t tokens, int64_t cols) {
    if (tokens == 0) return 0;
    const size_t keys = round256(sizeof(uint64_t) * (size_t)tokens);
    const size_t part = sizeof(float) * (size_t)(parts_of(tokens, kPiece) * 2 * parts_of(cols, 8) * 8);
    return 2 * keys + (tokens > kPiece ? part : 0);
}

hipError_t launch_embedding_grad(const Ids& ids, const Dense& dy, float scale, int64_t rows, int64_t cols,
                                 const Dense& grad, bool add, void* ws, hipStream_t st) {
    const int64_t n = ids.n, tiles = parts_of(n, kSortTile);
    Fill fill = {};
    if (!add) {
        const int64_t unit = grad.dtype == Q4MX_BF16 ? 2 : 4;
        const bool flat = grad.ld == cols || rows == 1;
        fill.p = grad.p;
        fill.rows = flat ? 1 : rows;
        fill.row_bytes = (flat ? rows * cols : cols) * unit;
        fill.pitch = grad.ld * unit;
        fill.row_blocks = parts_of(fill.row_bytes, kFillBytes);
        fill.blocks = fill.rows * fill.row_blocks;
    }
    uint64_t* keys = static_cast<uint64_t*>(ws);
    uint64_t* other = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + round256(sizeof(uint64_t) * (size_t)n));
    k_sort_tiles<<<grid_of(tiles + fill.blocks), dim3(256), 0, st>>>(ids, rows, keys, tiles, fill);
    if (n == 0) return hipGetLastError();
    GradArgs a = {};
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * round256(sizeof(uint64_t) * (size_t)n));
    for (int64_t run = kSortTile; run < n; run *= kMergeRuns) {
        k_merge_runs<<<grid_of(parts_of(n, 256)), dim3(256), 0, st>>>(keys, other, n, run);
        uint64_t* t = keys;
        keys = other, other = t;
    }
    a.keys = keys, a.n = n, a.pieces = parts_of(n, kPiece), a.slabs = parts_of(cols, kSlab);
    a.dy = static_cast<const uint16_t*>(dy.p), a.lddy = dy.ld;
    a.cols = cols, a.part_ld = parts_of(cols, 8) * 8;
    a.scale = scale, a.grad = grad;
    const bool bf = grad.dtype == Q4MX_BF16;
    if (bf && add) launch_sums<true, true>(a, st);
    else if (bf) launch_sums<true, false>(a, st);
    else if (add) launch_sums<false, true>(a, st);
    else launch_sums<false, false>(a, st);
    return hipGetLastError();
}

}  // namespace q4
