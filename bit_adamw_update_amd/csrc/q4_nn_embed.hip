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
// Rows gathered and scaled: memory (16384 tokens x 2560 from FP32 masters: 31 us,
// 107 MB read and 84 written at 6.1 TB/s, part of it from the last-level cache;
// from BF16, E4M3 and E2M1 23 us, 52, 48 and 34 MB read where the rows that are
// named have 31, 16 and 8: several XCDs read the same ones, and a row's scales
// are 4 bytes of a cache line for every 128 columns; one token's row of E2M1: 1.7
// us).  A lane takes 8 columns of a token; lanes
// follow the row-major order of the result, so odd widths leave none idle but
// at a row's end.
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
//      before the fill of a large vocabulary's table is, and writes alone run
//      at 6.6 to 7.9 TB/s where reads and writes together reach 5.1;
//   2. up to 16 sorted runs at a time are merged: an element's place is the
//      number of smaller ones in all of them (unless the first step placed it
//      already);
//   3. a wave takes the rows that begin in a piece of 2 to 32 sorted tokens, 512
//      columns of them.  A row of up to 32 tokens is summed whole, past the
//      piece's end where it has to; of a longer one every piece that it touches
//      leaves an FP32 sum in the workspace;
//   4. those are joined, in the order of the pieces.
// Up to 1024 tokens take all of that in one launch (k_grad_small).
// Memory bounds the large cases: 16384 tokens into 50304 x 2560 33 + 27 + 6 us
// (258 MB of zeros at 7.8 TB/s, 117 MB of sums at 4.4), 8192 into 151936 x 1024
// 46 + 10 + 5 (311 MB at 6.8; the rest is latency).
// Keys are (id << 32) | position; a token that counts for no row has the id
// kNone and lies behind all others.
constexpr int kSortTile = 1024, kMergeRuns = 16, kShort = 32, kSlab = 512;
// A sort that needs no merges (RANKED below) where the fill beside it takes
// longer: kHides bytes of zeros a tile, 1.5 us (8192 tokens into 151936 x 1024:
// 70.6 us, with merges 75.0; into 1000 x 64, with 16384 tokens: 40.3 and 26.2).
// Beside less, or added to a gradient, it gains nothing for few tiles either, in a
// graph: 2, 4, 8 tiles into 2000 x 768 20.0, 23.8, 30.9 us, with merges 19.9, 21.6,
// 24.2; added to it 20.8, 25.3, 32.2 and 20.6, 23.0, 25.5.
constexpr int64_t kRanked = 65536, kHides = 12 << 20;
constexpr int kJoinCols = 256, kJoinPieces = 8, kJoinWaves = 8;
constexpr uint32_t kNone = 0x80000000u;   // above every id; one more is a number too

__device__ __forceinline__ uint32_t id_of(uint64_t key) { return (uint32_t)(key >> 32); }

// Zeros into 16-byte pieces of grad, the last of a row shorter.
struct Fill {
    char* p;
    int64_t row_bytes, pitch;  // one row if the rows follow each other
    int64_t row_pieces, end;   // of all pieces, up to `end`
};
constexpr int kFillRounds = 8;  // pieces of a thread
template <int THREADS> __device__ __forceinline__ void fill_zero(const Fill& f, int64_t first) {
    const int64_t row = first / f.row_pieces;
    const uint32_t at = (uint32_t)(first - row * f.row_pieces);
#pragma unroll
    for (int k = 0; k < kFillRounds; ++k) {
        int64_t r = 0, i = first + k * THREADS + threadIdx.x;
        if (i >= f.end) return;
        if (f.pitch != 0) {
            const uint32_t local = at + k * THREADS + threadIdx.x, rows = local / (uint32_t)f.row_pieces;
            r = row + rows, i = local - rows * (uint32_t)f.row_pieces;
        }
        char* p = f.p + r * f.pitch + i * 16;
        const int64_t size = f.row_bytes - i * 16;
        if (size >= 16) {
            *reinterpret_cast<u32x4_any*>(p) = u32x4_any{0, 0, 0, 0};
        } else {
            for (int64_t n = 0; n < size; n += 2) *reinterpret_cast<uint16_t*>(p + n) = 0;
        }
    }
}

// The number of the 2^LOG sorted ids from `run` on that are below `bound`.
template <int LOG> __device__ __forceinline__ int count_below(const uint32_t* run, uint32_t bound) {
    int pos = 0;
#pragma unroll
    for (int step = 1 << (LOG - 1); step > 0; step /= 2)
        if (run[pos + step - 1] < bound) pos += step;
    return pos + (run[pos] < bound ? 1 : 0);
}

// A thread's id of one of four neighbouring sorted runs of 2^LOG: its place
// among all of them.  Equal ids keep the order of the runs.
template <int LOG> __device__ __forceinline__ int place_in_four(const uint32_t* four, int at, uint32_t id) {
    const int own = at >> LOG;
    int place = at & ((1 << LOG) - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int below = count_below<LOG>(four + (r << LOG), id + (r < own ? 1u : 0u));
        if (r != own) place += below;
    }
    return place;
}

__device__ __forceinline__ uint32_t valid_id(const Ids& ids, int64_t rows, int64_t t) {
    const int64_t v = t < ids.n ? load_id(ids, t) : -1;
    return v >= 0 && v < rows ? (uint32_t)v : kNone;
}

// A tile of 1024 tokens, the ids of those past the last kNone, sorted by a
// work-group: a thread's id, token and place.  A wave ranks its 64 ids by
// comparing each with each (equal ones by their position); four such runs, and
// then four of 256, become one by binary searches in shared memory.  (A bitonic
// sort's 55 exchanges took 11.8 us, 15 searches of 64 at once 7.2, this 5.7.)
struct SortRoom {
    uint32_t id[2][kSortTile], token[2][kSortTile];
};
struct Sorted {
    uint32_t id, token;
    int place;
};
__device__ __forceinline__ Sorted sort_tile(const Ids& ids, int64_t rows, int64_t tile, SortRoom& room) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t id = valid_id(ids, rows, tile * kSortTile + tid);
    // waves, and groups of 256, that lie past the last token hold kNone alone and stay as they are
    const bool wave_real = tile * kSortTile + (tid & ~63) < ids.n, group_real = tile * kSortTile + (tid & ~255) < ids.n;
    int rank = lane;
    if (wave_real) {
        rank = 0;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
            const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)id, j);
            rank += other < id + (j < lane ? 1u : 0u) ? 1 : 0;
        }
    }
    room.id[0][wave * 64 + rank] = id;
    room.token[0][wave * 64 + rank] = (uint32_t)(tile * kSortTile + tid);
    __syncthreads();
    Sorted s = {room.id[0][tid], room.token[0][tid], tid};
    if (group_real) s.place = (tid & ~255) + place_in_four<6>(room.id[0] + (tid & ~255), tid & 255, s.id);
    if (ids.n > 256) {
        room.id[1][s.place] = s.id;
        room.token[1][s.place] = s.token;
        __syncthreads();
        s = {room.id[1][tid], room.token[1][tid], tid};
        if (group_real) s.place = place_in_four<8>(room.id[1], tid, s.id);
    }
    return s;  // room.id[0] is free where there are more than 256 tokens
}

// RANKED (more than one tile): a tile finds its places among all tokens by
// itself.  It looks every other tile's ids up in its own sorted ones and counts
// them there: what is counted up to an element lies before it.  That takes 1.5
// us for each of the others (shared memory's rate), and saves the merges'
// launches.
template <bool RANKED>
__global__ __launch_bounds__(kSortTile) void k_sort_tiles(Ids ids, int64_t rows, uint64_t* keys, int64_t tiles,
                                                           Fill fill) {
    __shared__ SortRoom room;
    __shared__ uint32_t counted[RANKED ? kSortTile + 1 : 1], of_wave[16];
    const int64_t tile = group_index();
    if (tile >= tiles) return fill_zero<kSortTile>(fill, (tile - tiles) * (kSortTile * kFillRounds));
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Sorted s = sort_tile(ids, rows, tile, room);
    uint32_t* const sorted = room.id[0];
    int64_t before = tile * kSortTile;
    if (RANKED) {
        sorted[s.place] = s.id;
        counted[tid] = 0;
        if (tid == 0) counted[kSortTile] = 0;
        __syncthreads();
        constexpr int kAtOnce = 4;
        for (int64_t first = 0; first < tiles; first += kAtOnce) {
            uint32_t below[kAtOnce];
            int at[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                // of equal ids, those of a tile before this one come first
                below[k] = valid_id(ids, rows, (first + k) * kSortTile + tid) + (first + k < tile ? 0u : 1u);
                at[k] = 0;
            }
            // side by side: a step of one waits for shared memory
#pragma unroll
            for (int step = kSortTile / 2; step > 0; step /= 2)
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) at[k] += sorted[at[k] + step - 1] < below[k] ? step : 0;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) at[k] += sorted[at[k]] < below[k] ? 1 : 0;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (first + k != tile && (first + k) * kSortTile + tid < ids.n) atomicAdd(&counted[at[k]], 1u);
        }
        __syncthreads();
        // the running sums of `counted`
        int sum = (int)counted[tid];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int up = __shfl_up(sum, m);
            if (lane >= m) sum += up;
        }
        if (lane == 63) of_wave[wave] = (uint32_t)sum;
        __syncthreads();
        for (int w = 0; w < wave; ++w) sum += (int)of_wave[w];
        counted[tid] = (uint32_t)sum;
        __syncthreads();
        before = counted[s.place];
    }
    // past the last token: ids of kNone from the end of the last tile, the last of all
    if (s.token < ids.n) keys[before + s.place] = (uint64_t)s.id << 32 | s.token;
}

// Runs of `run` keys, the last one shorter: each kMergeRuns neighbours become
// one.  A wave takes one run, its lanes 64 neighbouring keys of any: their
// searches share cache lines step by step (10.8 us for the first merge of 65536
// keys; a lane to a run, 16 to a key: 17.9; a thread to a key, run after run: 32
// for 16384 keys).
__global__ __launch_bounds__(64 * kMergeRuns) void k_merge_runs(const uint64_t* src, uint64_t* dst, int64_t n,
                                                                int64_t run) {
    __shared__ uint32_t smaller[kMergeRuns][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = (int64_t)group_index() * 64, i = first + lane;
    if (first >= n) return;
    const int64_t group = first / (run * kMergeRuns) * (run * kMergeRuns);  // of all 64: runs are multiples of 64
    const int64_t begin = group + wave * run, end = begin + run < n ? begin + run : n;
    const uint64_t key = src[i < n ? i : n - 1];
    int64_t lo = begin, hi = end > begin ? end : begin;  // the first of this run that is not smaller (no two are equal)
    if (first >= lo && first < hi) lo = hi = i;
    while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (src[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    smaller[wave][lane] = (uint32_t)(lo - begin);
    __syncthreads();
    if (wave != 0 || i >= n) return;
    int64_t place = group;
#pragma unroll
    for (int r = 0; r < kMergeRuns; ++r) place += smaller[r][lane];
    dst[place] = key;
}

// scale * sum into 8 columns of a row, or added to what is there.
template <bool BF16, bool ADD>
__device__ __forceinline__ void store_grad8(const Dense& grad, int64_t at, float scale, const float* sum) {
    float v[8];
    if (ADD) load8<BF16>(grad.p, at, 8, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = ADD ? __builtin_fmaf(scale, sum[k], v[k]) : scale * sum[k];
    store8<BF16>(grad.p, at, 8, v);
}
// The same of N columns, of which those before `skip` and from `left` on are
// another lane's, or do not exist.
template <bool BF16, bool ADD, int N>
__device__ __forceinline__ void store_grad_some(const Dense& grad, int64_t at, int skip, int64_t left, float scale,
                                                const float* sum) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (k < skip || k >= left) continue;
        const float v = ADD ? __builtin_fmaf(scale, sum[k], load1<BF16>(grad.p, at + k)) : scale * sum[k];
        if (BF16) static_cast<uint16_t*>(grad.p)[at + k] = bf16_bits(v);
        else static_cast<float*>(grad.p)[at + k] = v;
    }
}

struct GradArgs {
    const uint64_t* keys;
    int64_t n, pieces, slabs;
    int piece;  // tokens of one
    const uint16_t* dy;
    int64_t lddy, cols, part_ld;
    float* part;     // [pieces][2][part_ld]: of a long row that the piece begins with, and of one that begins behind that
    uint32_t* long_begins;  // [pieces]: 0, or 1 + the place in part of the long row that begins in this piece
    float scale;
    Dense grad;
};

// WHOLE: whole vectors of 8 columns, whose code is a third of the others'
// (the walk below holds a row's end 16 times, and has to fit the instruction
// cache).  RAGGED: a lane whose 8 columns pass the end takes the last 8, and
// stores those that are its own.  NARROW: fewer than 8 columns.
enum Columns { WHOLE, RAGGED, NARROW };

// A lane's 8 columns of a slab.  Lanes past the columns go along on the first
// ones and store nothing: all 64 of a wave hold a token that it reads.
template <int COLS> struct LaneColumns {
    int64_t at;    // the first
    int skip;      // of the 8, that another lane stores
    int64_t here;  // of the 8, that exist
    bool whole;
    __device__ __forceinline__ LaneColumns(int64_t cols, int64_t slab) {
        const int lane = threadIdx.x & 63;
        const int64_t col = slab * kSlab + lane * 8, left = cols - col;
        at = COLS == NARROW ? 0 : left >= 8 ? col : left > 0 ? cols - 8 : 0;
        skip = left >= 8 || COLS == NARROW ? 0 : left > 0 ? (int)(8 - left) : 8;
        here = COLS == NARROW ? (lane == 0 ? cols : 0) : 8;
        whole = skip == 0 && here == 8;
    }
};
template <int COLS> __device__ __forceinline__ u32x4_any load_grad(const uint16_t* p, const LaneColumns<COLS>& c) {
    if (COLS != NARROW) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = k < c.here ? p[k] : 0;
    return u32x4_any{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
}
__device__ __forceinline__ void add8(float* sum, const u32x4_any& raw) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        sum[2 * k] += bf16_value(raw[k] & 0xFFFFu);
        sum[2 * k + 1] += __uint_as_float(raw[k] & 0xFFFF0000u);
    }
}
template <bool BF16, bool ADD, int COLS>
__device__ __forceinline__ void store_row(const GradArgs& a, uint32_t id, const LaneColumns<COLS>& c, const float* sum) {
    if (c.whole) store_grad8<BF16, ADD>(a.grad, id * a.grad.ld + c.at, a.scale, sum);
    else if (COLS != WHOLE) store_grad_some<BF16, ADD, 8>(a.grad, id * a.grad.ld + c.at, c.skip, c.here, a.scale, sum);
}

// The tokens of lanes from .. end - 1, by whole rows: row_end(id, first lane,
// lane behind the last, sums) at each row's end.
template <int COLS, class RowEnd>
__device__ __forceinline__ void walk_tokens(const GradArgs& a, uint32_t id, uint32_t token, int from, int end,
                                            const LaneColumns<COLS>& c, RowEnd row_end) {
    constexpr int kBatch = 16;
    float sum[8] = {};
    uint32_t current = (uint32_t)__builtin_amdgcn_readlane((int)id, from);
    int begun = from;
    for (int i = from; i < end; i += kBatch) {
        u32x4_any raw[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            // past the end: the last token once more, not added
            const int e = i + j < end ? i + j : end - 1;
            raw[j] = load_grad<COLS>(a.dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)token, e) * a.lddy + c.at, c);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (i + j >= end) break;
            const uint32_t now = (uint32_t)__builtin_amdgcn_readlane((int)id, i + j);
            if (now != current) {
                row_end(current, begun, i + j, sum);
                current = now, begun = i + j;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
            }
            add8(sum, raw[j]);
        }
    }
    row_end(current, begun, end, sum);
}

template <bool BF16, bool ADD, int COLS> __global__ __launch_bounds__(256) void k_grad_pieces(GradArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)group_index() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t piece = unit / a.slabs, slab = unit - piece * a.slabs;
    if (piece >= a.pieces) return;
    const int64_t begin = piece * a.piece;
    // the piece and what is behind it, 64 tokens; the 32 before it
    const uint64_t key = begin + lane < a.n ? a.keys[begin + lane] : ~uint64_t(0);
    const uint32_t id = id_of(key), token = (uint32_t)key;
    const uint32_t before = lane < kShort && begin - kShort + lane >= 0 ? id_of(a.keys[begin - kShort + lane]) : ~0u;
    const int real = __builtin_popcountll(__builtin_amdgcn_ballot_w64(id < kNone));
    const int count = real < a.piece ? real : a.piece;
    int from = 0, end = 0;
    bool first_long = false, last_long = false;
    if (count > 0) {
        const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)id, 0);
        const int back = __builtin_popcountll(__builtin_amdgcn_ballot_w64(before == first));
        const int ahead = __builtin_popcountll(__builtin_amdgcn_ballot_w64(id == first));
        first_long = back > 0 && back + ahead > kShort;
        from = back > 0 && !first_long ? ahead : 0;  // a short row that began before is another wave's
    }
    if (from < count) {
        const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)id, count - 1);
        const uint64_t mask = __builtin_amdgcn_ballot_w64(id == last);
        const int start = __builtin_ctzll(mask), length = __builtin_popcountll(mask);
        last_long = (start > 0 || !first_long) && length > kShort;  // begins here, and more than 32 follow
        end = last_long || (start == 0 && first_long) ? (start + length < a.piece ? start + length : a.piece) : start + length;
        if (slab == 0 && lane == 0) a.long_begins[piece] = last_long ? (start == 0 ? 1 : 2) : 0;
    } else {
        if (slab == 0 && lane == 0) a.long_begins[piece] = 0;
        return;
    }
    const LaneColumns<COLS> c(a.cols, slab);
    walk_tokens<COLS>(a, id, token, from, end, c, [&](uint32_t row, int begun, int to, const float* sum) {
        if ((begun == 0 && first_long) || (to == end && last_long)) {
            float* p = a.part + (piece * 2 + (begun == 0 ? 0 : 1)) * a.part_ld + c.at;
            if (c.whole) {
                *reinterpret_cast<float4*>(p) = make_float4(sum[0], sum[1], sum[2], sum[3]);
                *reinterpret_cast<float4*>(p + 4) = make_float4(sum[4], sum[5], sum[6], sum[7]);
            } else if (COLS != WHOLE) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= c.skip && k < c.here) p[k] = sum[k];
            }
        } else {
            store_row<BF16, ADD, COLS>(a, row, c, sum);
        }
    });
}

// The long rows that begin in one of 8 pieces: a wave adds every eighth of a
// row's sums, 4 columns to a lane, and the waves' sums are added in order.
template <bool BF16, bool ADD> __global__ __launch_bounds__(64 * kJoinWaves) void k_grad_join(GradArgs a, int64_t col_groups) {
    __shared__ float4 lds[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t block = group_index(), pg = block / col_groups;
    const int64_t col = (block - pg * col_groups) * kJoinCols + lane * 4, left = a.cols - col;
    // of 64 pieces from the group's first on: the ids that they begin and end with (its long row's, if one begins there)
    const int64_t mine = pg * kJoinPieces + lane, first = mine * a.piece, last = first + a.piece - 1;
    const uint32_t slot = lane < kJoinPieces && mine < a.pieces ? a.long_begins[mine] : 0;
    const uint32_t begins = first < a.n ? id_of(a.keys[first]) : ~0u;
    const uint32_t ends = id_of(a.keys[last < a.n ? last : a.n - 1]);
    uint64_t todo = __builtin_amdgcn_ballot_w64(slot != 0);
    while (todo) {
        const int which = __builtin_ctzll(todo);
        todo &= todo - 1;
        const int64_t piece = pg * kJoinPieces + which;
        const uint32_t id = (uint32_t)__builtin_amdgcn_readlane((int)ends, which);
        // the pieces behind it that begin with this row
        const uint64_t same = __builtin_amdgcn_ballot_w64(lane > which && begins == id);
        int64_t more = __builtin_popcountll(same);
        while (which + 1 + more >= 64) {
            const int64_t q = piece + 1 + more + lane;
            const uint64_t other = __builtin_amdgcn_ballot_w64(!(q < a.pieces && id_of(a.keys[q * a.piece]) == id));
            if (other) {
                more += __builtin_ctzll(other);
                break;
            }
            more += 64;
        }
        float sum[4] = {};
        const int own_slot = __builtin_amdgcn_readlane((int)slot, which) - 1;
        if (left > 0) {
            const float* own = a.part + (piece * 2 + own_slot) * a.part_ld + col;
            const float* next = a.part + (piece + 1) * 2 * a.part_ld + col;
#pragma unroll 8
            for (int64_t k = wave; k <= more; k += kJoinWaves) {
                const float4 v = *reinterpret_cast<const float4*>(k == 0 ? own : next + (k - 1) * 2 * a.part_ld);
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
            }
        }
        __syncthreads();
        lds[wave][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        if (wave == 0 && left > 0) {
#pragma unroll
            for (int w = 1; w < kJoinWaves; ++w) {
                const float4 v = lds[w][lane];
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
            }
            store_grad_some<BF16, ADD, 4>(a.grad, id * a.grad.ld + col, 0, left, a.scale, sum);
        }
    }
}

// Up to 1024 tokens in one launch: every work-group sorts them all for itself.
// The first ones then sum: a wave the short rows that begin in two sorted
// tokens, and all 16 together the long row that begins in the work-group's 32,
// if one does (it passes their end, so there is at most one).  All of them fill
// their share of the rows that no token reads.
constexpr int kSmallPiece = 2, kSegment = 16 * kSmallPiece;
static_assert(kSegment <= kShort, "two long rows could begin in one segment");
struct SmallArgs {
    Ids ids;
    int64_t rows, row_bytes, pitch, sum_groups;
    uint32_t row_pieces;  // 16 bytes each, the last one shorter
    int group_rows;       // rows of a work-group to fill, at most kSortTile
};
template <bool BF16, bool ADD, int COLS> __global__ __launch_bounds__(kSortTile) void k_grad_small(SmallArgs m, GradArgs a) {
    __shared__ SortRoom room;
    __shared__ uint32_t id_at[kSortTile], token_at[kSortTile];
    __shared__ float4 lds[16][64][2];
    __shared__ int long_begin;
    __shared__ bool touched[kSortTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t group = group_index();
    {
        const Sorted s = sort_tile(m.ids, m.rows, 0, room);
        id_at[s.place] = s.id, token_at[s.place] = s.token;
    }
    if (tid == 0) long_begin = -1;
    __syncthreads();
    if (group < m.sum_groups) {
        const int64_t segment = group / a.slabs, slab = group - segment * a.slabs;
        const LaneColumns<COLS> c(a.cols, slab);
        const int begin = (int)segment * kSegment + wave * kSmallPiece, at = begin + lane, ahead_of = begin - kShort + lane;
        const uint32_t id = at < kSortTile ? id_at[at] : ~0u, token = at < kSortTile ? token_at[at] : 0u;
        const uint32_t before = lane < kShort && ahead_of >= 0 ? id_at[ahead_of] : ~0u;
        const int real = __builtin_popcountll(__builtin_amdgcn_ballot_w64(id < kNone));
        const int count = real < kSmallPiece ? real : kSmallPiece;
        int from = 0, end = 0;
        if (count > 0) {
            const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)id, 0);
            const bool begun = __builtin_amdgcn_ballot_w64(before == first) != 0;
            from = begun ? __builtin_popcountll(__builtin_amdgcn_ballot_w64(id == first)) : 0;
        }
        if (from < count) {
            const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)id, count - 1);
            const uint64_t mask = __builtin_amdgcn_ballot_w64(id == last);
            const int start = __builtin_ctzll(mask), length = __builtin_popcountll(mask);
            end = length > kShort ? start : start + length;
            if (length > kShort && lane == 0) long_begin = begin + start;
            if (from < end)
                walk_tokens<COLS>(a, id, token, from, end, c, [&](uint32_t row, int, int, const float* sum) {
                    store_row<BF16, ADD, COLS>(a, row, c, sum);
                });
        }
        __syncthreads();
        const int first = long_begin;
        if (first >= 0) {
            const uint32_t row = id_at[first];
            const int stop = count_below<10>(id_at, row + 1);
            float sum[8] = {};
            constexpr int kBatch = 8;
            for (int i = first + wave; i < stop; i += 16 * kBatch) {
                u32x4_any raw[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int e = i + 16 * j < stop ? i + 16 * j : i;
                    raw[j] = load_grad<COLS>(a.dy + (int64_t)token_at[e] * a.lddy + c.at, c);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (i + 16 * j < stop) add8(sum, raw[j]);
            }
            lds[wave][lane][0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            lds[wave][lane][1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int w = 1; w < 16; ++w) {
                    const float4 u = lds[w][lane][0], v = lds[w][lane][1];
                    sum[0] += u.x, sum[1] += u.y, sum[2] += u.z, sum[3] += u.w;
                    sum[4] += v.x, sum[5] += v.y, sum[6] += v.z, sum[7] += v.w;
                }
                store_row<BF16, ADD, COLS>(a, row, c, sum);
            }
        }
    }
    if (ADD) return;
    const int64_t first_row = group * m.group_rows;
    if (first_row >= m.rows) return;
    const int n_rows = (int)(m.rows - first_row < m.group_rows ? m.rows - first_row : m.group_rows);
    if (tid < n_rows) {
        const uint32_t row = (uint32_t)(first_row + tid);
        const int place = count_below<10>(id_at, row);
        touched[tid] = place < kSortTile && id_at[place] == row;
    }
    __syncthreads();
    const uint32_t step_rows = kSortTile / m.row_pieces, step_pieces = kSortTile - step_rows * m.row_pieces;
    uint32_t row = tid / m.row_pieces, piece = tid - row * m.row_pieces;
    while (row < (uint32_t)n_rows) {
        if (!touched[row]) {
            char* p = static_cast<char*>(a.grad.p) + (first_row + row) * m.pitch + (int64_t)piece * 16;
            const int64_t size = m.row_bytes - (int64_t)piece * 16;
            if (size >= 16) {
                *reinterpret_cast<u32x4_any*>(p) = u32x4_any{0, 0, 0, 0};
            } else {
                for (int64_t k = 0; k < size; k += 2) *reinterpret_cast<uint16_t*>(p + k) = 0;
            }
        }
        row += step_rows, piece += step_pieces;
        if (piece >= m.row_pieces) piece -= m.row_pieces, ++row;
    }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t parts_of(int64_t n, int64_t part) { return (n + part - 1) / part; }

template <bool BF16, bool ADD> void launch_sums(const GradArgs& a, hipStream_t st) {
    const dim3 g = grid_of(parts_of(a.pieces * a.slabs, 4)), b(256);
    if (a.cols < 8) k_grad_pieces<BF16, ADD, NARROW><<<g, b, 0, st>>>(a);
    else if (a.cols % 8 != 0) k_grad_pieces<BF16, ADD, RAGGED><<<g, b, 0, st>>>(a);
    else k_grad_pieces<BF16, ADD, WHOLE><<<g, b, 0, st>>>(a);
    if (a.n > kShort) {
        const int64_t cg = parts_of(a.cols, kJoinCols);
        k_grad_join<BF16, ADD><<<grid_of(parts_of(a.pieces, kJoinPieces) * cg), dim3(64 * kJoinWaves), 0, st>>>(a, cg);
    }
}

template <bool BF16, bool ADD> void launch_small(SmallArgs m, const GradArgs& a, hipStream_t st) {
    m.sum_groups = parts_of(a.n, kSegment) * a.slabs;
    const int64_t fill = ADD ? 0 : parts_of(m.rows, m.group_rows);
    const dim3 g = grid_of(fill > m.sum_groups ? fill : m.sum_groups, kSortTile), b(kSortTile);
    if (a.cols < 8) k_grad_small<BF16, ADD, NARROW><<<g, b, 0, st>>>(m, a);
    else if (a.cols % 8 != 0) k_grad_small<BF16, ADD, RAGGED><<<g, b, 0, st>>>(m, a);
    else k_grad_small<BF16, ADD, WHOLE><<<g, b, 0, st>>>(m, a);
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

// Few pieces leave compute units idle and a wave's time is its steps': shorter
// ones; for many, fewer sums of long rows count: longer ones.  Microseconds of a
// call with pieces of 2, 4, 8, 16, 32: 301 tokens x 100 columns 12.5, 12.7, 13.7,
// 15.8, 19.4; 2048 x 768 25.5, 24.4, 24.3, 26.1, 30.7; 4096 x 1024 31.5, 29.2,
// 28.8, 30.4, 34.2; 16384 x 2560 110, 88, 79, 76.5, 78; 131072 x 512 223, 164,
// 133, 121, 117.  The wave sees 64 tokens from the piece's first on, so kShort +
// the piece is at most 64.
int piece_of(int64_t tokens, int64_t cols) {
    const int64_t n = tokens * parts_of(cols, kSlab);
    return n <= 1024 ? 2 : n <= 4096 ? 4 : n <= 16384 ? 8 : n < 131072 ? 16 : 32;
}

// The parts of a gradient's workspace: keys twice, the pieces' flags, the long rows' sums.
struct GradWorkspace {
    size_t keys, flags, part;
    GradWorkspace(int64_t tokens, int64_t cols) {
        const int64_t pieces = parts_of(tokens, piece_of(tokens, cols));
        keys = round256(sizeof(uint64_t) * (size_t)tokens);
        flags = round256(sizeof(uint32_t) * (size_t)pieces);
        part = tokens > kShort ? sizeof(float) * (size_t)(pieces * 2 * parts_of(cols, 8) * 8) : 0;
    }
};
size_t embedding_grad_workspace(int64_t tokens, int64_t cols) {
    const GradWorkspace w(tokens, cols);
    return tokens == 0 ? 0 : 2 * w.keys + w.flags + w.part;
}

// The form in one launch (k_grad_small): while its work-groups, one to a compute
// unit, run at once, and the zeros are few enough to wait for the sort in each
// of them.  Microseconds of a call, outside of a graph, and of the other form:
// 301 tokens x 100 into 1000 rows 10.1, 14.4; 1024 x 4096 into 500 13.8, 16.4;
// 1024 x 5120 18.9, 17.8; x 16384 39, 22; 1000 x 1024 into 4000 13.5, 15.6; in a
// graph 1000 x 256 into 32000 (16 MB) 20.0, 15.8.
constexpr int64_t kSmallGroups = 256, kSmallFill = 8 << 20, kSmallGroupFill = 32 << 10;
bool small(int64_t tokens, int64_t cols, int64_t fill_bytes) {
    return tokens > 0 && tokens <= kSortTile && fill_bytes <= kSmallFill &&
           parts_of(tokens, kSegment) * parts_of(cols, kSlab) <= kSmallGroups;
}

hipError_t launch_embedding_grad(const Ids& ids, const Dense& dy, float scale, int64_t rows, int64_t cols,
                                 const Dense& grad, bool add, void* ws, hipStream_t st) {
    const int64_t n = ids.n, tiles = parts_of(n, kSortTile);
    const int64_t unit = grad.dtype == Q4MX_BF16 ? 2 : 4, row_bytes = cols * unit;
    const bool bf = grad.dtype == Q4MX_BF16;
    GradArgs a = {};
    a.n = n, a.slabs = parts_of(cols, kSlab);
    a.dy = static_cast<const uint16_t*>(dy.p), a.lddy = dy.ld;
    a.cols = cols, a.scale = scale, a.grad = grad;
    if (small(n, cols, add ? 0 : rows * row_bytes)) {
        SmallArgs m = {};
        m.ids = ids, m.rows = rows, m.row_bytes = row_bytes, m.pitch = grad.ld * unit;
        m.row_pieces = (uint32_t)parts_of(row_bytes, 16);
        const int64_t most = kSmallGroupFill / row_bytes;
        m.group_rows = most < 1 ? 1 : most > kSortTile ? kSortTile : (int)most;
        if (bf && add) launch_small<true, true>(m, a, st);
        else if (bf) launch_small<true, false>(m, a, st);
        else if (add) launch_small<false, true>(m, a, st);
        else launch_small<false, false>(m, a, st);
        return hipGetLastError();
    }
    Fill fill = {};
    fill.row_pieces = 1;
    if (!add) {
        const bool flat = grad.ld == cols || rows == 1;
        fill.p = static_cast<char*>(grad.p);
        fill.row_bytes = flat ? rows * row_bytes : row_bytes;
        fill.pitch = flat ? 0 : grad.ld * unit;
        fill.row_pieces = parts_of(fill.row_bytes, 16);
        fill.end = (flat ? 1 : rows) * fill.row_pieces;
    }
    const GradWorkspace w(n, cols);
    char* p = static_cast<char*>(ws);
    uint64_t *keys = reinterpret_cast<uint64_t*>(p), *other = reinterpret_cast<uint64_t*>(p + w.keys);
    const bool ranked = tiles > 1 && n <= kRanked && fill.end * 16 >= tiles * kHides;
    const dim3 g = grid_of(tiles + parts_of(fill.end, kSortTile * kFillRounds), kSortTile), b(kSortTile);
    if (ranked) k_sort_tiles<true><<<g, b, 0, st>>>(ids, rows, keys, tiles, fill);
    else k_sort_tiles<false><<<g, b, 0, st>>>(ids, rows, keys, tiles, fill);
    if (n == 0) return hipGetLastError();
    a.long_begins = reinterpret_cast<uint32_t*>(p + 2 * w.keys);
    a.part = reinterpret_cast<float*>(p + 2 * w.keys + w.flags);
    for (int64_t run = kSortTile; run < n && !ranked; run *= kMergeRuns) {
        k_merge_runs<<<grid_of(parts_of(n, 64), 64 * kMergeRuns), dim3(64 * kMergeRuns), 0, st>>>(keys, other, n, run);
        uint64_t* t = keys;
        keys = other, other = t;
    }
    a.keys = keys, a.piece = piece_of(n, cols), a.pieces = parts_of(n, a.piece), a.part_ld = parts_of(cols, 8) * 8;
    if (bf && add) launch_sums<true, true>(a, st);
    else if (bf) launch_sums<true, false>(a, st);
    else if (add) launch_sums<false, true>(a, st);
    else launch_sums<false, false>(a, st);
    return hipGetLastError();
}

}  // namespace q4
