// The lookup of tokens' rows in a table, and its gradient.
//
//   lookup    out_i = f E[t_i]                         (0 for t_i < 0)
//   gradient  dE_v = dE0_v + f sum over t_i = v of dy_i
//
// Both move rows and compute next to nothing: HBM bounds them (a lookup of 16,384
// rows of 8 KB by frequent ids takes 32 us, 8.5 TB/s with what L2 gives again; the
// gradient of the same batch in a table of 131,072 rows 182 us, what its 1.2 GB
// take at a copy's rate).  The gradient reads dy once, in the order of the
// ids, which are sorted first, and writes every row of dE once: sums are held in
// float32 registers, in the tokens' order, so that no atomics are needed and the
// same inputs give the same bits.  Frequent ids would make one block add thousands
// of rows; so the sorted tokens are cut into chunks of 8 or 32 whatever their ids,
// and the partial sums of an id that crosses chunks are added by a third kernel.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "../../include/lct.h"
#include "codec_dev.cuh"
#include "internal.h"
#include "rows_dev.cuh"
#include "tensor_dev.cuh"

namespace lct {
namespace dev {

// -------------------------------------------- rows without tokens, sorted ids

// A row of a value, or of a base, in 16-byte pieces of the row between its ends,
// by `lanes` threads of which this is the lane-th.
__device__ __forceinline__ void fill_row(const FillArgs &f, int64_t r, int lane, int lanes)
{
    uint16_t *row = reinterpret_cast<uint16_t *>(static_cast<char *>(f.out) + r * f.ld_out);
    const uint16_t *base =
        f.base ? reinterpret_cast<const uint16_t *>(static_cast<const char *>(f.base) + r * f.ld_base) : nullptr;
    const int n = static_cast<int>((r == f.rows - 1 ? f.last : f.bytes) / 2);
    const uint16_t value = static_cast<uint16_t>(f.value);
    const int a = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 2), pieces = (n - a) / 8;
    for (int c = lane; c < a; c += lanes) row[c] = base ? base[c] : value;
    uint4 *q = reinterpret_cast<uint4 *>(row + a);
    if (base) {
        for (int c0 = lane; c0 < pieces; c0 += lanes * 4) {
            uint4 v[4];  // asked for together: nobody tells the compiler that the rows are apart
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + lanes * i < pieces) v[i] = load_any(base + a + 8 * (c0 + lanes * i), 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + lanes * i < pieces) q[c0 + lanes * i] = v[i];
        }
    } else {
        const uint4 v = make_uint4(f.value, f.value, f.value, f.value);
#pragma unroll 4
        for (int c = lane; c < pieces; c += lanes) q[c] = v;
    }
    for (int c = a + 8 * pieces + lane; c < n; c += lanes) row[c] = base ? base[c] : value;
}
// Threads of a row: a warp, or as many as a short row has pieces.
__device__ __forceinline__ int fill_lanes(const FillArgs &f)
{
    int lanes = 32;
    while (lanes > 1 && lanes * 16 >= 2 * f.bytes) lanes /= 2;
    return lanes;
}

// While the ids are being sorted, the other blocks of the same launch write what
// needs no order: the last rows, with or without tokens (those with tokens are
// replaced later), as many as that time allows.
__device__ __forceinline__ void fill(const FillArgs &f, int64_t block, int64_t blocks)
{
    const int lanes = fill_lanes(f), rows = blockDim.x / lanes;  // at a time
    for (int64_t r = f.rows - f.early + block * rows + threadIdx.x / lanes; r < f.rows; r += blocks * rows)
        fill_row(f, r, threadIdx.x % lanes, lanes);
}

// Ids outside 0 .. vocab - 1 become `vocab` and end up behind the others.
__device__ __forceinline__ int key_of(const SortArgs &g, int64_t i)
{
    const int64_t id = id_at(g.ids, g.wide, i);
    return id < 0 || id >= g.vocab ? g.vocab : static_cast<int>(id);
}

// Batches up to 8192 ids: an id's place is the number of smaller ones and of
// equal ones before it, and 67 million comparisons, IDS ids a block, are done
// before a cluster has met twice (8192 ids of a narrow table: 8 us, 18 by the sort).
constexpr int kRankThreads = 1024, kRankMost = 8192;
template <int IDS>
__global__ void __launch_bounds__(kRankThreads) k_rank_ids(const __grid_constant__ SortArgs g)
{
    constexpr int kParts = kRankThreads / IDS;  // of the ids that each of the block's is compared with
    extern __shared__ int4 keys4[];
    __shared__ int found[kParts][IDS];
    __shared__ int there;
    int *keys = reinterpret_cast<int *>(keys4);
    pdl_wait();
    pdl_launch_dependents();
    const int blocks = (g.tokens + IDS - 1) / IDS;
    if (static_cast<int>(blockIdx.x) >= blocks) {
        fill(g.fill, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    if (g.clear && blockIdx.x == 0 && threadIdx.x < 2) g.clear[threadIdx.x] = 0;
    if (threadIdx.x == 0) there = 0;
    constexpr int kRound = 4 * kParts;
    const int padded = (g.tokens + kRound - 1) / kRound * kRound;
    int valid = 0;
#pragma unroll 8
    for (int j = threadIdx.x; j < padded; j += kRankThreads) {
        const int key = j < g.tokens ? key_of(g, j) : INT32_MAX;
        keys[j] = key;
        valid += key < g.vocab;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        valid = __reduce_add_sync(kFull, valid);
        if ((threadIdx.x & 31) == 0) atomicAdd(&there, valid);
    }
    const int mine = threadIdx.x % IDS, part = threadIdx.x / IDS;
    const int i0 = blockIdx.x * IDS, i = i0 + mine;
    const int key = i < g.tokens ? keys[i] : 0;
    // a part of the ids: those before the block's, those among them, those behind
    const int share = padded / kParts, lo = part * share, hi = lo + share;
    auto smaller = [&](int from, int to, int than) {
        int n = 0;
#pragma unroll 4
        for (int j = from; j < to; j += 4) {
            const int4 k = keys4[j / 4];
            n += (k.x < than) + (k.y < than) + (k.z < than) + (k.w < than);
        }
        return n;
    };
    int n = smaller(lo, min(hi, i0), key + 1) + smaller(max(lo, i0 + IDS), hi, key);
    for (int j = max(lo, i0); j < min(hi, i0 + IDS); ++j) n += keys[j] < key + (j < i);
    found[part][mine] = n;
    __syncthreads();
    if (part == 0 && i < g.tokens) {
        int place = n;
#pragma unroll
        for (int p = 1; p < kParts; ++p) place += found[p][mine];
        g.key[0][place] = key;
        g.order[0][place] = i;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *g.count = there;
}

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortBlocks = 8;

// Longer batches: stable radix sort by one cluster, least digit first, a warp
// counting and placing 32 consecutive ids at a time.
__global__ void __launch_bounds__(kSortThreads) k_sort_ids(const __grid_constant__ SortArgs g)
{
    extern __shared__ uint32_t counts[];  // [warps][digits], then the block's totals [digits]
    __shared__ uint32_t part[kSortWarps];
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int digits = 1 << g.bits;
    uint32_t *total = counts + kSortWarps * digits;
    uint32_t *mine = counts + warp * digits;
    const int share = (g.tokens + static_cast<int>(size) * kSortThreads - 1) / (static_cast<int>(size) * kSortThreads) * 32;
    const int64_t lo = static_cast<int64_t>(rank * kSortWarps + warp) * share;
    const int64_t hi = min(lo + share, static_cast<int64_t>(g.tokens));
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= size) {
        fill(g.fill, blockIdx.x - size, gridDim.x - size);
        return;
    }
    if (g.clear && rank == 0 && threadIdx.x < 2) g.clear[threadIdx.x] = 0;
    for (int pass = 0; pass < g.passes; ++pass) {
        const int to = (g.passes - 1 - pass) & 1, shift = pass * g.bits;
        auto key_at = [&](int64_t i) -> int {
            if (i >= hi) return -1;
            if (pass) return __ldcg(&g.key[to ^ 1][i]);
            return key_of(g, i);
        };
        for (int d = lane; d < digits; d += 32) mine[d] = 0;
        __syncwarp();
        for (int64_t i = lo + lane; i - lane < hi; i += 32) {
            const int key = key_at(i);
            const int d = key < 0 ? -1 : key >> shift & (digits - 1);
            const uint32_t same = __match_any_sync(kFull, d);
            if (d >= 0 && lane == __ffs(same) - 1) mine[d] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // each warp's place within the block's ids of a digit
        for (int d = threadIdx.x; d < digits; d += kSortThreads) {
            uint32_t sum = 0;
#pragma unroll 1
            for (int w0 = 0; w0 < kSortWarps; w0 += 16) {
                uint32_t c[16];
#pragma unroll
                for (int w = 0; w < 16; ++w) c[w] = counts[(w0 + w) * digits + d];
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    counts[(w0 + w) * digits + d] = sum;
                    sum += c[w];
                }
            }
            total[d] = sum;
        }
        cluster_sync();
        // where the block's ids of a digit go: behind all smaller digits, and this digit's of earlier blocks
        uint32_t before = 0, all = 0;
        if (static_cast<int>(threadIdx.x) < digits)
            for (uint32_t r = 0; r < size; ++r) {
                const uint32_t c = ld_peer_shared(&total[threadIdx.x], r);
                if (r < rank) before += c;
                all += c;
            }
        uint32_t sum = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) part[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += part[w];
        cluster_sync();  // the totals have been read, and take the places
        if (static_cast<int>(threadIdx.x) < digits) total[threadIdx.x] = before + sum - all;
        __syncthreads();
        for (int64_t i = lo + lane; i - lane < hi; i += 32) {
            const int key = key_at(i);
            const int token = pass && i < hi ? __ldcg(&g.order[to ^ 1][i]) : static_cast<int>(i);
            const int d = key < 0 ? -1 : key >> shift & (digits - 1);
            const uint32_t same = __match_any_sync(kFull, d);
            uint32_t at = 0;
            if (d >= 0) at = mine[d];
            __syncwarp();
            if (d >= 0) {
                const uint32_t place = total[d] + at + __popc(same & ((1u << lane) - 1));
                g.key[to][place] = key;
                g.order[to][place] = token;
                if (lane == __ffs(same) - 1) mine[d] = at + __popc(same);
            }
            __syncwarp();
        }
        cluster_sync();
    }
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const int key = __ldcg(&g.key[0][i]), last = i ? __ldcg(&g.key[0][i - 1]) : -1;
        if (key != last && key >= g.vocab) *g.count = static_cast<int>(i);
        if (i == g.tokens - 1 && key < g.vocab) *g.count = g.tokens;
    }
}

// ------------------------------------------------------------------ lookup

// ROWS rows a block at a time: their ids are one trip to memory, the rows
// themselves the next, and all are asked for before the first is written.
template <typename T, bool AL, int ROWS>
__global__ void __launch_bounds__(kRowThreads) k_embedding(const __grid_constant__ LookupArgs g)
{
    const int piece = piece_of<T>(blockIdx.y);
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * ROWS;
    Piece<T, AL> p[ROWS];
    int64_t id[ROWS];
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) id[r] = i0 + r < g.tokens ? id_at(g.ids, g.wide, i0 + r) : -1;
    // whole pieces of rows that are all there: no branch between their reads
    bool inside = !AL;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int c = piece - skip_of_row<T, AL>(static_cast<T *>(g.out) + (i0 + r) * g.ld_out);
        inside = inside && id[r] >= g.row0 && id[r] < g.row0 + g.rows && c >= 0 && c + kVec<T> <= g.cols;
    }
    if (inside) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int c = piece - skip_of_row<T, AL>(static_cast<T *>(g.out) + (i0 + r) * g.ld_out);
            p[r].q = load_any(static_cast<const T *>(g.table) + (id[r] - g.row0) * g.ld_table + c, 16);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t at = id[r] - g.row0;
        if (inside) continue;
        if (at >= 0 && at < g.rows) {
            const int c = piece - skip_of_row<T, AL>(static_cast<T *>(g.out) + (i0 + r) * g.ld_out);
            p[r].load(static_cast<const T *>(g.table) + at * g.ld_table, c, g.cols);
        } else {
            const T fill = from_float<T>(id[r] < 0 ? 0.0f : __int_as_float(0x7FC00000));
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) p[r].v[e] = fill;
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t at = id[r] - g.row0;
        const bool there = at >= 0 && at < g.rows;
        if (i0 + r >= g.tokens || (!there && id[r] >= 0 && id[r] < g.vocab)) continue;  // another piece's row
        if (there && g.scale != 1.0f) {
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) p[r].v[e] = from_float<T>(to_float(p[r].v[e]) * g.scale);
        }
        T *row = static_cast<T *>(g.out) + (i0 + r) * g.ld_out;
        p[r].store(row, piece - skip_of_row<T, AL>(row), g.cols);
    }
}

// ---------------------------------------------------------------- gradient

constexpr int kSegTokens = 32;  // of a chunk, at most
// Rows asked for at a time.  Eight of them, with their bases, leave so few blocks
// on an SM that the rows without tokens, which the same launch writes, take 10% longer.
constexpr int kSegAhead = 4;

// The row that key's sum goes to, and the column of it at which this thread's piece begins.
template <typename T, bool AL>
__device__ __forceinline__ int first_col(const SegmentArgs &g, int key, int piece)
{
    return g.compact ? piece : piece - skip_of_row<T, AL>(static_cast<T *>(g.out) + key * g.ld_out);
}

// A finished row: scaled, added to its base, rounded once.  Compact sums
// (float32, unscaled) go to the row of the id's first token instead.
template <typename T, bool AL>
__device__ __forceinline__ void finish_row(const SegmentArgs &g, int key, int first, int piece, const float (&acc)[kVec<T>],
                                           const Piece<T, AL> &base)
{
    if (g.compact) {
        if (piece < g.cols) store_floats<T>(acc, static_cast<float *>(g.out) + first * g.ld_out, piece);
        if (piece == 0) g.first[key] = first;
        return;
    }
    Piece<T, AL> p;
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
        p.v[e] = from_float<T>(g.base ? fmaf(g.scale, acc[e], to_float(base.v[e])) : g.scale * acc[e]);
    p.store(static_cast<T *>(g.out) + key * g.ld_out, first_col<T, AL>(g, key, piece), g.cols);
}

// Partial sums of an id that crosses chunks, [chunk][2][pieces' values]: of one that began
// earlier (0), of one that begins here and goes on (1).
__device__ __forceinline__ float *partial(const SegmentArgs &g, int64_t chunk, int which)
{
    return g.part + (chunk * 2 + which) * LCT_EMBEDDING_PART(g.cols);
}

// The first of the sorted ids that is not smaller than v, by a warp: 32 of them
// are looked at in one trip to memory.
__device__ __forceinline__ int64_t lower_bound(const int32_t *key, int64_t count, int v)
{
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = count;  // the place is lo .. lo + n
    while (n > 0) {
        const int64_t step = (n + 31) / 32, at = lo + step * lane;
        const bool smaller = at < lo + n && key[at] < v;
        const int below = __popc(__ballot_sync(kFull, smaller));
        if (below == 0) return lo;
        const int64_t next = lo + step * (below - 1) + 1;
        n = min(step - 1, lo + n - next);
        lo = next;
    }
    return lo;
}

// Rows without tokens, of the block's (at most kFillRows).
constexpr int kFillRows = 4096;
__device__ __forceinline__ void fill_rest(const SegmentArgs &g, int64_t block)
{
    __shared__ uint32_t have[kFillRows / 32];
    __shared__ int64_t ends[2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, warps = blockDim.x / 32;
    const int64_t r0 = block * g.fill_rows, r1 = min(r0 + g.fill_rows, g.fill.rows - g.fill.early), count = *g.count;
    for (int i = threadIdx.x; i < kFillRows / 32; i += blockDim.x) have[i] = 0;
    for (int i = warp; i < 2; i += warps) {
        const int64_t at = lower_bound(g.key, count, static_cast<int>(i ? r1 : r0));
        if (lane == 0) ends[i] = at;
    }
    __syncthreads();
    for (int64_t i = ends[0] + threadIdx.x; i < ends[1]; i += blockDim.x) {
        const int r = g.key[i] - static_cast<int>(r0);
        atomicOr(&have[r / 32], 1u << (r & 31));
    }
    __syncthreads();
    const int lanes = fill_lanes(g.fill), rows = blockDim.x / lanes;
    for (int64_t r = r0 + threadIdx.x / lanes; r < r1; r += rows) {
        const int at = static_cast<int>(r - r0);
        if (!(have[at / 32] >> (at & 31) & 1)) fill_row(g.fill, r, threadIdx.x % lanes, lanes);
    }
}

// A chunk of sorted tokens and a slab of columns a block; rows without tokens by the blocks behind them.
template <typename T, bool AL, bool BASE>
__global__ void __launch_bounds__(kRowThreads, 4) k_segments(const __grid_constant__ SegmentArgs g)
{
    __shared__ int keys[kSegTokens], tokens[kSegTokens];
    __shared__ float coefs[kSegTokens];
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t blocks = g.chunks * g.slabs;
    if (blockIdx.x >= blocks) {
        fill_rest(g, blockIdx.x - blocks);
        return;
    }
    const int64_t chunk = blockIdx.x / g.slabs;
    const int piece = piece_of<T>(blockIdx.x % g.slabs);
    const bool used = piece < g.cols + (AL ? 0 : kVec<T> - 1);
    const int64_t i0 = chunk * g.chunk;
    const int64_t count = *g.count;
    for (int j = threadIdx.x; j < g.chunk && i0 + j < g.tokens; j += blockDim.x) {
        keys[j] = g.key[i0 + j];
        tokens[j] = g.order ? g.order[i0 + j] : static_cast<int>(i0 + j);
        coefs[j] = g.coef && i0 + j < count ? g.coef[i0 + j] : 1.0f;
    }
    const int before = i0 > 0 ? g.key[i0 - 1] : -1, behind = i0 + g.chunk < g.tokens ? g.key[i0 + g.chunk] : -1;
    __syncthreads();
    const int n = static_cast<int>(min(static_cast<int64_t>(g.chunk), count - i0));
    if (n <= 0) return;
    const bool goes_on = i0 + n < count && behind == keys[n - 1];
    int64_t began = before == keys[0] ? -1 : i0;  // where the id's tokens begin (-1: in an earlier chunk)
    float acc[kVec<T>];
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) acc[e] = 0.0f;
    constexpr int kAhead = AL ? kSegAhead : kSegAhead / 2;  // others take two reads
    for (int j0 = 0; j0 < n; j0 += kAhead) {
        Piece<T, AL> p[kAhead], base[BASE ? kAhead : 1];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int at = j0 + j;
            if (at >= n) continue;
            const int c = first_col<T, AL>(g, keys[at], piece);
            p[j].load(static_cast<const T *>(g.src) + tokens[at] * g.ld_src, c, g.cols);
            // an id's last row: its base is wanted as well
            if (BASE && (at + 1 == n || keys[at + 1] != keys[at]))
                base[j].load(static_cast<const T *>(g.base) + keys[at] * g.ld_base, c, g.cols);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int at = j0 + j;
            if (at >= n) break;
            const float f = coefs[at];
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) acc[e] = fmaf(f, to_float(p[j].v[e]), acc[e]);
            if (at + 1 < n && keys[at + 1] == keys[at]) continue;
            if (began < 0 || (at == n - 1 && goes_on)) {
                if (used) store_floats<T>(acc, partial(g, chunk, began < 0 ? 0 : 1), piece);
                // where it began, for the kernel that adds the parts
                if (g.compact && began >= 0 && piece == 0) g.first[keys[at]] = static_cast<int>(began);
            } else {
                finish_row<T, AL>(g, keys[at], static_cast<int>(began), piece, acc, base[BASE ? j : 0]);
            }
            began = i0 + at + 1;
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) acc[e] = 0.0f;
        }
    }
}

// Ids that cross chunks: the block of the chunk where one begins adds its parts.
template <typename T, bool AL>
__global__ void __launch_bounds__(kRowThreads) k_segment_ends(const __grid_constant__ SegmentArgs g)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t chunk = blockIdx.x / g.slabs, i0 = chunk * g.chunk, next = i0 + g.chunk;
    const int piece = piece_of<T>(blockIdx.x % g.slabs), lane = threadIdx.x & 31;
    // (there is a chunk behind this one, so that all of these are ids; those behind the last are no row's)
    const int64_t count = *g.count;
    const int key = g.key[next - 1], begins = g.key[i0], before = i0 ? g.key[i0 - 1] : -1, goes_on = g.key[next];
    if (next >= count || goes_on != key || (begins == key && before == key)) return;
    // the chunks that the id goes on in
    int64_t more = 0;
    for (;; more += 32) {
        const int64_t at = next + (more + lane) * g.chunk;
        const uint32_t same = __ballot_sync(kFull, at < count && g.key[at] == key);
        if (same != kFull) {
            more += __ffs(~same) - 1;
            break;
        }
    }
    float acc[kVec<T>];
    if (piece >= g.cols + (AL ? 0 : kVec<T> - 1)) return;
    load_floats<T>(acc, partial(g, chunk, 1), piece);
    Piece<T, AL> base;
    if (g.base) base.load(static_cast<const T *>(g.base) + key * g.ld_base, first_col<T, AL>(g, key, piece), g.cols);
    constexpr int kParts = 64 / kVec<T>;  // at a time
    for (int64_t c0 = 1; c0 <= more; c0 += kParts) {
        float v[kParts][kVec<T>];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            if (c0 + i <= more) load_floats<T>(v[i], partial(g, chunk + c0 + i, 0), piece);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (c0 + i > more) break;
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) acc[e] += v[i][e];
        }
    }
    const int first = g.compact ? g.first[key] : 0;
    finish_row<T, AL>(g, key, first, piece, acc, base);
}

}  // namespace dev

// ------------------------------------------------------------------ launches

// Fill blocks of `bytes_each` at a time, at most `most`.
static uint32_t fill_blocks(const FillArgs &f, uint64_t bytes_each, uint64_t most)
{
    if (!f.out || !f.early) return 0;
    const uint64_t bytes = static_cast<uint64_t>(f.early) * static_cast<uint64_t>(f.bytes);
    return static_cast<uint32_t>(std::min(most, (bytes + bytes_each - 1) / bytes_each));
}

cudaError_t launch_sort_ids(SortArgs g, cudaStream_t s)
{
    const uint32_t tokens = static_cast<uint32_t>(g.tokens);
    if (tokens <= dev::kRankMost) {
        // as few ids a block as there are SMs for
        const uint32_t ids = tokens <= 152 * 32 ? 32 : 64;
        const uint32_t blocks = (tokens + ids - 1) / ids + fill_blocks(g.fill, 131072, 152 * 2);
        const uint32_t smem = (tokens + 127) / 128 * 512;
        if (!blocks) return cudaSuccess;
        return ids == 32 ? launch<true>(dev::k_rank_ids<32>, dim3(blocks), dev::kRankThreads, smem, 1, s, g)
                         : launch<true>(dev::k_rank_ids<64>, dim3(blocks), dev::kRankThreads, smem, 1, s, g);
    }
    int need = 1;
    while (need < 31 && g.vocab >> need) ++need;  // bits of `vocab`, the largest key
    g.passes = (need + 8) / 9;
    g.bits = (need + g.passes - 1) / g.passes;
    const uint32_t smem = (dev::kSortWarps + 1) * (4u << g.bits);
    const uint32_t fills = fill_blocks(g.fill, 262144, 152 * 2 - dev::kSortBlocks);
    return launch<true>(dev::k_sort_ids, dim3((fills + dev::kSortBlocks - 1) / dev::kSortBlocks * dev::kSortBlocks + dev::kSortBlocks),
                        dev::kSortThreads, smem, dev::kSortBlocks, s, g);
}

namespace {

template <typename T, bool AL>
cudaError_t lookup(const LookupArgs &g, cudaStream_t s)
{
    uint32_t threads, slabs;
    row_shape(g.cols, dev::kVec<T>, AL, &threads, &slabs);
    if (g.tokens * static_cast<uint64_t>(slabs) <= 152 * 8)
        return launch<true>(dev::k_embedding<T, AL, 1>, dim3(static_cast<uint32_t>(g.tokens), slabs), threads, 0, 1, s, g);
    return launch<true>(dev::k_embedding<T, AL, 4>, dim3(static_cast<uint32_t>((g.tokens + 3) / 4), slabs), threads, 0, 1, s,
                        g);
}

template <typename T, bool AL>
cudaError_t segments(SegmentArgs g, cudaStream_t s)
{
    uint32_t threads;
    row_shape(g.cols, dev::kVec<T>, AL, &threads, &g.slabs);
    g.chunk = static_cast<int32_t>(LCT_EMBEDDING_CHUNK(static_cast<uint64_t>(g.tokens)));
    g.chunks = (static_cast<uint32_t>(g.tokens) + g.chunk - 1) / g.chunk;
    uint64_t fills = 0;
    const uint32_t row_threads = threads;
    const int64_t rest = g.fill.out ? g.fill.rows - g.fill.early : 0;
    if (rest) {
        // The blocks that fill have the threads of the others, 256 bytes each: at least four warps, as short rows' single
        // one with 64 KB takes 37 us for 131,072 rows of 128 bytes (12), 240 us for a million of 512 (134).  Eight
        // warps are no faster where tokens are few and leave less room for sums where they are many (20,000 in a million rows
        // of 126 bytes: 89 us, with four 84).
        threads = std::max<uint32_t>(threads, 128);
        g.fill_rows = static_cast<int32_t>(std::min<int64_t>(
            dev::kFillRows, std::max<int64_t>(threads / 32, 256 * static_cast<int64_t>(threads) / g.fill.bytes)));
        fills = (static_cast<uint64_t>(rest) + g.fill_rows - 1) / g.fill_rows;
    }
    if (!g.chunks && !fills) return cudaSuccess;
    const dim3 grid(static_cast<uint32_t>(g.chunks * g.slabs + fills));
    cudaError_t rc = g.base ? launch<true>(dev::k_segments<T, AL, true>, grid, threads, 0, 1, s, g)
                            : launch<true>(dev::k_segments<T, AL, false>, grid, threads, 0, 1, s, g);
    if (rc == cudaSuccess && g.chunks > 1)
        rc = launch<true>(dev::k_segment_ends<T, AL>, dim3((g.chunks - 1) * g.slabs), row_threads, 0, 1, s, g);
    return rc;
}

}  // namespace

cudaError_t launch_segments(const SegmentArgs &g, bool wide, bool aligned, cudaStream_t s)
{
    if (wide) return aligned ? segments<float, true>(g, s) : segments<float, false>(g, s);
    return aligned ? segments<__nv_bfloat16, true>(g, s) : segments<__nv_bfloat16, false>(g, s);
}

cudaError_t launch_lookup(const LookupArgs &g, bool wide, bool aligned, cudaStream_t s)
{
    if (wide) return aligned ? lookup<float, true>(g, s) : lookup<float, false>(g, s);
    return aligned ? lookup<__nv_bfloat16, true>(g, s) : lookup<__nv_bfloat16, false>(g, s);
}

lct_status check_ids(const lct_ids *ids)
{
    if (!ids || ids->vocab == 0) return LCT_ERR_INVALID_ARG;
    if (ids->tokens > LCT_VOCAB_MAX_TOKENS || ids->vocab > LCT_VOCAB_MAX) return LCT_ERR_UNSUPPORTED;
    if (ids->wide != 0 && ids->wide != 1) return LCT_ERR_INVALID_ARG;
    const uintptr_t at = reinterpret_cast<uintptr_t>(ids->d_ids);
    if (ids->tokens && (!at || at % (ids->wide ? 8 : 4))) return LCT_ERR_INVALID_ARG;
    return LCT_OK;
}

namespace {

// Bytes of rows that are written while ids are sorted, by the two ways of that (about 8 and 20 us).  Long batches: none
// makes 16,384 tokens of 8 KB 195 us, 160 MB 184, this 182.  Short ones: a table that is written whole here needs no more
// blocks (5000 tokens, 10,007 rows of 32 bytes: 20 us, none: 24); of larger ones it changes 1 to 2 us, either way.
constexpr int64_t kFillShort = 12 << 20, kFillLong = 100 << 20;

uint64_t value_bytes(int32_t dtype) { return dtype == LCT_DTYPE_F32 ? 4 : 2; }

}  // namespace
}  // namespace lct

using namespace lct;

extern "C" lct_status lct_embedding(const lct_ids *ids, const void *d_table, uint64_t ld_table, int32_t dtype,
                                    uint64_t first, uint64_t rows, uint64_t cols, float scale, void *d_out,
                                    uint64_t ld_out, void *stream)
{
    const lct_status rc = check_ids(ids);
    if (rc != LCT_OK) return rc;
    if (dtype != LCT_DTYPE_BF16 && dtype != LCT_DTYPE_F32) return LCT_ERR_UNSUPPORTED;
    if (cols == 0 || first > ids->vocab || rows > ids->vocab - first) return LCT_ERR_INVALID_ARG;
    if (cols > LCT_VOCAB_MAX_COLS) return LCT_ERR_UNSUPPORTED;
    if (ids->tokens == 0) return LCT_OK;
    const uint64_t size = value_bytes(dtype);
    const Matrix table{d_table, ld_table, cols, rows, size}, out{d_out, ld_out, cols, ids->tokens, size};
    if (!matrix_ok(table) || !matrix_ok(out)) return LCT_ERR_INVALID_ARG;
    if (!apart(out, table) || !apart(out, ids->d_ids, ids->tokens * (ids->wide ? 8 : 4))) return LCT_ERR_INVALID_ARG;
    LookupArgs g;
    g.ids = ids->d_ids;
    g.wide = ids->wide;
    g.table = d_table;
    g.out = d_out;
    g.ld_table = static_cast<int64_t>(ld_table);
    g.ld_out = static_cast<int64_t>(ld_out);
    g.row0 = static_cast<int64_t>(first);
    g.rows = static_cast<int64_t>(rows);
    g.vocab = static_cast<int64_t>(ids->vocab);
    g.tokens = static_cast<int64_t>(ids->tokens);
    g.cols = static_cast<int32_t>(cols);
    g.scale = scale;
    return launch_lookup(g, dtype == LCT_DTYPE_F32, matrix_al(table) && matrix_al(out) && cols * size % 16 == 0,
                         static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LCT_OK
               : LCT_ERR_CUDA;
}

extern "C" lct_status lct_embedding_grad(const lct_ids *ids, const void *d_dy, uint64_t ld_dy, int32_t dtype,
                                         uint64_t cols, float scale, const void *d_base, uint64_t ld_base, void *d_out,
                                         uint64_t ld_out, void *d_work, void *stream)
{
    const lct_status rc = check_ids(ids);
    if (rc != LCT_OK) return rc;
    if (dtype != LCT_DTYPE_BF16 && dtype != LCT_DTYPE_F32) return LCT_ERR_UNSUPPORTED;
    if (cols == 0) return LCT_ERR_INVALID_ARG;
    if (cols > LCT_VOCAB_MAX_COLS) return LCT_ERR_UNSUPPORTED;
    const uint64_t size = value_bytes(dtype), t = ids->tokens;
    const Matrix dy{d_dy, ld_dy, cols, t, size}, out{d_out, ld_out, cols, ids->vocab, size};
    const Matrix base{d_base, ld_base, cols, d_base ? ids->vocab : 0, size};
    const uint64_t work = LCT_EMBEDDING_WORK_BYTES(t, cols), id_bytes = t * (ids->wide ? 8 : 4);
    const bool in_place = d_base == d_out && ld_base == ld_out;
    if (!matrix_ok(dy) || !matrix_ok(out) || !matrix_ok(base)) return LCT_ERR_INVALID_ARG;
    if (!d_work || reinterpret_cast<uintptr_t>(d_work) % 16) return LCT_ERR_INVALID_ARG;
    if (!apart(out, dy) || (!in_place && !apart(out, base)) || !apart(out, ids->d_ids, id_bytes) ||
        !apart(out, d_work, work) || !apart(dy, d_work, work) || !apart(base, d_work, work) ||
        !apart(d_work, work, ids->d_ids, id_bytes))
        return LCT_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint64_t t4 = (t + 3) / 4 * 4;
    int32_t *w = static_cast<int32_t *>(d_work);
    SortArgs sort{};
    sort.ids = ids->d_ids;
    sort.wide = ids->wide;
    sort.count = w;
    sort.key[0] = w + 4;
    sort.key[1] = sort.key[0] + t4;
    sort.order[0] = sort.key[1] + t4;
    sort.order[1] = sort.order[0] + t4;
    sort.tokens = static_cast<int32_t>(t);
    sort.vocab = static_cast<int32_t>(ids->vocab);
    if (!in_place) {
        FillArgs &f = sort.fill;
        f.out = d_out;
        f.base = d_base;
        f.rows = static_cast<int64_t>(ids->vocab);
        f.bytes = f.last = static_cast<int64_t>(cols * size);
        f.ld_out = static_cast<int64_t>(ld_out * size);
        f.ld_base = static_cast<int64_t>(ld_base * size);
        // what the time of the sort is enough for
        f.early = t ? std::min<int64_t>(f.rows, (t <= dev::kRankMost ? kFillShort : kFillLong) / f.bytes) : f.rows;
    }
    if (launch_sort_ids(sort, s) != cudaSuccess) return LCT_ERR_CUDA;
    if (t == 0) return LCT_OK;  // every row has been written
    SegmentArgs g{};
    g.src = d_dy;
    g.ld_src = static_cast<int64_t>(ld_dy);
    g.key = sort.key[0];
    g.order = sort.order[0];
    g.count = sort.count;
    g.scale = scale;
    g.base = d_base;
    g.ld_base = static_cast<int64_t>(ld_base);
    g.out = d_out;
    g.ld_out = static_cast<int64_t>(ld_out);
    g.part = reinterpret_cast<float *>(sort.order[1] + t4);
    g.fill = sort.fill;
    g.cols = static_cast<int32_t>(cols);
    g.tokens = static_cast<int32_t>(t);
    const bool aligned = cols * size % 16 == 0 && matrix_al(out) && matrix_al(dy) && matrix_al(base);
    return launch_segments(g, dtype == LCT_DTYPE_F32, aligned, s) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
}
