// Low-rank adapters of many requests beside a shared projection, for training
// and serving.  For a token of adapter a, with A_a [R, K], B_a [N, R], s_a:
//
//   forward   out = y + s_a (x A_a^T) B_a^T
//   backward  d = s_a dy B_a,  dx' = dx + d A_a,
//             dA_a = sum d^T x,  dB_a = sum s_a dy^T (x A_a^T)
//
// Both directions of the tokens' part are one kernel (k_adapter): a product
// with a narrow matrix (In W1, R columns), whose result stays on the SM, and a
// product back to the full width added to a row that is there already.  The
// arithmetic is 4R operations a value of x or y, which HBM delivers in 2 to 4
// bytes: up to R = 64 HBM bounds the work, if the tensor cores take the
// products as they come (tcgen05, accumulators in TMEM).
//
// Rounding: the products take the BF16 inputs as they are and add in float32;
// the narrow result V is carried to the second product as the sum of two BF16
// (hi + lo, 16 bits of V), so only the final value is rounded to BF16.
#include <algorithm>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>

#include "../../include/lct.h"
#include "../../include/lct_debug.h"
#include "codec_dev.cuh"
#include "internal.h"
#include "tensor_dev.cuh"

namespace lct {

// Boxes of the matrices that the kernels read.
struct TokenMaps {
    CUtensorMap in, base, a, b;
};
struct GradMaps {
    CUtensorMap x, dy, d, v;
};

namespace dev {

constexpr int kAdThreads = 256;
constexpr int kTileTokens = LCT_ADAPTER_TILE;
constexpr int kChunk = 64;                        // columns of In (phase 1) or of the result (phase 2) at a time
constexpr int kInBytes = kTileTokens * 128;       // a tile of 128 tokens by 64 BF16 columns

// ------------------------------------------------------------ tile loads

__device__ __forceinline__ void async16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight BF16 values at any address, of which `valid` are there (the rest zero),
// in two steps, so that many are fetched before the first is waited for.  Six of
// them lie in three aligned words, from the first value on that begins one; the
// other two are read alone.
struct Eight {
    uint32_t a, b, c, h, t;
    bool odd, part;
};
__device__ __forceinline__ Eight fetch8(const __nv_bfloat16 *src, int valid)
{
    const uint16_t *p = reinterpret_cast<const uint16_t *>(src);
    Eight e = {0, 0, 0, 0, 0, (reinterpret_cast<uintptr_t>(p) & 2) != 0, valid < 8};
    if (valid >= 8) {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p + e.odd);
        e.a = q[0], e.b = q[1], e.c = q[2];
        e.h = p[e.odd ? 0 : 6], e.t = p[7];
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < valid) w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        e.a = w[0], e.b = w[1], e.c = w[2], e.h = w[3];
    }
    return e;
}
__device__ __forceinline__ uint4 join8(const Eight &e)
{
    if (e.part) return make_uint4(e.a, e.b, e.c, e.h);
    if (!e.odd) return make_uint4(e.a, e.b, e.c, e.h | e.t << 16);
    return make_uint4(e.h | e.a << 16, __funnelshift_r(e.a, e.b, 16), __funnelshift_r(e.b, e.c, 16),
                      e.c >> 16 | e.t << 16);
}

// The same into a 16-byte piece of shared memory: asynchronously where the
// address allows it.
template <bool FAST>
__device__ __forceinline__ void piece(uint32_t dst, const __nv_bfloat16 *src, int valid, bool aligned)
{
    if (FAST || aligned) {
        async16(dst, src, valid <= 0 ? 0u : static_cast<uint32_t>(min(valid, 8)) * 2);
    } else {
        store16(dst, join8(fetch8(src, valid)));
    }
}

// Rows at any address.  PIECES 16-byte pieces of a row are copied from the
// aligned address at or below its first value (the piece that holds that value
// lies in the tensor's allocation with all of its bytes), asynchronously like
// aligned ones, and moved down by the row's `skip` values when they are there.
// The last piece may need a part of one more, which goes to `extra`.  This is
// one piece's copy, from its aligned address; `valid` of the row's values are
// there, the rest is zero.
__device__ __forceinline__ uint32_t skip_of(const __nv_bfloat16 *row)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) >> 1) & 7;
}
template <int PIECES>
__device__ __forceinline__ void raw_piece(uint32_t dst, uint32_t extra, const __nv_bfloat16 *from, uint32_t skip,
                                          int piece, int valid)
{
    const int left = valid <= 0 ? 0 : min(valid, 8 * PIECES) + static_cast<int>(skip) - 8 * piece;
    async16(dst, from, 2 * max(0, min(left, 8)));
    if (piece == PIECES - 1 && skip) async16(extra, from + 8, 2 * max(0, left - 8));
}
// The eight values from the skip-th on of two pieces.
__device__ __forceinline__ uint4 move_down(const uint4 &x, const uint4 &y, uint32_t skip)
{
    const bool four = skip & 4, two = skip & 2;
    const uint32_t a0 = four ? x.z : x.x, a1 = four ? x.w : x.y, a2 = four ? y.x : x.z, a3 = four ? y.y : x.w,
                   a4 = four ? y.z : y.x, a5 = four ? y.w : y.y;
    const uint32_t b0 = two ? a1 : a0, b1 = two ? a2 : a1, b2 = two ? a3 : a2, b3 = two ? a4 : a3, b4 = two ? a5 : a4;
    const uint32_t odd = (skip & 1) * 16;
    return make_uint4(__funnelshift_r(b0, b1, odd), __funnelshift_r(b1, b2, odd), __funnelshift_r(b2, b3, odd),
                      __funnelshift_r(b3, b4, odd));
}

// What rounding v to the BF16 whose bits (as float32) are `kept` left out; an
// infinite or NaN value has no remainder.
__device__ __forceinline__ float rest(float v, uint32_t kept)
{
    const float h = __uint_as_float(kept);
    return isfinite(h) ? v - h : 0.0f;
}

// Eight float32 as hi + lo, each eight BF16.
__device__ __forceinline__ void split8(const float (&v)[8], uint4 &hi, uint4 &lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = pack2(v[2 * i], v[2 * i + 1]);
        l[i] = pack2(rest(v[2 * i], h[i] << 16), rest(v[2 * i + 1], h[i] & 0xFFFF0000u));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ float4 peer_float4(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void peer_store16(uint32_t at, uint4 v)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
// The two halves of a meeting of the cluster.
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float peer_float(uint32_t at)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// The rank an adapter uses, within the bank's.
__device__ __forceinline__ int used_rank(const AdapterArgs &g, int a)
{
    const int r = g.ranks ? g.ranks[a] : g.rank;
    return max(0, min(r, g.rank));
}

// Latches an error in the plan.
__device__ __forceinline__ void fail(const AdapterArgs &g, int code)
{
    atomicCAS(reinterpret_cast<unsigned int *>(g.status), 0u, static_cast<unsigned int>(code));
}

// Place i of the order (i < tokens), and a row of the tile table: one that is
// not a plan's reaches nothing out of bounds.
__device__ __forceinline__ int checked_token(const AdapterArgs &g, int t)
{
    if (static_cast<uint32_t>(t) < static_cast<uint32_t>(g.tokens)) return t;
    fail(g, LCT_ERR_CORRUPT);
    return 0;
}
__device__ __forceinline__ int token_at(const AdapterArgs &g, int i) { return checked_token(g, g.order[i]); }
__device__ __forceinline__ int4 tile_at(const AdapterArgs &g, int i)
{
    int4 t = reinterpret_cast<const int4 *>(g.tiles)[i];
    if (t.z <= 0) {
        t.z = 0;
    } else if (t.z > kTileTokens || t.y < 0 || t.y > g.tokens - t.z) {
        fail(g, LCT_ERR_CORRUPT);
        t.z = 0;
    }
    return t;
}

// A meeting of the cluster's eight result warps: each warp arrives at every
// block's barrier, and waits at its own.
__device__ __forceinline__ void arrive_cluster(uint64_t *bar, uint32_t size, int lane, const Waiter &waiter)
{
    __syncwarp();
    if (lane < static_cast<int>(size) && !waiter.dead) {
        const uint32_t there = peer_addr(smem_addr(bar), lane);
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(there) : "memory");
    }
}
// Four result warps that share chunks.
__device__ __forceinline__ void set_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(2 + half)); }

// The result warps alone.
__device__ __forceinline__ void out_warps_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Warps by what they do: eight turn sums into results, one issues the
// products, one loads boxes (TMA) and eight load what no box holds.  They meet
// at mbarriers only, so that a load never waits for a result to be written.
constexpr int kOutWarps = 8, kMmaWarp = 8, kBoxWarp = 9, kLoadWarp = 10, kLoadWarps = 8;
constexpr int kLoadGroup = 4;  // warps that load one chunk; the groups take chunks in turn
constexpr int kTokThreads = 32 * (kLoadWarp + kLoadWarps);

// A load warp's share of a chunk is there: when its asynchronous copies have
// landed (an arrival of every thread), and for pieces that it stored itself
// (one a warp).  It does not wait for them, and the fence that lets products
// read what ordinary stores and copies wrote is the product warp's: before a
// load warp's arrival that fence would wait for every copy in flight.
//
// Every load warp arrives for every chunk that is its group's, loads or not,
// and so does the box warp: a warp that fell two of a slot's turns behind would
// take its barrier's phase for another one.
constexpr uint32_t kFullArrivals = kLoadGroup * 33 + 1;
__device__ __forceinline__ void arrive_idle(uint64_t *bar, int lane, const Waiter &waiter)
{
    if (lane == 0 && !waiter.dead)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 33;" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void arrive_full(uint64_t *bar, int lane, const Waiter &waiter)
{
    if (!waiter.dead)
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
    __syncwarp();
    if (lane == 0 && !waiter.dead) mbar_arrive(bar);
}

__device__ __forceinline__ uint16_t load2(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}

// A box of a stack of matrices, as load_box of one.  (The lo part of V begins at a multiple of 16 columns.)
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
// Boxes are 32 rows high.  Bit i of the result: rows 32 i .. of a tile are not
// consecutive tokens, so that no box holds them; `y` is the first token of the
// group of 32 that lane 8 i belongs to.  (A box with rows past the tile's
// tokens brings others', which reach only themselves.)
constexpr int kBoxRows = 32;
__device__ __forceinline__ uint32_t scattered(const AdapterArgs &g, int first, int count, int lane, int &y)
{
    int t[4];
    bool in_line = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = lane * 4 + j < count ? token_at(g, first + lane * 4 + j) : 0;
    y = __shfl_sync(kFull, t[0], lane & ~7);
#pragma unroll
    for (int j = 0; j < 4; ++j) in_line = in_line && (lane * 4 + j >= count || t[j] == y + (lane & 7) * 4 + j);
    const uint32_t bad = __ballot_sync(kFull, !in_line);
    uint32_t groups = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) groups |= (bad >> (8 * i) & 0xFF ? 1u : 0u) << i;
    return groups;
}

// ------------------------------------------------------- the tokens' part

constexpr int kSums = 4;  // tiles of sums of the second product in TMEM, beside the narrow one's
constexpr uint32_t kTmemCols = 512;

// Shared memory: a ring of slots, each a 128 x 64 tile of In (or of the row to
// add to) and a tile of W1 or W2; then V, hi and lo, whose space first holds
// the block's partial sums.  It takes the whole SM.  Without boxes a slot has
// room beside it for the pieces that rows at any address end in.
template <int RANK, bool FAST>
struct Tok {
    static constexpr int kAtoms = RANK / 64;
    static constexpr uint32_t kWBytes = kAtoms * 64 * 128, kSlot = kInBytes + kWBytes;
    static constexpr uint32_t kVAtom = kTileTokens * 128, kVLo = kAtoms * kVAtom;
    static constexpr int kStages = RANK > 64 ? 4 : FAST ? 8 : 6;
    static_assert(kStages % 2 == 0, "a slot belongs to one load group, which sees each of its phases");
    static constexpr uint32_t kVAt = kStages * kSlot;
    static constexpr uint32_t kExtraAt = kVAt + 2 * kVLo, kExtraW = kTileTokens * 16;
    static constexpr uint32_t kExtra = FAST ? 0 : kExtraW + RANK * 16;
    static constexpr uint32_t kBytes = kExtraAt + kStages * kExtra + 1024;  // room to start at a 1024-byte boundary
    static constexpr int kUnits = RANK / 32;  // a warp's share of V's units in a cluster of two, at most
};

// One row of the plan's table, as a cluster's blocks share it.
struct TileWork {
    int a, first, count;  // count 0: no more tiles
    int used, r16;
    int n1, n2;           // this block's chunks of the two products
};
__device__ __forceinline__ TileWork tile_work(const AdapterArgs &g, int i, uint32_t rank, uint32_t size)
{
    TileWork w = {};
    if (i >= g.rows) return w;
    const int4 t = tile_at(g, i);
    w.a = t.x;
    w.first = t.y;
    w.count = t.z;
    w.used = t.x < 0 || t.x >= g.adapters || w.count <= 0 ? 0 : used_rank(g, t.x);
    w.r16 = (w.used + 15) & ~15;
    const int all1 = w.used ? (g.nin + kChunk - 1) / kChunk : 0;
    // rows without an adapter are copied, in place there is nothing to do
    const int all2 = g.out && (w.used || g.out != g.base) ? (g.nout + kChunk - 1) / kChunk : 0;
    w.n1 = all1 > static_cast<int>(rank) ? (all1 - rank + size - 1) / size : 0;
    w.n2 = all2 > static_cast<int>(rank) ? (all2 - rank + size - 1) / size : 0;
    return w;
}

// N 16-byte pieces, 16 rows apart, from src(0) on: `valid` of a row's eight
// values are there, and rows from `rows` on are empty.  (A copy of no bytes
// reads nothing, whatever its address.)
template <int N, typename Src>
__device__ __forceinline__ void pieces(uint32_t dst, Src src, int valid, int rows)
{
    const uint32_t bytes = valid <= 0 ? 0u : static_cast<uint32_t>(min(valid, 8)) * 2;
#pragma unroll
    for (int q = 0; q < N; ++q) async16(dst + q * 2048, src(q), 16 * q < rows ? bytes : 0u);
}

// A chunk whose pieces are on their way: its slot, and of each of a thread's
// rows, 16 apart, the values to skip (four bits each), In's and the weights'.
struct Late {
    uint32_t rows, weights;
    int slot;
};
// Moves a thread's pieces of one tile down, once its warp's copies are there.
template <int N>
__device__ __forceinline__ void move_rows(uint32_t tile, uint32_t next, uint32_t next_step, uint32_t skips)
{
    if (!__any_sync(kFull, skips != 0)) return;
#pragma unroll 1
    for (int h = 0; h < N; h += 4, skips >>= 16, tile += 4 * 2048, next += 4 * next_step) {
        uint4 x[4], y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q] = load16(tile + q * 2048);
            y[q] = load16(next + q * next_step);
        }
        __syncwarp();  // a row's threads have all read it
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t skip = skips >> 4 * q & 7;
            if (skip) store16(tile + q * 2048, move_down(x[q], y[q], skip));
        }
    }
}

// Tiles of at most 128 tokens of one adapter, by clusters that take tiles in
// turn.  A cluster's blocks take every c-th 64-column chunk of In for the
// narrow product, add up their partial sums through each other's shared memory
// in a fixed order, and take every c-th chunk of the result for the second
// product.  Loads run on through both products and into the next tile.
//
// BACK = false: In = x, W1 = A [R, K], W2 = B [N, R], V = s (x A^T).
// BACK = true:  In = dy, W1 = B [N, R], W2 = A [R, K], V = s (dy B).
// FAST: every row begins at a 16-byte boundary.  Then runs of 32 consecutive
// tokens, and the weights where g.boxes_w says so (a rank that is a multiple of
// 16, which all adapters use), come as boxes.  Boxes of 32 rows brought 5.7 to
// 5.9 TB/s to the SMs, of 16 rows 5.6, of 8 rows 3.8, and a gather of four
// single rows at a time 2.1, so scattered tokens stay with the threads' copies.
//
// Forward of 8192 tokens of 16 adapters in runs, rank 64, 4096 to 8192 columns:
// 67 us for 361 MB (5.4 TB/s, 80% of a copy's rate), the tensor pipe busy 15%
// of the time.
//
// Rows at any address come as aligned pieces too, and the load warps move them
// down in shared memory when they are there; a chunk later, so that a group has
// two on their way (three would wait for slots: 244 instead of 205 us at the
// time).  16,384 tokens, rank 64, 4095 to 4097 columns: 159 us forward (rows
// read through registers 435 us; aligned rows 76 us): the results' warps, which
// move rows up to the output's alignment, bound it.  777 scattered tokens of
// five adapters from 1001 to 2047 columns: 20 us, the few dependent steps of a
// tile (plan, chunks, meeting, second product).
template <bool BACK, int RANK, bool FAST>
__global__ void __launch_bounds__(kTokThreads, 1)
    k_adapter(const __grid_constant__ AdapterArgs g, const __grid_constant__ TokenMaps maps)
{
    using T = Tok<RANK, FAST>;
    constexpr int S = T::kStages;
    extern __shared__ uint8_t raw[];
    // a slot is full, and free again; the narrow product, and a tile of sums of the second one, is there, the latter
    // free again; the cluster's meetings
    __shared__ uint64_t full[S], freed[S], narrow, summed[kSums], sum_free[kSums], meet[3];
    __shared__ uint32_t tmem_at;

    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int clusters = gridDim.x / size, first_tile = blockIdx.x / size;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u, v_at = base + T::kVAt;
    if (BACK) pdl_launch_dependents();  // the weights' gradients may set themselves up
    const TileWork first_work = tile_work(g, first_tile, rank, size);  // on its way while the block sets itself up

    if (warp == 0) tmem_alloc(&tmem_at, kTmemCols);
    if (FAST && warp == kBoxWarp && lane == 0) {
        fetch_map(&maps.in);
        if (g.out) fetch_map(&maps.base);
        if (g.boxes_w) {
            fetch_map(&maps.a);
            fetch_map(&maps.b);
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], kFullArrivals);
            mbar_init(&freed[i], 1);
        }
        mbar_init(&narrow, 1);
        for (int i = 0; i < kSums; ++i) {
            mbar_init(&summed[i], 1);
            mbar_init(&sum_free[i], 4);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&meet[i], kOutWarps * size);
        fence_mbar_init();
    }
    tc_before();
    __syncthreads();
    tc_after();
    // barriers are there for the peers; who reaches out to theirs waits for that first
    if (size > 1) cluster_arrive();
    const uint32_t tmem = tmem_at;
    Waiter waiter;

    if (warp >= kLoadWarp) {
        // ------------------------------------------------------------ loads
        const int group = (warp - kLoadWarp) / kLoadGroup, id = (threadIdx.x - 32 * kLoadWarp) & 127;
        const int row0 = id >> 3, col = (id & 7) * 8;  // 8 threads a row of 64 columns, 16 rows at a time
        const uint32_t at = swz(row0, id & 7);
        int i = 0, s = 0;
        auto next = [&]() {
            ++i;
            s = s + 1 == S ? 0 : s + 1;
        };
        // rows at any address: the last chunk whose pieces are to be moved when they are there, if any
        Late late = {};
        bool flying = false;
        const uint32_t extra0 = base + T::kExtraAt + row0 * 16;
        auto settle = [&](const Late &c) {
            const uint32_t slot = base + c.slot * T::kSlot, extra = extra0 + c.slot * T::kExtra;
            const bool end = (id & 7) == 7;
            const uint32_t next = swz(row0, (id + 1) & 7);
            move_rows<8>(slot + at, end ? extra : slot + next, end ? 256 : 2048, c.rows);
            move_rows<RANK / 16>(slot + kInBytes + at, end ? extra + T::kExtraW : slot + kInBytes + next,
                                 end ? 256 : 2048, c.weights);
            __syncwarp();
            arrive_idle(&full[c.slot], lane, waiter);
        };
        for (int tile = first_tile;; tile += clusters) {
            const TileWork w = tile == first_tile ? first_work : tile_work(g, tile, rank, size);
            if (w.count <= 0) break;
            const int start = rank * kChunk + col, stride = static_cast<int>(size) * kChunk;
            const int left = w.count - row0;  // rows from this thread's first one on
            int y;
            const uint32_t loose = FAST ? scattered(g, w.first, w.count, lane, y) : 0xFu;
            const bool boxes_w = FAST && g.boxes_w;
            int t[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) t[q] = 16 * q < left ? token_at(g, w.first + row0 + 16 * q) : 0;
            // A: R rows, 64 columns; B: 64 rows, R columns
            const __nv_bfloat16 *A = g.a + (static_cast<int64_t>(w.a) * g.rank + row0) * g.k + start;
            const __nv_bfloat16 *B = g.b + (static_cast<int64_t>(w.a) * g.n + rank * kChunk + row0) * g.rank + col;
            auto load_a = [&](uint32_t to, int step) {
                const int valid = g.k - start - step, rows = w.used - row0;
                const int64_t down = static_cast<int64_t>(16) * g.k;
                if (RANK > 64 && w.r16 > 64)
                    pieces<RANK / 16>(to + at, [&](int q) { return A + step + q * down; }, valid, rows);
                else if (w.r16 > 32)
                    pieces<4>(to + at, [&](int q) { return A + step + q * down; }, valid, rows);
                else if (w.r16 > 16)
                    pieces<2>(to + at, [&](int q) { return A + step + q * down; }, valid, rows);
                else
                    pieces<1>(to + at, [&](int q) { return A + step + q * down; }, valid, rows);
            };
            auto load_b = [&](uint32_t to, int step) {
                const int rows = g.n - (start - col) - step - row0;
                const int64_t down = static_cast<int64_t>(16) * g.rank;
                const __nv_bfloat16 *from = B + static_cast<int64_t>(step) * g.rank;
#pragma unroll
                for (int h = 0; h < T::kAtoms; ++h)
                    if (col + 64 * h < w.r16)
                        pieces<4>(to + at + h * 64 * 128, [&](int q) { return from + 64 * h + q * down; },
                                  w.used - col - 64 * h, rows);
            };
            // the rows of In or of what is added to; rows past the tile's tokens stay as they are, by 16 at the
            // least: they reach only themselves
            // at any address: the values to skip, which no step changes (64 columns, and 64 rows, are 128 bytes or
            // a multiple), four bits a row, and the pieces' aligned addresses
            const int piece = id & 7;
            uint32_t skips_a = 0, skips_b = 0;
            if (!FAST) {
#pragma unroll
                for (int q = 0; q < RANK / 16; ++q) {
                    if (row0 + 16 * q < w.used) skips_a |= skip_of(A - col + static_cast<int64_t>(16 * q) * g.k) << 4 * q;
                    if (q / 4 * 64 < w.used)
                        skips_b |= skip_of(B - col + static_cast<int64_t>(q % 4 * 16) * g.rank + q / 4 * 64) << 4 * q;
                }
            }
            auto product = [&](const __nv_bfloat16 *m, int64_t ld, int cols, int chunks, bool two) {
                const __nv_bfloat16 *p[8];
                uint32_t skips = 0;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    p[q] = m + t[q] * ld + start;
                    if (!FAST) {
                        const uint32_t skip = skip_of(p[q] - col);
                        p[q] -= skip;
                        if (16 * q < left) skips |= skip << 4 * q;
                    }
                }
                int step = 0;  // columns from the first chunk
                for (int k = 0; k < chunks; ++k, next(), step += stride) {
                    if ((i & 1) != group) continue;
                    if (i >= S) waiter.wait(&freed[s], (i / S - 1) & 1);
                    const uint32_t slot = base + s * T::kSlot;
                    if (FAST) {
                        if (loose == 0 && (boxes_w || !w.used)) {  // boxes hold all of it
                            arrive_idle(&full[s], lane, waiter);
                            continue;
                        }
#pragma unroll
                        for (int q = 0; q < 8; q += 2)
                            if (loose >> q / 2 & 1)
                                pieces<2>(slot + at + q * 2048, [&](int e) { return p[q + e] + step; },
                                          cols - start - step, left - 16 * q);
                        if (w.used && !boxes_w)
                            two == BACK ? load_a(slot + kInBytes, step) : load_b(slot + kInBytes, step);
                        arrive_full(&full[s], lane, waiter);
                        continue;
                    }
                    const uint32_t extra = extra0 + s * T::kExtra, extra_w = extra + T::kExtraW;
                    const int here = start - col + step;  // the chunk's first column
                    if (cols - here >= kChunk) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (16 * q < w.count) async16(slot + at + q * 2048, p[q] + step, 16 * q < left ? 16 : 0);
                        if (piece == 7 && skips)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (skips >> 4 * q & 7)
                                    async16(extra + q * 256, p[q] + step + 8, 2 * (skips >> 4 * q & 7));
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (16 * q < w.count)
                                raw_piece<8>(slot + at + q * 2048, extra + q * 256, p[q] + step, skips >> 4 * q & 7, piece,
                                             16 * q < left ? cols - here : 0);
                    }
                    const uint32_t to = slot + kInBytes + at;
                    uint32_t skips_w = two == BACK ? skips_a : skips_b;
                    if (two == BACK) {
                        const __nv_bfloat16 *from = A + step;
                        const int64_t down = static_cast<int64_t>(16) * g.k;
#pragma unroll 2
                        for (int q = 0; 16 * q < w.r16; ++q, from += down) {
                            const uint32_t skip = skips_w >> 4 * q & 7;
                            raw_piece<8>(to + q * 2048, extra_w + q * 256, from - skip, skip, piece,
                                         row0 + 16 * q < w.used ? g.k - here : 0);
                        }
                    } else {
                        const __nv_bfloat16 *from = B + static_cast<int64_t>(step) * g.rank;
                        const int64_t down = static_cast<int64_t>(16) * g.rank;
#pragma unroll 2
                        for (int q = 0; q / 4 * 64 < w.r16; ++q) {
                            const uint32_t skip = skips_w >> 4 * q & 7;
                            raw_piece<8>(to + q * 2048, extra_w + q * 256, from + q % 4 * down + q / 4 * 64 - skip, skip,
                                         piece, here + row0 + q % 4 * 16 < g.n ? w.used - q / 4 * 64 : 0);
                        }
                    }
                    if (!__any_sync(kFull, (skips | skips_w) != 0)) {
                        if (flying) {
                            async_wait<0>();
                            __syncwarp();
                            settle(late);
                            flying = false;
                        }
                        arrive_full(&full[s], lane, waiter);
                        continue;
                    }
                    async_commit();
                    if (flying) {
                        async_wait<1>();
                        __syncwarp();
                        settle(late);
                    }
                    flying = true;
                    late = {skips, skips_w, s};
                }
            };
            product(g.in, g.ld_in, g.nin, w.n1, false);
            product(g.base, g.ld_base, g.nout, w.n2, true);
        }
        async_wait<0>();
        __syncwarp();
        if (flying) settle(late);
    } else if (warp == kBoxWarp) {
        // ------------------------------------------------------------ boxes
        int i = 0, s = 0;
        for (int tile = first_tile;; tile += clusters) {
            const TileWork w = tile == first_tile ? first_work : tile_work(g, tile, rank, size);
            if (w.count <= 0) break;
            int mine = 0, y[4];
            const uint32_t loose = FAST ? scattered(g, w.first, w.count, lane, mine) : 0xFu;
            uint32_t groups = 0, bytes = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = __shfl_sync(kFull, mine, 8 * j);
                if (j * kBoxRows < w.count && !(loose >> j & 1)) groups |= 1u << j, bytes += kBoxRows * 128;
            }
            const bool weights = FAST && g.boxes_w && w.used;
            // the weights' boxes: A, R rows of 64 columns; B, 64 rows of R columns
            const uint32_t a_bytes = weights ? g.rank * 128 : 0, b_bytes = weights ? T::kWBytes : 0;
            auto product = [&](const CUtensorMap *m, int chunks, bool two) {
                int c0 = rank * kChunk;
                for (int k = 0; k < chunks; ++k, ++i, s = s + 1 == S ? 0 : s + 1, c0 += size * kChunk) {
                    if (i >= S) waiter.wait(&freed[s], (i / S - 1) & 1);
                    if (elect() && !waiter.dead) {
                        const uint32_t slot = base + s * T::kSlot;
                        const uint32_t due = bytes + (two == BACK ? a_bytes : b_bytes);
                        if (due)
                            mbar_expect_tx(&full[s], due);
                        else
                            mbar_arrive(&full[s]);
                        if (FAST) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (groups >> j & 1) load_box(slot + j * kBoxRows * 128, m, c0, y[j], &full[s]);
                            if (weights) {
                                if (two == BACK) {
                                    load_box(slot + kInBytes, &maps.a, c0, 0, w.a, &full[s]);
                                } else {
#pragma unroll
                                    for (int h = 0; h < T::kAtoms; ++h)
                                        load_box(slot + kInBytes + h * 64 * 128, &maps.b, 64 * h, c0, w.a, &full[s]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            };
            product(&maps.in, w.n1, false);
            product(&maps.base, w.n2, true);
        }
        // the block does not end before its boxes are there
        for (int c = max(0, i - S); c < i; ++c) waiter.wait(&full[c % S], (c / S) & 1);
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------- products
        int i = 0, s = 0, q = 0, tiles = 0;  // chunks and their slot, chunks of second products, tiles with a product
        uint64_t *last = nullptr;            // what says that the last products are done
        uint32_t last_parity = 0;
        // descriptors of slot 0's tiles and of V; sixteenths of a byte offset add to them
        const uint64_t in0 = operand(base, 0), v0 = operand(v_at, 0);
        const uint64_t along0 = operand(base + kInBytes, 0), across0 = operand(base + kInBytes, 64 * 128);
        for (int tile = first_tile; !g.stalled; tile += clusters) {
            const TileWork w = tile == first_tile ? first_work : tile_work(g, tile, rank, size);
            if (w.count <= 0) break;
            const uint32_t word1 = mma_word(w.r16, false, BACK), word2 = mma_word(kChunk, false, BACK);
            for (int k = 0; k < w.n1; ++k, ++i, s = s + 1 == S ? 0 : s + 1) {
                waiter.wait(&full[s], (i / S) & 1);
                fence_proxy_async();
                tc_after();
                if (elect() && !waiter.dead) {
                    const uint64_t x = in0 + s * (T::kSlot >> 4), m = (BACK ? across0 : along0) + s * (T::kSlot >> 4);
#pragma unroll
                    for (int j = 0; j < kChunk / 16; ++j)
                        mma(tmem, x + j * 2, m + j * (BACK ? 128 : 2), word1, k > 0 || j > 0);
                    mma_commit(&freed[s]);
                    if (k == w.n1 - 1) mma_commit(&narrow);
                }
                __syncwarp();
            }
            if (w.n1 > 0) last = &narrow, last_parity = tiles & 1;
            for (int k = 0; k < w.n2; ++k, ++i, s = s + 1 == S ? 0 : s + 1, ++q) {
                waiter.wait(&full[s], (i / S) & 1);
                if (k == 0 && w.used) {
                    waiter.wait_cluster(&meet[2], tiles & 1);  // V is there
                    fence_proxy_all();
                }
                if (q >= kSums) waiter.wait(&sum_free[q % kSums], (q / kSums - 1) & 1);
                fence_proxy_async();
                tc_after();
                if (elect() && !waiter.dead) {
                    const uint32_t d = tmem + 128 + q % kSums * kChunk;
                    const uint64_t m = (BACK ? across0 : along0) + s * (T::kSlot >> 4);
#pragma unroll
                    for (int j = 0; j < RANK / 16; ++j) {
                        if (j * 16 >= w.r16) break;
                        const uint64_t v = v0 + (j >> 2) * (T::kVAtom >> 4) + (j & 3) * 2;
                        const uint64_t b = m + (BACK ? j * 128 : (j >> 2) * 512 + (j & 3) * 2);
                        mma(d, v, b, word2, j > 0);
                        mma(d, v + (T::kVLo >> 4), b, word2, true);
                    }
                    mma_commit(&summed[q % kSums]);
                }
                __syncwarp();
                last = &summed[q % kSums], last_parity = (q / kSums) & 1;
            }
            if (w.used) {
                // a block without a chunk of the second product still has to see its V's phase
                if (w.n2 == 0) waiter.wait_cluster(&meet[2], tiles & 1);
                ++tiles;
            }
        }
        if (last) waiter.wait(last, last_parity);
    } else {
        // ---------------------------------------------------------- results
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        int i = 0, q = 0, tiles = 0;
        if (size > 1) cluster_wait();
        for (int tile = first_tile;; tile += clusters) {
            const TileWork w = tile == first_tile ? first_work : tile_work(g, tile, rank, size);
            if (w.count <= 0) break;
            // ranks that the adapter does not use
            if (!BACK && g.keep)
                for (int e = rank * 32 * kOutWarps + threadIdx.x; e < w.count * (g.rank - w.used);
                     e += size * 32 * kOutWarps) {
                    const int r = e / (g.rank - w.used), c = w.used + e - r * (g.rank - w.used);
                    g.keep[static_cast<int64_t>(token_at(g, w.first + r)) * g.rank + c] = 0.0f;
                }
            int t[8];  // the rows that this thread writes: 8 threads a row
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = quarter * 32 + j * 4 + lane / 8;
                t[j] = r < w.count ? token_at(g, w.first + r) : 0;
            }
            if (w.used) {
                // V from the blocks' partial sums.  A unit is 8 of its columns for 32 rows, one row a lane; the
                // cluster's blocks share the units out, and each one adds up its units' partial sums, block by
                // block, and hands the result to every block.
                const int npieces = w.r16 / 8, groups = (w.count + 31) / 32;  // groups of 32 rows
                const float scale = g.scale[w.a];
                out_warps_sync();  // the last tile's second product has been waited for
                if (w.n1 > 0) waiter.wait(&narrow, tiles & 1);
                tc_after();
                __syncwarp();
                float sum[T::kUnits][8] = {};
                auto emit = [&](float (&x)[8], int p, int gr) {
                    const int row = gr * 32 + lane;
                    const bool writes = row < w.count;
                    const int64_t token = writes && (BACK ? g.work != nullptr : g.keep != nullptr)
                                              ? token_at(g, w.first + row) : 0;
                    if (!BACK && g.keep && writes) {
                        float *k = g.keep + token * g.rank + p * 8;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (p * 8 + j < w.used) k[j] = x[j];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] *= scale;
                    if (p * 8 + 8 > w.used)  // the ranks up to the next 16 are products with zeros: zero, whatever In holds
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = p * 8 + j < w.used ? x[j] : 0.0f;
                    uint4 hi, lo;
                    split8(x, hi, lo);
                    const uint32_t to = v_at + (p >> 3) * T::kVAtom + swz(row, p & 7);
                    for (uint32_t peer = 0; peer < size; ++peer) {
                        const uint32_t there = size > 1 ? peer_addr(to, peer) : 0;
                        if (size > 1) {
                            peer_store16(there, hi);
                            peer_store16(there + T::kVLo, lo);
                        } else {
                            store16(to, hi);
                            store16(to + T::kVLo, lo);
                        }
                    }
                    if (BACK && g.work && writes) {
                        // for the weights' gradients, in the plan's order: s dy B, and s (x A^T), as hi and lo
                        const int64_t line = static_cast<int64_t>(w.first + row) * 2 * g.rank16 + p * 8;
                        *reinterpret_cast<uint4 *>(g.work + line) = hi;
                        *reinterpret_cast<uint4 *>(g.work + line + g.rank16) = lo;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = p * 8 + j < w.used ? scale * g.kept[token * g.rank + p * 8 + j] : 0.0f;
                        split8(x, hi, lo);
                        const int64_t far = static_cast<int64_t>(g.tokens) * 2 * g.rank16;
                        *reinterpret_cast<uint4 *>(g.work + far + line) = hi;
                        *reinterpret_cast<uint4 *>(g.work + far + line + g.rank16) = lo;
                    }
                };
                if (size > 1) {
                    if (quarter < groups)
                        for (int p = half; p < npieces; p += 2) {
                            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                            if (w.n1 > 0) {
                                tmem_load8(lanes + p * 8, v);
                                tmem_wait();
                            }
                            const uint32_t to = v_at + (p * 2 * kTileTokens + quarter * 32 + lane) * 16;
                            store16(to, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                   __float_as_uint(v[3])));
                            store16(to + kTileTokens * 16,
                                    make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                               __float_as_uint(v[7])));
                        }
                    arrive_cluster(&meet[0], size, lane, waiter);
                    waiter.wait_cluster(&meet[0], tiles & 1);
                }
                if (size > 1) {
#pragma unroll 1
                    for (int u = 0; u < T::kUnits; ++u) {
                        const int e = static_cast<int>(rank) + static_cast<int>(size) * (warp + kOutWarps * u);
                        if (e >= npieces * groups) break;
                        const int p = e / groups, gr = e - p * groups;
                        const uint32_t from = v_at + (p * 2 * kTileTokens + gr * 32 + lane) * 16;
                        float one[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                        // four blocks' at a time, so that their reads are in flight together
#pragma unroll 1
                        for (uint32_t peer = 0; peer < size; peer += 4) {
                            float4 x[4], y[4];
#pragma unroll
                            for (uint32_t j = 0; j < 4; ++j) {
                                x[j] = y[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                if (peer + j < size) {
                                    const uint32_t there = peer_addr(from, peer + j);
                                    x[j] = peer_float4(there);
                                    y[j] = peer_float4(there + kTileTokens * 16);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                one[0] += x[j].x, one[1] += x[j].y, one[2] += x[j].z, one[3] += x[j].w;
                                one[4] += y[j].x, one[5] += y[j].y, one[6] += y[j].z, one[7] += y[j].w;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < T::kUnits; ++k)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (k == u) sum[k][j] = one[j];
                    }
                    // everyone has read the partial sums that V's place held
                    arrive_cluster(&meet[1], size, lane, waiter);
                    waiter.wait_cluster(&meet[1], tiles & 1);
                }
                // loops of one copy each: this runs once a tile, and fetching its code is most of what it takes
#pragma unroll 1
                for (int u = 0; u < (size > 1 ? T::kUnits : npieces / 2); ++u) {
                    float one[8];
                    int p = half + 2 * u, gr = quarter;
                    if (size > 1) {
                        const int e = static_cast<int>(rank) + static_cast<int>(size) * (warp + kOutWarps * u);
                        if (e >= npieces * groups) break;
                        p = e / groups, gr = e - p * groups;
#pragma unroll
                        for (int k = 0; k < T::kUnits; ++k)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (k == u) one[j] = sum[k][j];
                    } else {
                        if (quarter >= groups) break;
                        tmem_load8(lanes + p * 8, one);
                        tmem_wait();
                    }
                    emit(one, p, gr);
                }
                fence_proxy_all();
                tc_before();
                arrive_cluster(&meet[2], size, lane, waiter);
                ++tiles;
            }
            i += w.n1;
            // Adds the second product's sums to the rows and writes them out, every other chunk.
            __nv_bfloat16 *o[8];
            const int mine = rank * kChunk + (lane & 7) * 8;  // the column of this thread's pieces in its first chunk
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = g.out + t[j] * g.ld_out + mine;
            const int rows_left = w.count - quarter * 32 - lane / 8;  // of the rows it writes, four apart
            for (int k = 0; k < w.n2; ++k, ++i, ++q) {
                if ((q & 1) != half) continue;
                const int s = i % S, step = k * static_cast<int>(size) * kChunk;
                const uint32_t slot = base + s * T::kSlot;
                waiter.wait_both(&full[s], (i / S) & 1, &summed[q % kSums], (q / kSums) & 1);
                tc_after();
                __syncwarp();
                if (quarter * 32 < w.count && w.used) {
                    const int row = quarter * 32 + lane;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[4][8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) tmem_load8(lanes + 128 + q % kSums * kChunk + h * 32 + j * 8, v[j]);
                        tmem_wait();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t at = slot + swz(row, h * 4 + j);
                            const uint4 y = load16(at);
                            const uint32_t x[4] = {y.x, y.y, y.z, y.w};
                            uint32_t r[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                r[e] = pack2(__uint_as_float(x[e] << 16) + v[j][2 * e],
                                             __uint_as_float(x[e] & 0xFFFF0000u) + v[j][2 * e + 1]);
                            store16(at, make_uint4(r[0], r[1], r[2], r[3]));
                        }
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0 && !waiter.dead) mbar_arrive(&sum_free[q % kSums]);
                if (FAST || g.al_out) {
                    const int there = g.nout - mine - step;
                    uint4 v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = load16(slot + swz(quarter * 32 + j * 4 + lane / 8, lane & 7));
                    if (there >= 8) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (4 * j < rows_left) *reinterpret_cast<uint4 *>(o[j] + step) = v[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                            for (int e = 0; e < 7; ++e)
                                if (4 * j < rows_left && e < there)
                                    reinterpret_cast<uint16_t *>(o[j] + step)[e] =
                                        static_cast<uint16_t>(x[e / 2] >> (16 * (e & 1)));
                        }
                    }
                } else {
                    // rows at any address: eight threads write a row's seven whole pieces, and one each of the eight
                    // values that are left at its two ends; four rows' at a time, without a branch inside
                    const int c = lane & 7, here = mine - c * 8 + step;
                    const bool whole = g.nout - here >= kChunk;
#pragma unroll
                    for (int j0 = 0; j0 < 8; j0 += 4) {
                        uint4 x[4], y[4];
                        uint16_t one[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t row = quarter * 32 + (j0 + j) * 4 + lane / 8;
                            const int skip = skip_of(o[j0 + j]), e = c < 8 - skip ? c : 56 + c;
                            x[j] = load16(slot + swz(row, skip ? (c + 7) & 7 : c));
                            y[j] = load16(slot + swz(row, c));
                            one[j] = load2(slot + swz(row, e >> 3) + (e & 7) * 2);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int skip = skip_of(o[j0 + j]), e = c < 8 - skip ? c : 56 + c;
                            const bool mine_too = 4 * (j0 + j) < rows_left;
                            __nv_bfloat16 *to = o[j0 + j] + step;
                            const uint4 v = move_down(x[j], y[j], 8 - skip);  // (moved by eight it is x)
                            if (mine_too && skip && here + e < g.nout)
                                reinterpret_cast<uint16_t *>(to)[e - c * 8] = one[j];
                            if (whole) {
                                if (mine_too && (!skip || c)) *reinterpret_cast<uint4 *>(to - skip) = v;
                            } else if (mine_too && (!skip || c)) {
                                const int there = g.nout - here - c * 8 + skip;
                                const uint32_t z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (e < there)
                                        reinterpret_cast<uint16_t *>(to - skip)[e] =
                                            static_cast<uint16_t>(z[e / 2] >> (16 * (e & 1)));
                            }
                        }
                    }
                }
                fence_proxy_async();  // the slot's next chunk may be a box
                set_sync(half);
                if ((threadIdx.x & 127) == 0 && !waiter.dead) mbar_arrive(&freed[s]);
            }
        }
    }
    if (waiter.dead) fail(g, LCT_ERR_TIMEOUT);
    __syncwarp();
    if (size > 1 && warp >= kOutWarps) cluster_wait();
    tc_before();
    __syncthreads();
    if (size > 1) cluster_sync();  // no block leaves while a peer may still reach its memory
    if (warp == 0) tmem_free(tmem, kTmemCols);
}

// Rows without an adapter: out = base, and nothing to keep.
__device__ __forceinline__ void copy_rows(const AdapterArgs &g, const int *tok, int count)
{
    const uint32_t rank = cluster_rank(), size = cluster_size();
    if (g.out && g.out != g.base) {
        const bool vec = g.al_base && g.al_out;
        const int step = vec ? 8 : 1, per = (g.nout + step - 1) / step;
        const int64_t all = static_cast<int64_t>(count) * per;
        for (int64_t i = rank * kAdThreads + threadIdx.x; i < all; i += size * kAdThreads) {
            const int row = static_cast<int>(i / per), c = static_cast<int>(i - static_cast<int64_t>(row) * per) * step;
            const __nv_bfloat16 *s = g.base + tok[row] * g.ld_base + c;
            __nv_bfloat16 *d = g.out + tok[row] * g.ld_out + c;
            if (vec && c + 8 <= g.nout)
                *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(s);
            else
                for (int j = 0; j < step && c + j < g.nout; ++j) d[j] = s[j];
        }
    }
    if (g.keep)
        for (int i = rank * kAdThreads + threadIdx.x; i < count * g.rank; i += size * kAdThreads)
            g.keep[static_cast<int64_t>(tok[i / g.rank]) * g.rank + i % g.rank] = 0.0f;
}

// ------------------------------------------------ the forward of few tokens

// Where requests bring a token each, an adapter has a handful of rows, and
// what counts is how early its weights are asked for.  Here a cluster takes a
// tile as before, but 16 rows at a time, by warp-wide 16 x 8 products (a tile
// of 128 rows would be empty), in chunks of 128 columns that are all in flight
// at once at the usual sizes: one round trip to memory, one meeting of the
// cluster.  A tile of more than 16 rows makes more passes, its weights then
// coming from L2.  A batch of 17 to 32 tokens whose adapters have more than
// eight on average takes 32 rows at a time: 30 tokens of one adapter of rank 16
// at 4096 columns took 14.9 us in two passes or by the tile kernel, 10.5 us so;
// with an adapter a token it would cost shared memory that a second block on
// the SM needs (32 of 32: 8.2 us, 14.2 us so).  Passes of 32 or 64 rows for
// larger batches were no faster than the tile kernel (64 tokens of one adapter
// 15.6 and 15.2 us, 512 of eight 21.6 and 16.1 us).
//
// One token at rank 16 and 4096 columns takes 7.0 us, of which about 2 us is an
// empty launch's and the rest two dependent trips to memory (plan, then data)
// and the cluster's meeting; 64 tokens of 64 adapters 8.9 us, floor 2.8 us.
constexpr int kFewCols = 128;

template <int RT, int ROWS>
struct Few {
    static constexpr int kTiles = ROWS / 16;  // of 16 rows
    static constexpr int kStages = RT <= 32 ? 8 : 4;
    static constexpr int kWBytes = RT * kFewCols * 2, kSlot = kWBytes + ROWS * kFewCols * 2;
    static constexpr int kSplitR = RT / 16, kSplitK = 8 / kSplitR;  // warps over R, and over a chunk's columns
    static constexpr int kPart = kStages * kSlot;                   // [kSplitK][ROWS][RT] float32
    static constexpr int kSum = kPart + kSplitK * ROWS * RT * 4;    // [ROWS][RT] float32
    static constexpr int kV = kSum + ROWS * RT * 4;                 // hi, lo: [ROWS][RT] BF16
    static constexpr int kBytes = kV + 2 * ROWS * RT * 2;
};

// 16-byte piece c of row r in rows of `pieces` pieces, so that eight rows'
// pieces of one column lie in eight different 16-byte banks.
template <int PIECES>
__device__ __forceinline__ uint32_t few_at(int r, int c)
{
    const int x = PIECES >= 8 ? r & 7 : PIECES == 4 ? (r >> 1) & 3 : (r >> 2) & 1;
    return (r * PIECES + (c ^ x)) * 16;
}

__device__ __forceinline__ void ldm4(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// FAST: every row begins at a 16-byte boundary, so that no load needs a case
// for its alignment (less code, which a launch of a few microseconds notices:
// nothing of it is cached at first).
template <int RT, int ROWS, bool FAST>
__global__ void __launch_bounds__(kAdThreads) k_adapter_few(const __grid_constant__ AdapterArgs g)
{
    using F = Few<RT, ROWS>;
    constexpr int S = F::kStages, TILES = F::kTiles;
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ int tok[kTileTokens];
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int4 tile = tile_at(g, blockIdx.x / size);
    const int count = tile.z;
    if (count <= 0) return;
    for (int i = threadIdx.x; i < count; i += kAdThreads) tok[i] = token_at(g, tile.y + i);
    const int a = tile.x;
    const int used = a < 0 || a >= g.adapters ? 0 : used_rank(g, a);
    if (used == 0) {
        __syncthreads();
        copy_rows(g, tok, count);
        return;
    }
    const uint32_t base = smem_addr(raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const __nv_bfloat16 *A = g.a + static_cast<int64_t>(a) * g.rank * g.k;
    const __nv_bfloat16 *B = g.b + static_cast<int64_t>(a) * g.rank * g.n;
    const int all1 = (g.nin + kFewCols - 1) / kFewCols, all2 = (g.nout + kFewCols - 1) / kFewCols;
    const int n1 = all1 > (int)rank ? (all1 - rank + size - 1) / size : 0;
    const int n2 = all2 > (int)rank ? (all2 - rank + size - 1) / size : 0;
    const int n = n1 + n2;
    // a thread's piece of a row tile
    const int row = threadIdx.x >> 4, c16 = threadIdx.x & 15;
    // a warp's part of the narrow product: 16 ranks from r0, and the 16-column steps k0, k0 + kSplitK ..
    const int r0 = warp % F::kSplitR * 16, k0 = warp / F::kSplitR;

    // chunk i's weights into its slot
    auto load_w = [&](int i) {
        const uint32_t slot = base + (i % S) * F::kSlot;
        if (i < n1) {
            const int at = (rank + i * size) * kFewCols + c16 * 8;
#pragma unroll
            for (int q = 0; q < RT / 16; ++q) {
                const int r = row + 16 * q;
                piece<FAST>(slot + few_at<16>(r, c16), A + static_cast<int64_t>(r) * g.k + at, r < used ? g.k - at : 0,
                            g.al_a);
            }
        } else if (i < n) {
            const int c0 = (rank + (i - n1) * size) * kFewCols;
#pragma unroll
            for (int q = 0; q < RT / 16; ++q) {
                constexpr int P = RT / 8;
                const int id = threadIdx.x + q * kAdThreads, r = id / P, c = id % P;
                piece<FAST>(slot + few_at<P>(r, c), B + static_cast<int64_t>(c0 + r) * g.rank + c * 8,
                            c0 + r < g.n ? used - c * 8 : 0, g.al_b);
            }
        }
    };
    // Where every chunk has a slot of its own, as at the usual sizes, all of them are asked for at once, the weights
    // before the tokens are known, and nothing but the cluster's meeting is waited for on the way.
    const bool at_once = n <= S && count <= ROWS;
    const int ahead = at_once ? S : S - 1;
    // the scale at a thread's four ranks of V, 0 where the adapter has no such rank
    static_assert(kAdThreads % (RT / 4) == 0, "");
    const float scale = g.scale[a];
    float scales[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) scales[j] = static_cast<int>(threadIdx.x) % (RT / 4) * 4 + j < used ? scale : 0.0f;

    for (int first = 0; first < count; first += ROWS) {
#pragma unroll 1
        for (int i = 0; i < ahead; ++i) load_w(i);
        if (first == 0) __syncthreads();  // the tokens are there
        const int rows = min(ROWS, count - first);
        auto load_rows = [&](int i) {
            if (i < n) {
                const bool two = i >= n1;
                const int at = (rank + (two ? i - n1 : i) * size) * kFewCols + c16 * 8;
#pragma unroll
                for (int q = 0; q < TILES; ++q) {
                    if (row + 16 * q >= rows) break;
                    const int64_t t = tok[first + row + 16 * q];
                    piece<FAST>(base + (i % S) * F::kSlot + F::kWBytes + few_at<16>(row + 16 * q, c16),
                                (two ? g.base + t * g.ld_base : g.in + t * g.ld_in) + at, (two ? g.nout : g.nin) - at,
                                two ? g.al_base : g.al_in);
                }
            }
            async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < ahead; ++i) load_rows(i);
        // chunk i is there; every warp has read its slot's last one, so the next one can come
        auto chunk = [&](int i) {
            if (at_once && i > 0) return;
            if (at_once)
                async_wait<0>();
            else
                async_wait<S - 2>();
            __syncthreads();
            if (at_once) return;
            load_w(i + S - 1);
            load_rows(i + S - 1);
        };

        // the narrow product
        float acc[TILES][2][4] = {};
#pragma unroll 1
        for (int i = 0; i < n1; ++i) {
            chunk(i);
            const uint32_t slot = base + (i % S) * F::kSlot, tile_at = slot + F::kWBytes;
#pragma unroll
            for (int k = k0; k < 8; k += F::kSplitK) {
                uint32_t w[4];
                ldm4(slot + few_at<16>(r0 + (lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)), w);
#pragma unroll
                for (int q = 0; q < TILES; ++q) {
                    uint32_t x[4];
                    ldm4(tile_at + few_at<16>(16 * q + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), x);
                    mma16(acc[q][0], x, w[0], w[1]);
                    mma16(acc[q][1], x, w[2], w[3]);
                }
            }
        }
        // the block's sums, over its warps in their order
        float *part = reinterpret_cast<float *>(raw + F::kPart), *sum = reinterpret_cast<float *>(raw + F::kSum);
#pragma unroll
        for (int q = 0; q < TILES; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[(k0 * ROWS + 16 * q + lane / 4 + (j >> 1) * 8) * RT + r0 + h * 8 + (lane & 3) * 2 + (j & 1)] =
                        acc[q][h][j];
        __syncthreads();
        for (int e = threadIdx.x; e < ROWS * RT; e += kAdThreads) {
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < F::kSplitK; ++q) v += part[q * ROWS * RT + e];
            sum[e] = e % RT < used ? v : 0.0f;  // the others are products with zeros: zero, whatever In holds
        }
        __syncwarp();
        if (size > 1)
            cluster_sync();
        else
            __syncthreads();
        // everyone's, over the blocks in their order; V as hi and lo
        for (int e = threadIdx.x; e < ROWS * RT / 4; e += kAdThreads) {
            const int r = e / (RT / 4), c = e % (RT / 4) * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows) {
                float4 x[8];  // all blocks' at once: one after another they took as long as the rest of the launch
#pragma unroll
                for (uint32_t p = 0; p < 8; ++p)
                    x[p] = p < size ? peer_float4(peer_addr(smem_addr(sum + e * 4), p)) : make_float4(0, 0, 0, 0);
#pragma unroll
                for (int p = 0; p < 8; ++p) v.x += x[p].x, v.y += x[p].y, v.z += x[p].z, v.w += x[p].w;
                if (g.keep && e % size == rank) {
                    const float k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // zero where the adapter has no such rank
                        if (c + j < g.rank) g.keep[static_cast<int64_t>(tok[first + r]) * g.rank + c + j] = k[j];
                }
            }
            v.x *= scales[0], v.y *= scales[1], v.z *= scales[2], v.w *= scales[3];
            const uint2 hi = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
            const uint2 lo = make_uint2(pack2(rest(v.x, hi.x << 16), rest(v.y, hi.x & 0xFFFF0000u)),
                                        pack2(rest(v.z, hi.y << 16), rest(v.w, hi.y & 0xFFFF0000u)));
            uint8_t *at = raw + F::kV + few_at<RT / 8>(r, c / 8) + (c & 4) * 2;
            *reinterpret_cast<uint2 *>(at) = hi;
            *reinterpret_cast<uint2 *>(at + ROWS * RT * 2) = lo;
        }
        __syncwarp();
        if (size > 1) cluster_arrive();  // the sums have been read
        __syncthreads();

        // the product back to the full width
#pragma unroll 1
        for (int i = n1; i < n; ++i) {
            chunk(i);
            const uint32_t slot = base + (i % S) * F::kSlot;
            const int c0 = (rank + (i - n1) * size) * kFewCols;
#pragma unroll
            for (int q = 0; q < TILES; ++q) {
                if (16 * q >= rows) break;
                float d[2][4] = {};
#pragma unroll
                for (int k = 0; k < RT / 16; ++k) {
                    uint32_t hi[4], lo[4], w[4];
                    const uint32_t v = base + F::kV + few_at<RT / 8>(16 * q + (lane & 7) + ((lane >> 3) & 1) * 8,
                                                                     2 * k + (lane >> 4));
                    ldm4(v, hi);
                    ldm4(v + ROWS * RT * 2, lo);
                    ldm4(slot + few_at<RT / 8>(warp * 16 + (lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)), w);
                    mma16(d[0], hi, w[0], w[1]);
                    mma16(d[0], lo, w[0], w[1]);
                    mma16(d[1], hi, w[2], w[3]);
                    mma16(d[1], lo, w[2], w[3]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // rows lane / 4 and 8 on, columns 2 (lane % 4) and 8 on
                    const int r = 16 * q + lane / 4 + (j & 1) * 8, h = j >> 1;
                    const int col = warp * 16 + h * 8 + (lane & 3) * 2;
                    if (r >= rows || c0 + col >= g.nout) continue;
                    const uint32_t y = *reinterpret_cast<const uint32_t *>(raw + (slot - base) + F::kWBytes +
                                                                           few_at<16>(r, col >> 3) + (col & 7) * 2);
                    const uint32_t o = pack2(__uint_as_float(y << 16) + d[h][(j & 1) * 2],
                                             __uint_as_float(y & 0xFFFF0000u) + d[h][(j & 1) * 2 + 1]);
                    uint16_t *at = reinterpret_cast<uint16_t *>(g.out) + tok[first + r] * g.ld_out + c0 + col;
                    if ((FAST || g.al_out) && c0 + col + 1 < g.nout) {
                        *reinterpret_cast<uint32_t *>(at) = o;
                    } else {
                        at[0] = static_cast<uint16_t>(o);
                        if (c0 + col + 1 < g.nout) at[1] = static_cast<uint16_t>(o >> 16);
                    }
                }
            }
        }
        async_wait<0>();
        __syncwarp();
        if (size > 1) cluster_wait();  // no block changes its sums, or leaves, before everyone has read them
        __syncthreads();
    }
}

// --------------------------------------------------- the weights' gradients

// dA^T [K, R] = x^T (s dy B) and dB [N, R] = dy^T (s x A^T) of one adapter:
// 256 columns of x or dy by one cluster, whose blocks take every c-th run of
// 64 of the adapter's tokens; their partial sums meet in shared memory in a
// fixed order.  The tokens are the products' inner dimension, so tiles are
// read across: rows of a tile of x are columns of the operand.  256 columns,
// because every block of columns reads V again: 16 KB at R = 64 for 32 KB of x.
//
// 16,384 tokens of one adapter, R = 64, K = N = 4096: 51 us for 277 MB from HBM
// (5.4 TB/s, 81% of a copy's rate), tensor pipe busy 28% of the time; reading
// the tokens from the last one on, for what L2 still holds of dy, changed
// nothing.  2048 tokens of four adapters, R = 32, 1024 to 4096: the two launches
// of the backward pass take 31 us, each a chain of set-up, one trip to memory a
// turn and a meeting, against 4.8 us for the bytes.
//
// The products' rows are V's columns, up to R = 64 its hi part's and below
// them its lo part's, and their 256 columns x's: 12 KB of operands for what
// four products with x's 128 columns as rows would read 24 KB for, which is
// what bounded them (57 cycles each, where 256 x 128 x 16 takes 128).
constexpr int kGradCols = 256, kGradTokens = 64;
constexpr int kGradLoadWarps = 8;  // which write the results at the end
constexpr int kGradMmaWarp = kGradLoadWarps, kGradBoxWarp = kGradMmaWarp + 1;
constexpr int kGradAdThreads = 32 * (kGradBoxWarp + 1);

template <int RANK, int STAGES, bool FAST>
struct Grad {
    static constexpr int kAtoms = RANK / 64;
    // V's hi and lo parts have sums of their own, in lanes of their own or, above R = 64, in columns of their own
    static constexpr uint32_t kTmemCols = RANK <= 64 ? 256 : 512;
    // two load groups take slots in turn, and slots come free in order: of two or more, a group that waits for a
    // slot's last chunk has seen the one before it go
    static_assert(STAGES >= 2, "");
    static constexpr uint32_t kTile = kGradTokens * 128;  // 64 tokens by 64 columns
    static constexpr uint32_t kIn = kGradCols / 64 * kTile, kV = kAtoms * kTile, kSlot = kIn + 2 * kV;
    static constexpr uint32_t kSumRow = (kGradCols + 1) * 4;  // one rank's sums, an odd number of words
    static constexpr uint32_t kSums = RANK * kSumRow;
    static constexpr uint32_t kExtraAt = STAGES * kSlot, kExtra = FAST ? 0 : kGradTokens * 16;  // as in Tok
    static constexpr uint32_t kRing = STAGES * (kSlot + kExtra);
    static constexpr uint32_t kBytes = (kRing > kSums ? kRing : kSums) + 1024;
};
// Blocks that take an SM's whole TMEM share it with no block that takes TMEM too (1 KB of each block's shared memory is
// the system's), so that none waits for another's.
static_assert(Grad<64, 2, true>::kBytes + Grad<128, 2, true>::kBytes + 2048 >= 228 * 1024, "");

// The tokens of a chunk of 64, two a lane, and whether they are two runs of 32
// consecutive ones.
struct ChunkTokens {
    int near, far;
    bool runs;
};
__device__ __forceinline__ ChunkTokens chunk_tokens(const AdapterArgs &g, int at, int last, bool there, int lane)
{
    ChunkTokens c = {0, 0, false};
    if (!there) return c;
    if (at + lane < last) c.near = g.order[at + lane];
    if (at + 32 + lane < last) c.far = g.order[at + 32 + lane];
    const int near0 = __shfl_sync(kFull, c.near, 0), far0 = __shfl_sync(kFull, c.far, 0);
    const int in_line = __all_sync(kFull, c.near == near0 + lane && c.far == far0 + lane);
    c.runs = in_line && at + kGradTokens <= last;  // (a box outside the matrix is zero)
    return c;
}

// The z-th adapter that has tokens, or -1, by a whole block: the rows of the
// plan's table that begin an adapter, counted in order.
__device__ __forceinline__ int busy_adapter(const AdapterArgs &g, int z)
{
    __shared__ int found, counts[kGradAdThreads / 32];
    if (threadIdx.x == 0) found = -1;
    int seen = 0;
    for (int r0 = 0; r0 < g.rows && seen <= z; r0 += kGradAdThreads) {
        const int i = r0 + threadIdx.x;
        const int4 t = i < g.rows ? tile_at(g, i) : make_int4(-1, 0, 0, 0);
        const bool begins = t.z > 0 && t.x >= 0 && t.x < g.adapters && t.y == g.starts[t.x];
        const uint32_t lanes = __ballot_sync(kFull, begins);
        __syncthreads();  // the last round's counts have been read
        if ((threadIdx.x & 31) == 0) counts[threadIdx.x / 32] = __popc(lanes);
        __syncthreads();
        int before = seen;
        for (int w = 0; w < kGradAdThreads / 32; ++w) {
            if (w < static_cast<int>(threadIdx.x / 32)) before += counts[w];
            seen += counts[w];
        }
        if (begins && before + __popc(lanes & ((1u << (threadIdx.x & 31)) - 1)) == z) found = t.x;
    }
    __syncthreads();
    return found;
}

// FAST: every row begins at a 16-byte boundary.  Then a chunk of 64 tokens that
// are two runs of 32 comes as boxes.
template <int RANK, int STAGES, bool FAST>
__global__ void __launch_bounds__(kGradAdThreads)
    k_adapter_grad(const __grid_constant__ AdapterArgs g, const __grid_constant__ GradMaps maps)
{
    using T = Grad<RANK, STAGES, FAST>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[STAGES], freed[STAGES], all_done;
    __shared__ uint32_t tmem_at;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int blocks_x = (g.k + kGradCols - 1) / kGradCols;
    const bool is_a = static_cast<int>(blockIdx.y) < blocks_x;
    const int c0 = (is_a ? blockIdx.y : blockIdx.y - blocks_x) * kGradCols;
    // more adapters than tokens: the gradients are zero already, and only adapters with tokens get blocks
    const int a = g.sparse ? busy_adapter(g, blockIdx.z) : blockIdx.z;
    // every block waits for the tokens' kernel, with work or without: what follows in the stream is ordered behind this
    // grid, and a grid in which nobody waits may end before the one it depends on
    if (a < 0) {
        pdl_wait();
        return;
    }
    const int first = max(0, min(g.starts[a], g.tokens)), last = max(first, min(g.starts[a + 1], g.tokens));
    const int used = last > first ? used_rank(g, a) : 0, r16 = (used + 15) & ~15;
    const int cols = is_a ? g.k : g.n;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    float *sums = reinterpret_cast<float *>(raw + (base - smem_addr(raw)));
    const int all = (last - first + kGradTokens - 1) / kGradTokens;
    const int n = used && all > static_cast<int>(rank) ? (all - rank + size - 1) / size : 0;
    uint32_t tmem = 0;
    Waiter waiter;
    if (used) {
        if (warp == 0) tmem_alloc(&tmem_at, T::kTmemCols);
        if (FAST && warp == kGradBoxWarp && lane < 2) fetch_map(is_a ? (lane ? &maps.d : &maps.x) : (lane ? &maps.v : &maps.dy));
        if (threadIdx.x == 0) {
            for (int i = 0; i < STAGES; ++i) {
                mbar_init(&full[i], kFullArrivals);
                mbar_init(&freed[i], 1);
            }
            mbar_init(&all_done, 1);
            fence_mbar_init();
        }
        tc_before();
        __syncthreads();
        tc_after();
        tmem = tmem_at;
        pdl_wait();  // V is the tokens' kernel's
        auto chunk_at = [&](int i) {
            return first + (static_cast<int>(rank) + i * static_cast<int>(size)) * kGradTokens;
        };
        if (warp < kGradLoadWarps) {
            // Two groups of four warps take chunks in turn.  A warp loads 512 bytes of one token at a time.
            const __nv_bfloat16 *in = is_a ? g.x : g.in;
            const int64_t ld = is_a ? g.ld_x : g.ld_in;
            const __nv_bfloat16 *v = g.work + (is_a ? 0 : static_cast<int64_t>(g.tokens) * 2 * g.rank16);
            const int group = warp / kLoadGroup, id = threadIdx.x & 127, w4 = id >> 5;
            const int at = c0 + lane * 8, valid = cols - at;
            const uint32_t bytes = valid <= 0 ? 0u : static_cast<uint32_t>(min(valid, 8)) * 2;
            const __nv_bfloat16 *from = in + at;
            // its tokens lie four rows apart, so in two places of the eight that the swizzle has
            const uint32_t even = (lane >> 3) * T::kTile + swz(w4, lane & 7);
            const uint32_t odd = (lane >> 3) * T::kTile + swz(w4 + 4, lane & 7);
            // V: 16 threads a token, eight of them its hi part
            const int v_row = id >> 4, v_lo = (id >> 3) & 1, v_c = id & 7;
            const uint32_t v_to = T::kIn + v_lo * T::kV + swz(v_row, v_c);
            // at any address: the last chunk whose pieces are to be moved when they are there, if any, and the values to
            // skip in each of its tokens' rows, four bits each
            uint64_t late = 0;
            int late_slot = -1;
            auto settle = [&]() {
                const uint32_t slot = base + late_slot * T::kSlot;
                const int next = lane + 1, tile = (next >> 3) * T::kTile;
                const uint32_t extra = base + T::kExtraAt + late_slot * T::kExtra + w4 * 16;
                uint32_t far0 = lane == 31 ? extra : slot + tile + swz(w4, next & 7);
                uint32_t far1 = lane == 31 ? extra + 64 : slot + tile + swz(w4 + 4, next & 7);
                const uint32_t down = lane == 31 ? 128 : 1024;
#pragma unroll 1
                for (int h = 0; h < 16; h += 4, far0 += 2 * down, far1 += 2 * down, late >>= 16) {
                    uint4 x[4], y[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x[q] = load16(slot + (q & 1 ? odd : even) + (h + q) / 2 * 1024);
                        y[q] = load16((q & 1 ? far1 : far0) + q / 2 * down);
                    }
                    __syncwarp();  // a row's threads have all read it
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t skip = static_cast<uint32_t>(late >> 4 * q) & 7;
                        if (skip) store16(slot + (q & 1 ? odd : even) + (h + q) / 2 * 1024, move_down(x[q], y[q], skip));
                    }
                }
                __syncwarp();
                arrive_idle(&full[late_slot], lane, waiter);
                late_slot = -1;
            };
            ChunkTokens tokens = chunk_tokens(g, chunk_at(group), last, group < n, lane);
            for (int i = group; i < n; i += 2) {
                const int s = i % STAGES;
                const uint32_t slot = base + s * T::kSlot;
                uint64_t skips = 0;
                const int t0 = chunk_at(i);
                const int left = last - t0;  // tokens from this chunk's first one on; the rest of it is zero
                ChunkTokens now = tokens;
                tokens = chunk_tokens(g, chunk_at(i + 2), last, i + 2 < n, lane);
                if (i >= STAGES) waiter.wait(&freed[s], (i / STAGES - 1) & 1);
                if (FAST && now.runs) {  // boxes hold it
                    arrive_idle(&full[s], lane, waiter);
                    continue;
                }
                now.near = checked_token(g, now.near);
                now.far = checked_token(g, now.far);
                auto token = [&](int row) { return __shfl_sync(kFull, row < 32 ? now.near : now.far, row & 31); };
                if (FAST) {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        async16(slot + (q & 1 ? odd : even) + q / 2 * 1024,
                                from + static_cast<int64_t>(token(w4 + 4 * q)) * ld, w4 + 4 * q < left ? bytes : 0u);
                } else {
                    const uint32_t extra = base + T::kExtraAt + s * T::kExtra + w4 * 16;
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const __nv_bfloat16 *line = in + static_cast<int64_t>(token(w4 + 4 * q)) * ld + c0;
                        const uint32_t skip = w4 + 4 * q < left ? skip_of(line) : 0;
                        raw_piece<32>(slot + (q & 1 ? odd : even) + q / 2 * 1024, extra + q * 64,
                                      line - skip + lane * 8, skip, lane, w4 + 4 * q < left ? cols - c0 : 0);
                        skips |= static_cast<uint64_t>(skip) << 4 * q;
                    }
                }
                for (int c = v_c * 8; c < r16; c += 64) {
                    const __nv_bfloat16 *p = v + (static_cast<int64_t>(t0 + v_row) * 2 + v_lo) * g.rank16 + c;
                    const uint32_t to = slot + v_to + (c >> 6) * T::kTile;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        async16(to + q * 1024, p + q * 16 * g.rank16, v_row + 8 * q < left ? 16 : 0);
                }
                if (FAST) {
                    arrive_full(&full[s], lane, waiter);
                    continue;
                }
                async_commit();
                if (late_slot >= 0) {
                    async_wait<1>();
                    __syncwarp();
                    settle();
                }
                late = skips;
                late_slot = s;
                if (STAGES == 2) {  // the group's only slot
                    async_wait<0>();
                    __syncwarp();
                    settle();
                }
            }
            async_wait<0>();
            __syncwarp();
            if (late_slot >= 0) settle();
            if (n > 0) waiter.wait(&all_done, 0);
        } else if (warp == kGradBoxWarp) {
            ChunkTokens tokens = chunk_tokens(g, chunk_at(0), last, FAST && n > 0, lane);
            for (int i = 0; i < n; ++i) {
                const int s = i % STAGES;
                const ChunkTokens now = tokens;
                tokens = chunk_tokens(g, chunk_at(i + 1), last, FAST && i + 1 < n, lane);
                if (i >= STAGES) waiter.wait(&freed[s], (i / STAGES - 1) & 1);
                const int y[2] = {__shfl_sync(kFull, now.near, 0), __shfl_sync(kFull, now.far, 0)};
                if (!elect() || waiter.dead) {
                } else if (!now.runs) {
                    mbar_arrive(&full[s]);
                } else {
                    const uint32_t slot = base + s * T::kSlot;
                    const CUtensorMap *m = is_a ? &maps.x : &maps.dy, *v = is_a ? &maps.d : &maps.v;
                    mbar_expect_tx(&full[s], T::kSlot);
#pragma unroll
                    for (int j = 0; j < kGradCols / 64; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            load_box(slot + j * T::kTile + h * kBoxRows * 128, m, c0 + 64 * j, y[h], &full[s]);
#pragma unroll
                    for (int j = 0; j < 2 * T::kAtoms; ++j)
                        load_box(slot + T::kIn + j * T::kTile, v, (j >= T::kAtoms) * g.rank16 + j % T::kAtoms * 64,
                                 chunk_at(i), &full[s]);
                }
                __syncwarp();
            }
            if (n > 0) waiter.wait(&all_done, 0);
        } else {
            const uint32_t word = mma_word(min(kGradCols, (cols - c0 + 15) & ~15), true, true);
            const uint64_t in0 = operand(base, T::kTile), v0 = operand(base + T::kIn, T::kTile);
            for (int i = 0; i < n && !g.stalled; ++i) {
                const int s = i % STAGES;
                waiter.wait(&full[s], (i / STAGES) & 1);
                fence_proxy_async();
                tc_after();
                if (elect() && !waiter.dead) {
                    const uint64_t x = in0 + s * (T::kSlot >> 4), v = v0 + s * (T::kSlot >> 4);
#pragma unroll
                    for (int k = 0; k < kGradTokens / 16; ++k) {
                        mma(tmem, v + k * 128, x + k * 128, word, i > 0 || k > 0);
                        if (RANK > 64) mma(tmem + 256, v + (T::kV >> 4) + k * 128, x + k * 128, word, i > 0 || k > 0);
                    }
                    mma_commit(&freed[s]);
                    if (i == n - 1) mma_commit(&all_done);
                }
                __syncwarp();
            }
            if (n > 0) waiter.wait(&all_done, 0);
        }
        tc_after();
        __syncthreads();
        // The block's sums, [rank][column]: lanes hold ranks, up to R = 64 those of the upper half the lo part's (which
        // come first).  Beside an infinity in x or dy, hi and lo of opposite signs would give NaN: lo's sums are taken as
        // finite (they are, where hi's are), so that hi's decide.
        const int quarter = warp & 3, half = warp >> 2;
        const bool lo = RANK <= 64 && quarter >= 2;
        const int r = (RANK <= 64 ? quarter & 1 : quarter) * 32 + lane;
        const uint32_t lanes = tmem + half * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
        const int end = min(128, cols - c0 - half * 128);
        const auto finite = [](float v) { return fmaxf(fminf(v, 0x1.fffffep127f), -0x1.fffffep127f); };
        for (int turn = 0; turn < (RANK <= 64 ? 2 : 1); ++turn) {
            if (warp < kGradLoadWarps && lo == (RANK <= 64 && turn == 0) && r - lane < r16)
                for (int c = 0; c < end; c += 8) {
                    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (n > 0) {
                        tmem_load8(lanes + c, x);
                        if (RANK > 64) tmem_load8(lanes + 256 + c, y);
                        tmem_wait();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float *to = sums + r * (kGradCols + 1) + half * 128 + c + j;
                        *to = RANK > 64 ? x[j] + finite(y[j]) : turn ? *to + x[j] : finite(x[j]);
                    }
                }
            __syncthreads();
        }
        tc_before();
    } else {
        pdl_wait();
    }
    __syncwarp();
    cluster_sync();
    // Everyone's, eight ranks of a column at a time, by the blocks in turn.
    const int col = threadIdx.x;
    if (col < kGradCols && c0 + col < cols)
        for (int p = rank; p * 8 < g.rank; p += size) {
            float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (p * 8 < used)  // sums beyond the used ranks, up to the next 16, are zero
                for (uint32_t peer = 0; peer < size; ++peer) {
                    const uint32_t there = peer_addr(base + p * 8 * T::kSumRow + col * 4, peer);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] += peer_float(there + j * T::kSumRow);
                }
            if (is_a) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (p * 8 + j < g.rank)
                        g.da[(static_cast<int64_t>(a) * g.rank + p * 8 + j) * g.k + c0 + col] =
                            __float2bfloat16_rn(p * 8 + j < used ? x[j] : 0.0f);
            } else {
                __nv_bfloat16 *to = g.db + (static_cast<int64_t>(a) * g.n + c0 + col) * g.rank + p * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = p * 8 + j < used ? x[j] : 0.0f;
                if (g.al_db)
                    *reinterpret_cast<uint4 *>(to) =
                        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (p * 8 + j < g.rank) to[j] = __float2bfloat16_rn(x[j]);
            }
        }
    if (waiter.dead) fail(g, LCT_ERR_TIMEOUT);
    __syncwarp();
    cluster_sync();
    if (used && warp == 0) tmem_free(tmem, T::kTmemCols);
}

// -------------------------------------------------------------- the plan

// The tokens in stable order of their adapter.  Each warp counts a contiguous
// share of the tokens, one row of shared counters an adapter; a scan over
// adapters and warps turns the counts into places, and each warp deals its
// tokens out.  Lanes with the same adapter find each other by a match.  A plan
// is made once for a batch, and what it costs is latency and instructions, not
// its few bytes: 256 tokens of 64 adapters take 4.3 us in one block of few
// warps.  From 4096 tokens on a cluster of eight shares the work and reads each
// other's totals: 16,384 tokens took one block 12 us, two thirds of its issue
// slots in use, and take the cluster 9.3 us.  Tokens are fetched sixteen rounds
// at a time (up to 16,384 in a block once, for both passes).
constexpr int kPlanRounds = 16, kPlanBlocks = 8;
// The lanes with this lane's value; runs of one adapter need no match.
__device__ __forceinline__ unsigned same_adapter(int a)
{
    const int first = __shfl_sync(kFull, a, 0);
    return __all_sync(kFull, a == first) ? kFull : __match_any_sync(kFull, a);
}
__global__ void __launch_bounds__(1024) k_adapter_plan(const __grid_constant__ PlanArgs g)
{
    extern __shared__ int counts[];  // [adapters + 1][warps, and the block's total (which also spreads the banks)]
    __shared__ int part[32], tile_part[32];
    __shared__ int bad;
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31, pitch = warps + 1;
    const int block = cluster_rank(), blocks = cluster_size();
    const int groups = g.adapters + 1;
    const int share = ((g.tokens + warps * blocks - 1) / (warps * blocks) + 31) & ~31;
    const int lo = min(static_cast<int64_t>(g.tokens), static_cast<int64_t>(block * warps + warp) * share);
    const int hi = min(g.tokens, lo + share);
    // a round's adapters, -1 past the end; those outside the bank are as none
    auto fetch = [&](int t0, int (&a)[kPlanRounds]) {
#pragma unroll
        for (int i = 0; i < kPlanRounds; ++i) {
            const int t = t0 + 32 * i + lane;
            a[i] = t < hi ? g.index[t] : -2;
        }
#pragma unroll
        for (int i = 0; i < kPlanRounds; ++i) {
            const bool there = t0 + 32 * i + lane < hi;
            if (there && (a[i] >= g.adapters || a[i] < -1)) bad = 1;
            a[i] = !there ? -1 : a[i] < 0 || a[i] >= g.adapters ? g.adapters : a[i];
        }
    };
    int mine[kPlanRounds];
    if (threadIdx.x == 0) bad = 0;
    for (int i = threadIdx.x; i < groups * pitch; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    for (int t0 = lo; t0 < hi; t0 += 32 * kPlanRounds) {
        fetch(t0, mine);
#pragma unroll
        for (int i = 0; i < kPlanRounds; ++i) {
            if (t0 + 32 * i >= hi) break;
            const unsigned same = same_adapter(mine[i]);
            if (mine[i] >= 0 && lane == __ffs(same) - 1) counts[mine[i] * pitch + warp] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // exclusive places over (adapter, block, warp), and tiles over adapters: each thread takes a run of adapters
    const int run = (groups + blockDim.x - 1) / blockDim.x;
    const int a0 = min(groups, static_cast<int>(threadIdx.x) * run), a1 = min(groups, a0 + run);
    for (int a = a0; a < a1; ++a) {
        int c = 0;
        for (int w = 0; w < warps; ++w) c += counts[a * pitch + w];
        counts[a * pitch + warps] = c;
    }
    __syncwarp();
    if (blocks > 1) cluster_sync();
    // an adapter's tokens in all blocks, and in those before this one
    auto totals = [&](int a, int &earlier) {
        int all = 0;
        earlier = 0;
#pragma unroll
        for (int p = 0; p < kPlanBlocks; ++p) {
            const int c = p >= blocks  ? 0
                          : blocks > 1 ? static_cast<int>(ld_peer_shared(&counts[a * pitch + warps], p))
                                       : counts[a * pitch + warps];
            all += c;
            if (p < block) earlier += c;
        }
        return all;
    };
    bool any_bad = bad;
    if (blocks > 1) {
        any_bad = false;
        for (int p = 0; p < blocks; ++p) any_bad = any_bad || ld_peer_shared(&bad, p);
    }
    int sum = 0, tiles = 0, earlier;
    for (int a = a0; a < a1; ++a) {
        const int c = totals(a, earlier);
        sum += c;
        tiles += (c + kTileTokens - 1) / kTileTokens;
    }
    int before = sum, tiles_before = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, before, o), y = __shfl_up_sync(kFull, tiles_before, o);
        if (lane >= o) before += x, tiles_before += y;
    }
    if (lane == 31) part[warp] = before, tile_part[warp] = tiles_before;
    __syncthreads();
    int all_tiles = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += part[w], tiles_before += tile_part[w];
        all_tiles += tile_part[w];
    }
    before -= sum;
    tiles_before -= tiles;
    int4 *table = reinterpret_cast<int4 *>(g.tiles);
    for (int a = a0; a < a1; ++a) {
        const int first = before;
        before += totals(a, earlier);
        int place = first + earlier;
        for (int w = 0; w < warps; ++w) {
            const int c = counts[a * pitch + w];
            counts[a * pitch + w] = place;
            place += c;
        }
        if (block == 0) g.starts[a] = first;
        for (int t = first; t < before; t += kTileTokens) {
            const int flag = tiles_before == 0 && any_bad ? LCT_ERR_INVALID_ARG : 0;
            if (block == 0) table[tiles_before] = make_int4(a == g.adapters ? -1 : a, t, min(kTileTokens, before - t), flag);
            ++tiles_before;
        }
    }
    __syncwarp();
    if (blocks > 1) cluster_arrive();  // the totals have been read
    if (block == 0 && threadIdx.x == 0) g.starts[groups] = g.tokens;
    for (int i = all_tiles + block * blockDim.x + threadIdx.x; i < g.rows; i += blocks * blockDim.x)
        table[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int t0 = lo; t0 < hi; t0 += 32 * kPlanRounds) {
        if (hi - lo > 32 * kPlanRounds) fetch(t0, mine);  // a shorter share is still there
#pragma unroll
        for (int i = 0; i < kPlanRounds; ++i) {
            if (t0 + 32 * i >= hi) break;
            const unsigned same = same_adapter(mine[i]);
            int at = 0;
            if (mine[i] >= 0) at = counts[mine[i] * pitch + warp];
            __syncwarp();
            if (mine[i] >= 0) {
                g.order[at + __popc(same & ((1u << lane) - 1))] = t0 + 32 * i + lane;
                if (lane == __ffs(same) - 1) counts[mine[i] * pitch + warp] = at + __popc(same);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    if (blocks > 1) cluster_wait();  // no block leaves before its totals have been read
}

}  // namespace dev

namespace {

// Clusters take tiles in turn, one block on an SM.  Larger clusters end a
// tile sooner, but fewer of them fit (36 of four and 15 of eight on 152 SMs),
// and a turn has a part that no cluster shortens (filling the ring, the
// meetings), which measures like about 12 chunks: the size with the least
// turns x (chunks of a turn + 12) is taken, a chunk of the second product
// counting twice for what it writes.  Clusters of 12 and 16, of which 8 and 7
// fit, are for 4096 columns and more, ranks up to 64 and batches whose tiles all
// fit at once, whatever the plan holds: 512 tokens of one adapter, rank 16, 8192
// columns take 24.0 us by eight, 18.2 by 16.  Their meetings take longer, the
// more so the higher the rank (500 tokens, rank 64, 1024 columns: 13.8 and 15.8
// us; 128 tokens, rank 128, 4096 columns: 24.1 and 26.8), and a second turn
// costs most (1000 tokens of two adapters, 1024 to 4096 columns: 16.5 us by
// eight, 24.3 by 12).
template <bool BACK, int RANK, bool FAST>
cudaError_t launch_tokens_at(const AdapterArgs &args, cudaStream_t s)
{
    AdapterArgs a = args;
    TokenMaps maps = {};
    if (FAST) {
        bool ok = box_map(&maps.in, a.in, a.nin, a.tokens, a.ld_in, 0, dev::kBoxRows);
        if (ok && a.out) ok = box_map(&maps.base, a.base, a.nout, a.tokens, a.ld_base, 0, dev::kBoxRows);
        a.boxes_w = !a.ranks && a.rank % 16 == 0;
        if (ok && a.boxes_w)
            ok = box_map(&maps.a, a.a, a.k, a.rank, a.k, a.adapters, a.rank) &&
                 box_map(&maps.b, a.b, a.rank, a.n, a.rank, a.adapters, 64);
        if (!ok) return cudaErrorInvalidValue;
    }
    const auto kernel = dev::k_adapter<BACK, RANK, FAST>;
    constexpr uint32_t smem = dev::Tok<RANK, FAST>::kBytes;
    cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (rc != cudaSuccess) return rc;
    const uint64_t n1 = (a.nin + 63) / 64, n2 = a.out ? (a.nout + 63) / 64 : 0;
    // an adapter's last tile is half full at a guess, and with few tokens an adapter it is the only one
    const uint64_t busy = std::min(a.adapters, a.tokens);
    const uint64_t tiles = std::max(a.tokens / 128 + (busy + 1) / 2, busy + a.tokens / 256);
    uint64_t best = ~0ull;
    uint32_t c = 0, fit = 0;
    // (more rows than the smaller of them has clusters: not asked)
    const bool wide = RANK <= 64 && std::max(n1, n2) >= 64 && a.rows <= 152 / 12;
    if (wide) {
        rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (rc != cudaSuccess) return rc;
    }
    for (uint32_t d = 1; d <= (wide ? 16u : 8u) && d <= std::max(n1, n2); d += d < 8 ? 1 : 4) {
        const uint32_t f = clusters_at_once(kernel, dev::kTokThreads, smem, d);
        if (!f || (d > 8 && a.rows > static_cast<int32_t>(f))) continue;
        const uint64_t cost = (tiles + f - 1) / f * ((n1 + d - 1) / d + 2 * ((n2 + d - 1) / d) + 12);
        if (cost < best) best = cost, c = d, fit = f;
    }
    if (!c) return cudaErrorInvalidConfiguration;
    return launch(kernel, dim3(c * std::min(static_cast<uint32_t>(a.rows), fit)), dev::kTokThreads, smem, c, s, a, maps);
}
template <bool BACK>
cudaError_t launch_tokens(const AdapterArgs &a, cudaStream_t s)
{
    const bool fast = a.al_in && a.al_a && a.al_b && (!a.out || (a.al_base && a.al_out));
    if (a.rank <= 64) return fast ? launch_tokens_at<BACK, 64, true>(a, s) : launch_tokens_at<BACK, 64, false>(a, s);
    return fast ? launch_tokens_at<BACK, 128, true>(a, s) : launch_tokens_at<BACK, 128, false>(a, s);
}

// The forward of few tokens, in passes of ROWS.
template <int RT, int ROWS>
cudaError_t launch_few_at(const AdapterArgs &a, cudaStream_t s)
{
    const bool fast = a.al_in && a.al_a && a.al_b && a.al_base && a.al_out;
    const uint32_t chunks = (std::max(a.nin, a.nout) + dev::kFewCols - 1) / dev::kFewCols;
    uint32_t c = 1;
    while (c < 8 && a.rows * c * 2ull <= 608 && 2 * c <= chunks) c *= 2;
    return launch(fast ? dev::k_adapter_few<RT, ROWS, true> : dev::k_adapter_few<RT, ROWS, false>, dim3(c * a.rows),
                  dev::kAdThreads, dev::Few<RT, ROWS>::kBytes, c, s, a);
}
template <int ROWS>
cudaError_t launch_few(const AdapterArgs &a, cudaStream_t s)
{
    return a.rank <= 16   ? launch_few_at<16, ROWS>(a, s)
           : a.rank <= 32 ? launch_few_at<32, ROWS>(a, s)
           : a.rank <= 64 ? launch_few_at<64, ROWS>(a, s)
                          : launch_few_at<128, ROWS>(a, s);
}

}  // namespace

cudaError_t launch_adapter(const AdapterArgs &a, bool back, cudaStream_t s)
{
    const int64_t busy = std::min(a.adapters, a.tokens);
    if (a.stalled) return back ? launch_tokens<true>(a, s) : launch_tokens<false>(a, s);
    if (!back && a.tokens > 16 && a.tokens <= 32 && a.tokens > 8 * busy) return launch_few<32>(a, s);
    if (!back && a.tokens <= 16 * busy) return launch_few<16>(a, s);
    return back ? launch_tokens<true>(a, s) : launch_tokens<false>(a, s);
}

namespace {

// As for the tokens' part; a turn's fixed part measures like about 8 chunks.
// Where an adapter has a chunk or two, the ring is short, so that two blocks
// share an SM.
template <int RANK, int STAGES, bool FAST>
cudaError_t launch_grad_at(const AdapterArgs &a, uint64_t blocks, uint64_t chunks, cudaStream_t s)
{
    const auto kernel = dev::k_adapter_grad<RANK, STAGES, FAST>;
    constexpr uint32_t smem = dev::Grad<RANK, STAGES, FAST>::kBytes;
    const cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (rc != cudaSuccess) return rc;
    uint64_t best = ~0ull;
    uint32_t c = 0;
    for (uint32_t d = 1; d <= 8 && d <= chunks; ++d) {
        const uint32_t f = clusters_at_once(kernel, dev::kGradAdThreads, smem, d);
        if (!f) continue;
        const uint64_t cost = (blocks + f - 1) / f * ((chunks + d - 1) / d + 8);
        if (cost < best) best = cost, c = d;
    }
    if (!c) return cudaErrorInvalidConfiguration;
    const uint32_t cols = (a.k + dev::kGradCols - 1) / dev::kGradCols + (a.n + dev::kGradCols - 1) / dev::kGradCols;
    GradMaps maps = {};
    const uint64_t half = static_cast<uint64_t>(a.tokens) * 2 * a.rank16;
    if (FAST && (!box_map(&maps.x, a.x, a.k, a.tokens, a.ld_x, 0, dev::kBoxRows) ||
                 !box_map(&maps.dy, a.in, a.n, a.tokens, a.ld_in, 0, dev::kBoxRows) ||
                 !box_map(&maps.d, a.work, 2 * a.rank16, a.tokens, 2 * a.rank16, 0, dev::kGradTokens) ||
                 !box_map(&maps.v, a.work + half, 2 * a.rank16, a.tokens, 2 * a.rank16, 0, dev::kGradTokens)))
        return cudaErrorInvalidValue;
    return launch<true>(kernel, dim3(c, cols, a.sparse ? a.tokens : a.adapters), dev::kGradAdThreads, smem, c, s, a, maps);
}

template <int RANK, int STAGES>
cudaError_t launch_grad(const AdapterArgs &a, bool fast, uint64_t blocks, uint64_t chunks, cudaStream_t s)
{
    return fast ? launch_grad_at<RANK, STAGES, true>(a, blocks, chunks, s)
                : launch_grad_at<RANK, STAGES, false>(a, blocks, chunks, s);
}

}  // namespace

cudaError_t launch_adapter_grad(const AdapterArgs &a, cudaStream_t s)
{
    const uint64_t busy = std::min(a.adapters, a.tokens);
    const uint64_t chunks = (a.tokens / busy + dev::kGradTokens - 1) / dev::kGradTokens;
    const uint64_t blocks = ((a.k + dev::kGradCols - 1) / dev::kGradCols + (a.n + dev::kGradCols - 1) / dev::kGradCols) * busy;
    const bool fast = a.al_x && a.al_in, few = chunks <= 2;
    if (a.rank <= 64)
        return few ? launch_grad<64, 2>(a, fast, blocks, chunks, s) : launch_grad<64, 4>(a, fast, blocks, chunks, s);
    return few ? launch_grad<128, 2>(a, fast, blocks, chunks, s) : launch_grad<128, 3>(a, fast, blocks, chunks, s);
}

cudaError_t launch_adapter_plan(const PlanArgs &a, cudaStream_t s)
{
    const uint32_t blocks = a.tokens > 4096 ? dev::kPlanBlocks : 1;
    // two rounds of 32 tokens a warp, as far as the counters leave room for warps
    uint32_t warps = 1;
    while (warps < 32 && warps * blocks * 64 < static_cast<uint32_t>(a.tokens) &&
           (a.adapters + 1ull) * (2 * warps + 1) * 4 <= 200 * 1024)
        warps *= 2;
    return launch(dev::k_adapter_plan, dim3(blocks), warps * 32, (a.adapters + 1) * (warps + 1) * 4, blocks, s, a);
}

namespace {

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A matrix of BF16 rows in memory.
struct Rows {
    const void *p;
    uint64_t ld, cols, rows;
};
bool rows_ok(const Rows &m) { return m.p && al(m.p, 2) && m.ld >= m.cols && m.ld <= kMaxN; }
bool rows_al(const Rows &m) { return al16(m.p) && ((m.ld % 8 == 0 && m.ld < 1ull << 38) || m.rows == 1); }

// Whether two matrices share no value: apart in memory, or column slices of
// rows with one stride that do not meet.
bool rows_apart(const Rows &x, const Rows &y)
{
    if (!x.rows || !y.rows) return true;
    const uint64_t xl = reinterpret_cast<uint64_t>(x.p), yl = reinterpret_cast<uint64_t>(y.p);
    const uint64_t xh = xl + 2 * ((x.rows - 1) * x.ld + x.cols), yh = yl + 2 * ((y.rows - 1) * y.ld + y.cols);
    if (xh <= yl || yh <= xl) return true;
    if (x.ld != y.ld || ((xl ^ yl) & 1)) return false;
    const uint64_t d = yl >= xl ? ((yl - xl) / 2) % x.ld : (x.ld - ((xl - yl) / 2) % x.ld) % x.ld;
    return d >= x.cols && d + y.cols <= x.ld;
}
bool same_rows(const Rows &x, const Rows &y) { return x.p == y.p && x.ld == y.ld; }

bool bytes_apart(const Rows &x, const void *p, uint64_t bytes)
{
    if (!x.rows || !p || !bytes) return true;
    const uint64_t xl = reinterpret_cast<uint64_t>(x.p), pl = reinterpret_cast<uint64_t>(p);
    return xl + 2 * ((x.rows - 1) * x.ld + x.cols) <= pl || pl + bytes <= xl;
}
bool bytes_apart(const void *x, uint64_t xn, const void *p, uint64_t n)
{
    const uint64_t xl = reinterpret_cast<uint64_t>(x), pl = reinterpret_cast<uint64_t>(p);
    return !x || !p || !xn || !n || xl + xn <= pl || pl + n <= xl;
}

lct_status check_bank(const lct_adapters *b, const lct_token_plan *p, AdapterArgs *g)
{
    if (!b || !p) return LCT_ERR_INVALID_ARG;
    if (b->adapters == 0 || b->rank == 0 || b->k == 0 || b->n == 0 || p->adapters != b->adapters)
        return LCT_ERR_INVALID_ARG;
    if (b->rank > LCT_ADAPTER_MAX_RANK || b->adapters > LCT_ADAPTER_MAX || p->tokens > LCT_ADAPTER_MAX_TOKENS ||
        b->k > LCT_ADAPTER_MAX_COLS || b->n > LCT_ADAPTER_MAX_COLS)
        return LCT_ERR_UNSUPPORTED;
    if (!b->d_a || !b->d_b || !b->d_scale || !al(b->d_a, 2) || !al(b->d_b, 2) || !al(b->d_scale, 4) ||
        !al(b->d_ranks, 4))
        return LCT_ERR_INVALID_ARG;
    if ((p->tokens && !p->d_order) || !p->d_starts || !p->d_tiles || !al(p->d_order, 4) || !al(p->d_starts, 4) || !al16(p->d_tiles))
        return LCT_ERR_INVALID_ARG;
    *g = AdapterArgs{};
    g->a = reinterpret_cast<const __nv_bfloat16 *>(b->d_a);
    g->b = reinterpret_cast<const __nv_bfloat16 *>(b->d_b);
    g->scale = b->d_scale;
    g->ranks = b->d_ranks;
    g->adapters = static_cast<int>(b->adapters);
    g->rank = static_cast<int>(b->rank);
    g->rank16 = (g->rank + 15) & ~15;
    g->k = static_cast<int>(b->k);
    g->n = static_cast<int>(b->n);
    g->al_a = al16(b->d_a) && g->k % 8 == 0;
    g->al_b = al16(b->d_b) && g->rank % 8 == 0;
    g->tokens = static_cast<int>(p->tokens);
    g->order = p->d_order;
    g->starts = p->d_starts;
    g->tiles = p->d_tiles;
    g->rows = static_cast<int>(LCT_ADAPTER_TILE_ROWS(p->tokens, p->adapters));
    g->status = p->d_tiles + 3;
    return LCT_OK;
}

// Whether a written region leaves the bank and the plan alone.
bool apart_from_bank(const Rows &m, const AdapterArgs &g)
{
    const uint64_t ab = 2ull * g.adapters * g.rank * g.k, bb = 2ull * g.adapters * g.rank * g.n;
    return bytes_apart(m, g.a, ab) && bytes_apart(m, g.b, bb) && bytes_apart(m, g.scale, 4ull * g.adapters) &&
           bytes_apart(m, g.ranks, 4ull * g.adapters) && bytes_apart(m, g.order, 4ull * g.tokens) &&
           bytes_apart(m, g.starts, 4ull * (g.adapters + 2)) && bytes_apart(m, g.tiles, 16ull * g.rows);
}
Rows flat(const void *p, uint64_t bytes) { return Rows{p, bytes / 2, bytes / 2, p && bytes ? 1ull : 0ull}; }

}  // namespace
}  // namespace lct

using namespace lct;

extern "C" lct_status lct_adapter_plan(const int32_t *d_index, uint64_t tokens, uint64_t adapters, int32_t *d_order,
                                       int32_t *d_starts, int32_t *d_tiles, void *stream)
{
    if (adapters == 0) return LCT_ERR_INVALID_ARG;
    if (adapters > LCT_ADAPTER_MAX || tokens > LCT_ADAPTER_MAX_TOKENS) return LCT_ERR_UNSUPPORTED;
    if (!d_starts || !d_tiles || !al(d_starts, 4) || !al16(d_tiles)) return LCT_ERR_INVALID_ARG;
    if (tokens && (!d_index || !d_order || !al(d_index, 4) || !al(d_order, 4))) return LCT_ERR_INVALID_ARG;
    PlanArgs g;
    g.index = d_index;
    g.order = d_order;
    g.starts = d_starts;
    g.tiles = d_tiles;
    g.tokens = static_cast<int>(tokens);
    g.adapters = static_cast<int>(adapters);
    g.rows = static_cast<int>(LCT_ADAPTER_TILE_ROWS(tokens, adapters));
    const void *out[3] = {d_order, d_starts, d_tiles};
    const uint64_t len[3] = {4 * tokens, 4 * (adapters + 2), 16ull * g.rows};
    for (int i = 0; i < 3; ++i) {
        if (!bytes_apart(out[i], len[i], d_index, 4 * tokens)) return LCT_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (!bytes_apart(out[i], len[i], out[j], len[j])) return LCT_ERR_INVALID_ARG;
    }
    return launch_adapter_plan(g, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
}

namespace {

lct_status forward(const lct_adapters *bank, const lct_token_plan *plan, const uint16_t *d_x, uint64_t ld_x,
                   const uint16_t *d_y, uint64_t ld_y, uint16_t *d_out, uint64_t ld_out, float *d_xa, bool stalled,
                   void *stream)
{
    AdapterArgs g;
    const lct_status rc = check_bank(bank, plan, &g);
    if (rc != LCT_OK) return rc;
    if (plan->tokens == 0) return LCT_OK;
    const uint64_t t = plan->tokens;
    const Rows x{d_x, ld_x, bank->k, t}, y{d_y, ld_y, bank->n, t}, out{d_out, ld_out, bank->n, t};
    if (!rows_ok(x) || !rows_ok(y) || !rows_ok(out) || !al(d_xa, 4)) return LCT_ERR_INVALID_ARG;
    if (!rows_apart(out, x) || (!same_rows(out, y) && !rows_apart(out, y)) || !apart_from_bank(out, g))
        return LCT_ERR_INVALID_ARG;
    const uint64_t kept = d_xa ? 4 * t * bank->rank : 0;
    if (!bytes_apart(x, d_xa, kept) || !bytes_apart(y, d_xa, kept) || !bytes_apart(out, d_xa, kept) ||
        !apart_from_bank(flat(d_xa, kept), g))
        return LCT_ERR_INVALID_ARG;
    g.in = reinterpret_cast<const __nv_bfloat16 *>(d_x);
    g.ld_in = static_cast<int64_t>(ld_x);
    g.nin = g.k;
    g.al_in = rows_al(x);
    g.base = reinterpret_cast<const __nv_bfloat16 *>(d_y);
    g.ld_base = static_cast<int64_t>(ld_y);
    g.al_base = rows_al(y);
    g.out = reinterpret_cast<__nv_bfloat16 *>(d_out);
    g.ld_out = static_cast<int64_t>(ld_out);
    g.al_out = rows_al(out);
    g.nout = g.n;
    g.keep = d_xa;
    g.stalled = stalled;
    return launch_adapter(g, false, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
}

lct_status backward(const lct_adapters *bank, const lct_token_plan *plan, const uint16_t *d_dy, uint64_t ld_dy,
                    const uint16_t *d_x, uint64_t ld_x, const float *d_xa, const uint16_t *d_dx, uint64_t ld_dx,
                    uint16_t *d_dx_out, uint64_t ld_dx_out, uint16_t *d_da, uint16_t *d_db, void *d_work, bool stalled,
                    void *stream)
{
    AdapterArgs g;
    const lct_status rc = check_bank(bank, plan, &g);
    if (rc != LCT_OK) return rc;
    const uint64_t t = plan->tokens;
    const uint64_t abytes = 2ull * bank->adapters * bank->rank * bank->k;
    const uint64_t bbytes = 2ull * bank->adapters * bank->rank * bank->n;
    if (!d_da != !d_db || (!d_da && !d_dx_out) || !al(d_da, 2) || !al(d_db, 2)) return LCT_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (t == 0) {
        if (!d_da) return LCT_OK;
        return cudaMemsetAsync(d_da, 0, abytes, s) == cudaSuccess && cudaMemsetAsync(d_db, 0, bbytes, s) == cudaSuccess
                   ? LCT_OK
                   : LCT_ERR_CUDA;
    }
    const uint64_t kept = 4 * t * bank->rank, work = LCT_ADAPTER_WORK_BYTES(t, bank->rank);
    const Rows dy{d_dy, ld_dy, bank->n, t}, x{d_x, ld_x, bank->k, d_da ? t : 0};
    const Rows dx{d_dx, ld_dx, bank->k, d_dx_out ? t : 0}, out{d_dx_out, ld_dx_out, bank->k, d_dx_out ? t : 0};
    if (!rows_ok(dy) || (d_dx_out && (!rows_ok(dx) || !rows_ok(out)))) return LCT_ERR_INVALID_ARG;
    if (d_da && (!rows_ok(x) || !d_xa || !al(d_xa, 4) || !d_work || !al16(d_work))) return LCT_ERR_INVALID_ARG;
    const Rows written[4] = {out, flat(d_da, d_da ? abytes : 0), flat(d_db, d_db ? bbytes : 0),
                             flat(d_work, d_da ? work : 0)};
    for (int i = 0; i < 4; ++i) {
        if (!written[i].rows) continue;
        if (!rows_apart(written[i], dy) || !rows_apart(written[i], x) || !apart_from_bank(written[i], g) ||
            (d_da && !bytes_apart(written[i], d_xa, kept)))
            return LCT_ERR_INVALID_ARG;
        if (!(i == 0 && same_rows(out, dx)) && !rows_apart(written[i], dx)) return LCT_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (!rows_apart(written[i], written[j])) return LCT_ERR_INVALID_ARG;
    }
    g.in = reinterpret_cast<const __nv_bfloat16 *>(d_dy);
    g.ld_in = static_cast<int64_t>(ld_dy);
    g.nin = g.n;
    g.al_in = rows_al(dy);
    if (d_dx_out) {
        g.base = reinterpret_cast<const __nv_bfloat16 *>(d_dx);
        g.ld_base = static_cast<int64_t>(ld_dx);
        g.al_base = rows_al(dx);
        g.out = reinterpret_cast<__nv_bfloat16 *>(d_dx_out);
        g.ld_out = static_cast<int64_t>(ld_dx_out);
        g.al_out = rows_al(out);
    }
    g.nout = g.k;
    if (d_da) {
        g.x = reinterpret_cast<const __nv_bfloat16 *>(d_x);
        g.ld_x = static_cast<int64_t>(ld_x);
        g.al_x = rows_al(x);
        g.kept = d_xa;
        g.work = static_cast<__nv_bfloat16 *>(d_work);
        g.da = reinterpret_cast<__nv_bfloat16 *>(d_da);
        g.db = reinterpret_cast<__nv_bfloat16 *>(d_db);
        g.al_db = al16(d_db) && g.rank % 8 == 0;
    }
    g.sparse = plan->tokens < bank->adapters;
    g.stalled = stalled;
    if (d_da && g.sparse && (cudaMemsetAsync(d_da, 0, abytes, s) != cudaSuccess ||
                             cudaMemsetAsync(d_db, 0, bbytes, s) != cudaSuccess))
        return LCT_ERR_CUDA;
    if (launch_adapter(g, true, s) != cudaSuccess) return LCT_ERR_CUDA;
    if (d_da && launch_adapter_grad(g, s) != cudaSuccess) return LCT_ERR_CUDA;
    return LCT_OK;
}

}  // namespace

extern "C" lct_status lct_adapter_forward(const lct_adapters *bank, const lct_token_plan *plan, const uint16_t *d_x,
                                          uint64_t ld_x, const uint16_t *d_y, uint64_t ld_y, uint16_t *d_out,
                                          uint64_t ld_out, float *d_xa, void *stream)
{
    return forward(bank, plan, d_x, ld_x, d_y, ld_y, d_out, ld_out, d_xa, false, stream);
}

extern "C" lct_status lct_adapter_backward(const lct_adapters *bank, const lct_token_plan *plan, const uint16_t *d_dy,
                                           uint64_t ld_dy, const uint16_t *d_x, uint64_t ld_x, const float *d_xa,
                                           const uint16_t *d_dx, uint64_t ld_dx, uint16_t *d_dx_out, uint64_t ld_dx_out,
                                           uint16_t *d_da, uint16_t *d_db, void *d_work, void *stream)
{
    return backward(bank, plan, d_dy, ld_dy, d_x, ld_x, d_xa, d_dx, ld_dx, d_dx_out, ld_dx_out, d_da, d_db, d_work, false,
                    stream);
}

extern "C" lct_status lct_debug_adapter_forward_timeout(const lct_adapters *bank, const lct_token_plan *plan,
                                                        const uint16_t *d_x, uint64_t ld_x, const uint16_t *d_y,
                                                        uint64_t ld_y, uint16_t *d_out, uint64_t ld_out, float *d_xa,
                                                        void *stream)
{
    return forward(bank, plan, d_x, ld_x, d_y, ld_y, d_out, ld_out, d_xa, true, stream);
}

extern "C" lct_status lct_debug_adapter_backward_timeout(const lct_adapters *bank, const lct_token_plan *plan,
                                                         const uint16_t *d_dy, uint64_t ld_dy, const uint16_t *d_x,
                                                         uint64_t ld_x, const float *d_xa, const uint16_t *d_dx,
                                                         uint64_t ld_dx, uint16_t *d_dx_out, uint64_t ld_dx_out,
                                                         uint16_t *d_da, uint16_t *d_db, void *d_work, void *stream)
{
    return backward(bank, plan, d_dy, ld_dy, d_x, ld_x, d_xa, d_dx, ld_dx, d_dx_out, ld_dx_out, d_da, d_db, d_work, true,
                    stream);
}
