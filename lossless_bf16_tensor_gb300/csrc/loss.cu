// The cross entropy of a projection onto a large vocabulary, and its gradients,
// a piece of the vocabulary at a time, without keeping logits.  For a token i
// with target t_i, and c_i the gradient of its loss:
//
//   z_iv = x_i W_v,  l_i = log sum_v exp z_iv,  loss_i = l_i - z_{i,t_i}
//   g_iv = c_i (exp(z_iv - l_i) - [v = t_i]),  dx = g W,  dW = g^T x
//
// The four products (z, z again, g W, g^T x) are one kernel, k_product, with four
// ends (of one or two tokens, z is k_logits_few's).  The first turns its tile of z into
// each row's maximum and sum of exponentials, which k_loss_merge joins over the
// tiles and pieces: what leaves the SMs is 8 bytes a token and 64 columns.  The
// second computes z again and writes g as BF16, for a part of the piece that is
// bounded (kGradValues), which the other two read.  Tensor cores bound all of them
// where tokens are many (8192 tokens, 32,768 rows of 4096, in calls: z 1.19 to 1.23 ms,
// 1.8 PFLOP/s, 97% of the tensor pipe's cycles; the gradients 3.8 to 4.1 ms); where they
// are few, reading W from HBM does.
//
// Rounding: products take BF16 and add in float32.  g is rounded to BF16 without
// its target's entry: that one, c_i (exp(-loss_i) - 1), is as large as all others
// of its row together, and goes into dx and dW in float32 (dx: in k_loss_finish;
// dW: sums over the tokens of one target, k_segments, added as dW's tile is
// written), so that both are rounded once.  What g's rounding leaves: rows of dW
// that are nobody's target are 2.3e-3 off (2-norm; 1.66e-3 with one rounding), all
// others and dx 1.66e-3.  g in float32 would double what its products read, each of which
// would become several, of BF16 parts.
//
// The logits of the backward pass are summed over the whole depth by the tensor
// cores, which drop what does not fit, towards zero (sum_steps says what the forward
// pass does against that).  g comes out smaller by the same share for all of a row but
// its target: 1e-4 of it for logits of 12 and 4e-4 of 50, 4096 deep, below the 1.7e-3
// of its rounding; as much as that only for logits of 200 at 4096 or 50 at 16,384 (2.2e-3
// and 1.2e-3).
//
// Tokens without a target are left out of the gradients' products: the others are
// packed in the order of their targets, which the sums over a target's tokens
// need anyway.  What stands in the x of such a token reaches nothing.
#include <algorithm>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>

#include "../../include/lct.h"
#include "../../include/lct_debug.h"
#include "codec_dev.cuh"
#include "internal.h"
#include "rows_dev.cuh"
#include "tensor_dev.cuh"

namespace lct {

enum Product { kLogits, kSoftmax, kDx, kDw };

struct ProductArgs {
    int32_t m, n, k;        // rows, columns and depth of the result
    uint32_t a_rows;        // of a box of A that is not across
    const int32_t *count;   // tokens that are there (rows, or dW's depth); NULL: as given
    int32_t *status;        // latched: a wait that ran out
    int32_t splits;         // kDx: parts of the depth at most, each with a result of its own
    int32_t depth, pairs;   // what their number goes by: the same for all pieces
    int32_t sum_steps;      // kLogits: steps of depth that tensor cores add by themselves
    bool add;               // kDx: to what is there
    bool begins;            // kLogits: a call's first product clears the status and the counter behind it
    const void *ids;        // kLogits: the targets
    bool wide;
    int64_t row0;           // the vocabulary's row that column 0 (kDw: row 0) is
    float2 *part;           // kLogits: [units of 64 columns][m], maximum (in log 2) and sum of exponentials
    float *mine;            // kLogits: the targets' logits, in log 2
    const int32_t *target;  // kSoftmax, packed: targets, l and c
    const float *lse, *share;
    const float *extra;     // kDw: the targets' sums, row first[v] (-1: none)
    const int32_t *first;
    int64_t ld_extra;
    __nv_bfloat16 *out;     // kDw, for rows at any address and where a wait ran out
    int64_t ld_out;
    bool boxes;             // the result is written by boxes (maps.c)
    bool stalled;           // a test: no products are made, so that waits run out
};
struct ProductMaps {
    CUtensorMap a, b, c;
};
struct FewArgs {
    const __nv_bfloat16 *x, *w;
    int64_t ld_x, ld_w;
};
struct MergeArgs {
    const float2 *part;     // [slots][tokens]
    float2 *state;          // [tokens], from piece to piece
    const float *mine;
    const void *ids;
    float *loss, *lse, *total;  // total: sum, mean, 1 / count (or NULL)
    double *sums;           // a block's, for the total
    int32_t *counts, *counter;
    const int32_t *status;
    int64_t tokens, vocab;
    int32_t slots, blocks, block0;
    bool wide, begins, ends;
};
struct PackArgs {
    const __nv_bfloat16 *src;
    __nv_bfloat16 *dst;
    const int32_t *order, *count;  // or NULL: all rows, as they are
    const float *dloss, *scale, *loss, *lse;
    float *lse_out, *share_out, *coef_out;
    int64_t ld_src, ld_dst, dloss_stride;
    int32_t rows, cols;
};
struct FinishArgs {
    const float *part;             // [splits][tokens][ld_part]
    const int32_t *key, *order, *count, *status;
    const float *coef;
    const __nv_bfloat16 *w;        // the vocabulary's matrix, or (gathered) the targets' rows in the packed order
    const void *ids;
    __nv_bfloat16 *dx;
    int64_t ld_part, ld_w, ld_dx, tokens;
    int32_t splits, cols, depth, pairs;  // what dx's product had
    bool gathered, wide;
};

namespace dev {

// --------------------------------------------------------- products by pairs

// A tile of 256 by 256 belongs to two blocks of a cluster, which multiply as
// one (cta_group::2): each holds 128 rows of A, half of the columns of B, and the
// sums of its rows.  Against a block alone on 128 by 256, each operand byte in
// shared memory is used twice as often.
constexpr int kTile = 256, kHalfTile = 128, kDepth = 64;
constexpr int kUnit = 64;  // columns that a warp turns into results at a time
constexpr uint32_t kOperand = kHalfTile * 128;  // 128 rows (or columns) by 64 of depth
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kFirstEndWarp = 4;
constexpr uint32_t kStaging = 32 * 128;  // a warp's 32 rows of 128 bytes
constexpr int kGroup = 16;               // tiles of rows that are worked on side by side
constexpr float kLog2e = 1.4426950408889634f;  // 1 / log 2
// Warps that turn sums into results, two for each quarter of the rows.  (Four,
// for the exponentials of a short depth: 255 columns 8% faster, 1024 and more 3%
// slower.)  Where results leave by boxes, their staging takes the room of a slot.
constexpr int kGroups = 2, kEndWarps = 4 * kGroups, kProductThreads = 32 * (kFirstEndWarp + kEndWarps);
constexpr int kStages = 6;
constexpr uint32_t kStagingAt = kStages * kStage, kProductBytes = kStagingAt + kEndWarps * kStaging + 1024;

__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t word, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// The barrier at this place in both blocks gets an arrival when the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t *at, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// A box into this block's shared memory, which tells a barrier of the pair's first block (`bar`: its address in the
// cluster).
__device__ __forceinline__ void pair_box(uint32_t dst, const CUtensorMap *m, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap *m, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap *m, int x, int y, int z, uint32_t src, bool add)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                         m),
                     "r"(x), "r"(y), "r"(z), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(m),
                     "r"(x), "r"(y), "r"(z), "r"(src)
                     : "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Columns of this lane's row, and the wait for them (one statement: nothing that uses them can come between).
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Parts of dx's depth that give the pairs as much to do as can be.  In steps of a
// pair: tiles go round in turns, in each of which a tile's result takes about
// six, and what every part has to write and k_loss_finish to read takes 0.3 for
// each tile.
__device__ __forceinline__ int parts_of(int tiles, int depth, int most, int pairs)  // by a whole warp
{
    const uint32_t end = static_cast<uint32_t>(max(1, min(most, depth / 4)));
    uint64_t best = ~0ull;
    for (uint32_t s = (threadIdx.x & 31) + 1; s <= end; s += 32) {
        const uint32_t rounds = (tiles * s + pairs - 1) / pairs, steps = (depth + s - 1) / s;
        const uint64_t cost = 10ull * rounds * (steps + 6) + 3ull * s * tiles;
        best = min(best, cost << 8 | s);  // the fewest of the cheapest
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) best = min(best, __shfl_xor_sync(kFull, best, o));
    return static_cast<int>(best & 255);
}

// An item of work: a tile, and the steps of depth that it takes.
struct Item {
    int tm, tn, split, k0, k1;
};
// A pair's items: every `pairs`-th tile, in groups of kGroup tiles of rows, whose
// operand stays in L2 while the columns go by.
struct Items {
    int tiles_m, tiles_n, splits, depth, at, end;
    __device__ __forceinline__ Items(const ProductArgs &g, int m, int k)
    {
        tiles_m = (m + kTile - 1) / kTile;
        tiles_n = (g.n + kTile - 1) / kTile;
        depth = (k + kDepth - 1) / kDepth;
        splits = g.splits > 1 ? parts_of(tiles_m * tiles_n, g.depth, g.splits, g.pairs) : 1;
        at = blockIdx.x / 2;
        end = tiles_m * tiles_n * splits;
    }
    __device__ __forceinline__ bool next(Item &w)
    {
        if (at >= end) return false;
        const int tiles = tiles_m * tiles_n;
        w.split = at / tiles;
        const int t = at - w.split * tiles, g = t / (kGroup * tiles_n), in = t - g * kGroup * tiles_n;
        const int high = min(kGroup, tiles_m - g * kGroup);
        w.tn = in / high;
        w.tm = g * kGroup + in - w.tn * high;
        w.k0 = static_cast<int>(static_cast<int64_t>(depth) * w.split / splits);
        w.k1 = static_cast<int>(static_cast<int64_t>(depth) * (w.split + 1) / splits);
        at += gridDim.x / 2;
        return true;
    }
};

// Logits are held in units of log 2, from the sums over depth on: a difference and
// an exponential of base 2 then have no rounding between them, and the largest
// counts as exactly 1 where the others are next to nothing.

// Each row's maximum and sum of exponentials of N columns joins (m, s).
template <int N>
__device__ __forceinline__ void join_columns(const float (&z)[N], float &m, float &s)
{
    float t[4] = {m, z[1], z[2], z[3]};
    t[0] = fmaxf(t[0], z[0]);
#pragma unroll
    for (int i = 4; i < N; ++i) t[i & 3] = fmaxf(t[i & 3], z[i]);
    const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    const float at = top == -INFINITY ? 0.0f : top;
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) a[i & 3] += exp2_fast(z[i] - at);
    s = fmaf(s, exp2_fast(m - at), (a[0] + a[1]) + (a[2] + a[3]));
    m = top;
}

// dW's values of 32 rows by a unit of columns where a wait ran out: no number that could pass for a gradient.
__device__ __forceinline__ void store_nan(const ProductArgs &g, int row0, int m, int col0)
{
    for (int r = row0; r < min(row0 + 32, m); ++r)
        for (int c = col0 + static_cast<int>(threadIdx.x & 31); c < min(col0 + kUnit, g.n); c += 32)
            g.out[r * g.ld_out + c] = __ushort_as_bfloat16(0x7FFF);
}

// Warps by what they do: warp 0 loads boxes (TMA), warp 1 of the first block
// issues the products, the others turn sums into results, each warp those of a
// quarter of the rows.  Sums are double-buffered in TMEM, so that a tile's end
// runs while the next one's products do.
template <int OP>
__global__ void __launch_bounds__(kProductThreads, 1)
    k_product(const __grid_constant__ ProductArgs g, const __grid_constant__ ProductMaps maps)
{
    constexpr bool kAcrossA = OP == kDw, kAcrossB = OP == kDx || OP == kDw;
    constexpr int S = kStages;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[S], freed[S], done[2], drained[2];
    __shared__ uint32_t tmem_at;
    const uint32_t rank = cluster_rank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    if (warp == 0) pair_alloc(&tmem_at, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&freed[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&drained[i], 2 * kEndWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1 && lane < (OP == kLogits || (OP == kDw && !g.boxes) ? 2 : 3))
        fetch_map(lane == 0 ? &maps.a : lane == 1 ? &maps.b : &maps.c);
    tc_before();
    cluster_sync();
    tc_after();
    const uint32_t tmem = tmem_at;
    pdl_wait();
    if (OP == kLogits && g.begins && blockIdx.x == 0 && threadIdx.x == 0) {
        g.status[0] = 0;
        g.status[1] = 0;
    }
    int m = g.m, k = g.k;
    if (g.count) {
        const int there = max(0, *g.count);
        if (OP == kDw)
            k = min(k, there);
        else
            m = min(m, there);
    }
    // g is not what it should be: no products, and dW says so
    const bool failed = OP == kDw && *g.status;
    Items items(g, m, k);
    Item w;
    Waiter waiter;
    // Barriers tell of boxes, products and reads of TMEM that are done, and of no ordinary write: waits order nothing beyond
    // the block, and arrivals at a peer's barrier nothing at all (a release would wait for the results on their way to memory).
    // Sums that are handed back are in registers by then: tcgen05.wait::ld comes before the arrival, and a fence between.
    auto wait = [&](uint64_t *bar, int parity) { waiter.wait(bar, parity); };
    // where the lanes have to give up together (a vote a step would cost the product's warp 3%)
    auto wait_all = [&](uint64_t *bar, int parity) {
        waiter.wait(bar, parity);
        waiter.dead = __any_sync(kFull, waiter.dead);
    };

    if (warp == 0) {
        // ------------------------------------------------------------- boxes
        int i = 0;
        while (!failed && items.next(w)) {
            const int row = w.tm * kTile + rank * kHalfTile, col = w.tn * kTile + rank * kHalfTile;
            // rows of a second block that has none are not fetched: what is there in their place reaches only itself
            const bool rows = kAcrossA || row < g.m;
            const uint32_t a_bytes = kAcrossA ? kOperand : g.a_rows * 128;
            const uint32_t bytes = 2 * kOperand + (kAcrossA || w.tm * kTile + kHalfTile < g.m ? 2 * a_bytes : a_bytes);
            for (int d = w.k0; d < w.k1; ++d, ++i) {
                const int s = i % S;
                if (i >= S) wait(&freed[s], (i / S - 1) & 1);
                if (elect() && !waiter.dead) {
                    const uint32_t bar = peer_addr(smem_addr(&full[s]), 0), a = base + s * kStage, b = a + kOperand;
                    if (rank == 0) mbar_expect_tx(&full[s], bytes);
                    if (kAcrossA) {
                        pair_box(a, &maps.a, row, d * kDepth, bar);
                        pair_box(a + kOperand / 2, &maps.a, row + 64, d * kDepth, bar);
                    } else if (rows) {
                        pair_box(a, &maps.a, d * kDepth, row, bar);
                    }
                    if (kAcrossB) {
                        pair_box(b, &maps.b, col, d * kDepth, bar);
                        pair_box(b + kOperand / 2, &maps.b, col + 64, d * kDepth, bar);
                    } else {
                        pair_box(b, &maps.b, d * kDepth, col, bar);
                    }
                }
                __syncwarp();
            }
        }
        pdl_launch_dependents();  // (blocks that only wait, from the start, make the product 1 to 2% slower)
        // the block does not end before its boxes have been used
        for (int j = max(0, i - S); j < i; ++j) wait(&freed[j % S], (j / S) & 1);
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------- products
        constexpr uint32_t word = (1u << 4) | (1u << 7) | (1u << 10) | (kAcrossA ? 1u << 15 : 0u) |
                                  (kAcrossB ? 1u << 16 : 0u) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
        const uint64_t a0 = operand(base, kAcrossA ? kOperand / 2 : 0);
        const uint64_t b0 = operand(base + kOperand, kAcrossB ? kOperand / 2 : 0);
        int i = 0, t = 0;
        while (!g.stalled && !failed && items.next(w)) {
            int left = 0;  // steps until these sums are done
            uint32_t sums = tmem;
            bool add = false;
            for (int d = w.k0; d < w.k1; ++d, ++i) {
                if (left == 0) {
                    left = OP == kLogits ? min(g.sum_steps, w.k1 - d) : w.k1 - d;
                    if (t >= 2) wait(&drained[t & 1], (t / 2 - 1) & 1);
                    sums = tmem + (t & 1) * kTile;
                    add = false;
                }
                const int s = i % S;
                wait(&full[s], (i / S) & 1);
                tc_after();
                --left;
                if (elect() && !waiter.dead) {
                    const uint64_t a = a0 + s * (kStage >> 4), b = b0 + s * (kStage >> 4);
#pragma unroll
                    for (int j = 0; j < kDepth / 16; ++j)
                        pair_mma(sums, a + j * (kAcrossA ? 128 : 2), b + j * (kAcrossB ? 128 : 2), word, add || j > 0);
                    pair_commit(&freed[s]);
                    if (left == 0) pair_commit(&done[t & 1]);
                }
                __syncwarp();
                add = true;
                if (left == 0) ++t;
            }
        }
        // every product has ended before the block does
        for (int j = max(0, t - 2); j < t; ++j) wait(&done[j & 1], (j / 2) & 1);
    } else if (warp >= kFirstEndWarp) {
        // -------------------------------------------------------------- ends
        const int quarter = warp & 3, group = (warp - kFirstEndWarp) / 4;
        const uint32_t staging = base + kStagingAt + (warp - kFirstEndWarp) * kStaging;
        int t = 0;
        // the products after the next may take these sums' place
        auto arrive = [&] {
            tc_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                 peer_addr(smem_addr(&drained[t & 1]), 0))
                             : "memory");
        };
        // what a row's results need beside its sums, asked for a tile ahead
        struct RowInfo {
            int target;
            float lse, share;
            int64_t id;
        };
        auto info_of = [&](const Item &of) {
            RowInfo r = {-1, 0.0f, 0.0f, -1};
            const int row = of.tm * kTile + rank * kHalfTile + quarter * 32 + lane;
            if (row < m) {
                if (OP == kLogits) r.id = id_at(g.ids, g.wide, row);
                if (OP == kSoftmax) r.target = g.target[row], r.lse = g.lse[row], r.share = g.share[row];
                if (OP == kDw) r.target = g.first[g.row0 + row];
            }
            return r;
        };
        waiter.dead = failed;
        Item ahead;
        bool more = items.next(ahead);
        RowInfo info = {}, info_ahead = {};
        if (more) info_ahead = info_of(ahead);
        while (more) {
            w = ahead;
            info = info_ahead;
            more = items.next(ahead);
            if (more) info_ahead = info_of(ahead);
            const int row0 = w.tm * kTile + rank * kHalfTile + quarter * 32, row = row0 + lane;
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            if constexpr (OP == kLogits) {
                // this warp's units, their sums over the depth in registers
                constexpr int kUnits = kTile / kUnit / kGroups;
                float z[kUnits][kUnit];
#pragma unroll
                for (int u = 0; u < kUnits; ++u)
#pragma unroll
                    for (int e = 0; e < kUnit; ++e) z[u][e] = 0.0f;
                const int first = w.tn * kTile + group * kUnits * kUnit;
#pragma unroll 1
                for (int d = w.k0; d < w.k1; d += g.sum_steps, ++t) {
                    wait_all(&done[t & 1], (t / 2) & 1);
                    if (waiter.dead) break;
                    tc_after();
                    const uint32_t sums = lanes + (t & 1) * kTile + group * kUnits * kUnit;
#pragma unroll
                    for (int u = 0; u < kUnits; ++u)
#pragma unroll
                        for (int c = 0; c < kUnit; c += 8) {
                            float v[8];
                            tmem_load(sums + u * kUnit + c, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e) z[u][c + e] = fmaf(v[e], kLog2e, z[u][c + e]);
                        }
                    arrive();
                }
                if (waiter.dead) break;
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const int col0 = first + u * kUnit;
                    if (col0 >= g.n) break;
                    int mine = -1;  // the target's column among these
                    if (row < m) {
                        const int64_t id = info.id - g.row0 - col0;
                        if (id >= 0 && id < min(kUnit, g.n - col0)) mine = static_cast<int>(id);
                    }
                    float top = -INFINITY, sum = 0.0f;
                    if (col0 + kUnit > g.n) {
#pragma unroll
                        for (int e = 0; e < kUnit; ++e)
                            if (col0 + e >= g.n) z[u][e] = -INFINITY;
                    }
                    if (mine >= 0) {
#pragma unroll
                        for (int e = 0; e < kUnit; ++e)
                            if (e == mine) g.mine[row] = z[u][e];
                    }
                    join_columns(z[u], top, sum);
                    if (row < m) g.part[static_cast<int64_t>(col0 / kUnit) * m + row] = make_float2(top, sum);
                }
            } else {
                const bool some = w.k1 > w.k0;
                if (some) {
                    wait_all(&done[t & 1], (t / 2) & 1);
                    tc_after();
                }
                if (OP == kDw && waiter.dead) {
                    for (int u = group; u < kTile / kUnit; u += kGroups) store_nan(g, row0, m, w.tn * kTile + u * kUnit);
                    continue;
                }
                if (waiter.dead) break;
                const uint32_t sums = lanes + (t & 1) * kTile;
                const int target = static_cast<int>(info.target - g.row0);
                const float lse = info.lse * kLog2e, share = info.share;
                const float *extra = nullptr;
                if (OP == kDw && info.target >= 0) extra = g.extra + info.target * g.ld_extra;
#pragma unroll 1
                for (int u = group; u < kTile / kUnit; u += kGroups) {
                    const int col0 = w.tn * kTile + u * kUnit;
                    const bool last = u + kGroups >= kTile / kUnit;
                    if constexpr (OP == kDx) {
#pragma unroll 1
                        for (int c = 0; c < kUnit; c += 32) {
                            float v[32];
                            if (some) {
                                tmem_load(sums + u * kUnit + c, v);
                                if (last && c == kUnit - 32) arrive();
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                            }
                            if (lane == 0) bulk_wait_read();  // the last box has left
                            __syncwarp();
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                store16(staging + swz(lane, q),
                                        make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                                   __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])));
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0 && col0 + c < g.n && row0 < m) {
                                store_box(&maps.c, col0 + c, row0, w.split, staging, g.add);
                                bulk_commit();
                            }
                        }
                    } else {
                        uint32_t packed[32];
                        float4 more_of[OP == kDw ? kUnit / 4 : 1];
                        if (OP == kDw && extra) {
#pragma unroll
                            for (int q = 0; q < kUnit / 4; ++q)
                                if (col0 + 4 * q < g.n) more_of[q] = *reinterpret_cast<const float4 *>(extra + col0 + 4 * q);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v[32];
                            if (some) {
                                tmem_load(sums + u * kUnit + 32 * h, v);
                                if (last && h == 1) arrive();
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                            }
                            if (OP == kSoftmax) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = exp2_fast(fmaf(v[e], kLog2e, -lse)) * share;
                                const int at = target - col0 - 32 * h;
                                if (row >= m || (at >= 0 && at < 32)) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (e == at || row >= m) v[e] = 0.0f;
                                }
                            } else if (extra) {
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    if (col0 + 32 * h + 4 * q >= g.n) break;
                                    const float4 add = more_of[OP == kDw ? 8 * h + q : 0];
                                    v[4 * q] += add.x, v[4 * q + 1] += add.y, v[4 * q + 2] += add.z, v[4 * q + 3] += add.w;
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e) packed[16 * h + e] = pack2(v[2 * e], v[2 * e + 1]);
                        }
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            store16(staging + swz(lane, q),
                                    make_uint4(packed[4 * q], packed[4 * q + 1], packed[4 * q + 2], packed[4 * q + 3]));
                        if (OP == kSoftmax || g.boxes) {
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0 && row0 < g.m && col0 < g.n) {
                                store_box(&maps.c, col0, row0, staging);
                                bulk_commit();
                            }
                        } else {
                            __syncwarp();
                            for (int r = 0; r < 32 && row0 + r < m; ++r) {
                                __nv_bfloat16 *to = g.out + (row0 + r) * g.ld_out + col0;
#pragma unroll
                                for (int e = lane; e < kUnit; e += 32) {
                                    uint16_t x;
                                    asm volatile("ld.shared.u16 %0, [%1];"
                                                 : "=h"(x)
                                                 : "r"(staging + swz(r, e / 8) + (e & 7) * 2)
                                                 : "memory");
                                    if (col0 + e < g.n) to[e] = __ushort_as_bfloat16(x);
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
                if (some) ++t;
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    if (waiter.dead) atomicCAS(reinterpret_cast<unsigned int *>(g.status), 0u, static_cast<unsigned int>(LCT_ERR_TIMEOUT));
    __syncwarp();
    tc_before();
    cluster_sync();
    tc_after();
    if (warp == 0) pair_free(tmem, 512);
}

// -------------------------------------------------- the loss from its pieces

constexpr int kMergeTokens = 32, kMergeGroups = 32;

__device__ __forceinline__ void join(float &m, float &s, float2 o)
{
    const float top = fmaxf(m, o.x), at = top == -INFINITY ? 0.0f : top;
    s = s * exp2_fast(m - at) + o.y * exp2_fast(o.x - at);
    m = top;
}

// ------------------------------------------------------------- few tokens

// Logits of one or two tokens, which reading W bounds (32,768 rows of 4096, with
// the merge: 47 us for one token, 5.7 TB/s, 55 for two; by tiles 53 to 62 for up to
// 256).  A warp takes two rows of W at a time, a lane eight columns of 256; x is in
// shared memory.  Sums are float32 multiply-adds, rounded to nearest: with a single
// token's loss there is nothing that an error averages out over, and tiles would
// have to add every 64 of depth in registers to be as exact, which takes them three
// times as long.  W's rows may begin anywhere.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kFewBlocks = 304, kFewMost = 2;

__host__ __device__ constexpr uint32_t few_pitch(uint32_t cols) { return (cols + 255) / 256 * 512; }

// The products of two pairs of BF16 values join two sums.
__device__ __forceinline__ void add_products(float2 &acc, uint32_t a, uint32_t b)
{
    const float2 x = make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    const float2 y = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
    acc = __ffma2_rn(x, y, acc);
}

template <int TOKENS, bool AL>
__global__ void __launch_bounds__(kFewThreads, 2) k_logits_few(const __grid_constant__ ProductArgs g,
                                                                 const __grid_constant__ FewArgs f)
{
    constexpr int ROWS = 2, kSteps = 4;  // of 256 columns, asked for at a time
    extern __shared__ uint4 raw4[];
    __shared__ float2 joined[kFewWarps][TOKENS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t xs = smem_addr(raw4), pitch = few_pitch(g.k);
    pdl_wait();
    pdl_launch_dependents();
    if (g.begins && blockIdx.x == 0 && threadIdx.x < 2) g.status[threadIdx.x] = 0;
    const int pieces = pitch / 16;
    for (int i = threadIdx.x; i < TOKENS * pieces; i += kFewThreads) {
        const int token = i / pieces, c = (i - token * pieces) * 8;
        Piece<__nv_bfloat16, false> p;
        p.q = make_uint4(0, 0, 0, 0);
        if (token < g.m && c < g.k) p.load(f.x + token * f.ld_x, c, g.k);
        store16(xs + token * pitch + c * 2, p.q);
    }
    __syncthreads();
    const int64_t target = lane < g.m ? id_at(g.ids, g.wide, lane) - g.row0 : -1;  // lane t's results are token t's
    float top = -INFINITY, sum = 0.0f;
    for (int row = (blockIdx.x * kFewWarps + warp) * ROWS; row < g.n; row += gridDim.x * kFewWarps * ROWS) {
        float2 acc[ROWS][TOKENS];  // of even and odd columns
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) acc[r][t] = make_float2(0.0f, 0.0f);
        for (int c0 = 0; c0 < g.k; c0 += 256 * kSteps) {
            Piece<__nv_bfloat16, AL> w[kSteps][ROWS];
            auto ask = [&](auto load) {
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
                        load(w[j][r], f.w + min(row + r, g.n - 1) * f.ld_w, c0 + 256 * j + lane * 8);
            };
            if (!AL && c0 + 256 * kSteps <= g.k)
                ask([](auto &p, const __nv_bfloat16 *from, int c) { p.q = load_any(from + c, 16); });
            else
                ask([&](auto &p, const __nv_bfloat16 *from, int c) { p.load(from, c, g.k); });
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                if (c0 + 256 * j >= g.k) break;
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    const uint4 x = load16(xs + t * pitch + (c0 + 256 * j + lane * 8) * 2);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        add_products(acc[r][t], w[j][r].q.x, x.x);
                        add_products(acc[r][t], w[j][r].q.y, x.y);
                        add_products(acc[r][t], w[j][r].q.z, x.z);
                        add_products(acc[r][t], w[j][r].q.w, x.w);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float mine = -INFINITY;
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) {
                float z = acc[r][t].x + acc[r][t].y;
#pragma unroll
                for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
                if (lane == t) mine = z * kLog2e;
            }
            if (row + r >= g.n) break;
            if (target == row + r) g.mine[lane] = mine;
            const float most = fmaxf(top, mine), at = most == -INFINITY ? 0.0f : most;
            sum = sum * exp2_fast(top - at) + exp2_fast(mine - at);
            top = most;
        }
    }
    if (lane < TOKENS) joined[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (warp == 0 && lane < g.m) {
        for (int i = 1; i < kFewWarps; ++i) join(top, sum, joined[i][lane]);
        g.part[static_cast<int64_t>(blockIdx.x) * g.m + lane] = make_float2(top, sum);
    }
}

// Joins the tiles' maxima and sums of 32 tokens a block with the state of the
// pieces before; after the last piece, the losses.  Their sum (double, in the
// order of the blocks) is made by the last block to come.
__global__ void __launch_bounds__(1024) k_loss_merge(const __grid_constant__ MergeArgs g)
{
    __shared__ float2 joined[kMergeGroups][kMergeTokens + 1];
    __shared__ double sums[32];
    __shared__ int counts[32];
    __shared__ bool is_last;
    const int lane = threadIdx.x & 31, group = threadIdx.x / 32;
    const int64_t token0 = static_cast<int64_t>(blockIdx.x) * kMergeTokens;
    pdl_wait();
    pdl_launch_dependents();
    float m = -INFINITY, s = 0.0f;
    if (token0 + lane < g.tokens) {
#pragma unroll 4
        for (int i = group; i < g.slots; i += kMergeGroups) join(m, s, g.part[static_cast<int64_t>(i) * g.tokens + token0 + lane]);
    }
    joined[group][lane] = make_float2(m, s);
    __syncthreads();
    // each warp joins the groups of one token
    const int64_t token = token0 + group;
    const float2 mine = joined[lane][group];
    m = mine.x, s = mine.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float2 other = make_float2(__shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, s, o));
        join(m, s, other);
    }
    double loss = 0.0;
    int counted = 0;
    if (lane == 0 && token < g.tokens) {
        if (!g.begins) join(m, s, g.state[token]);
        if (!g.ends) {
            g.state[token] = make_float2(m, s);
        } else {
            const int64_t id = id_at(g.ids, g.wide, token);
            // the loss of a token that is sure is far smaller than its logits: not by way of lse
            constexpr float kLn2 = 0.6931471805599453f;
            const float tail = *g.status ? __int_as_float(0x7FC00000) : logf(s);
            const float l = id < 0 ? 0.0f : id >= g.vocab ? __int_as_float(0x7FC00000) : fmaf(m - g.mine[token], kLn2, tail);
            g.lse[token] = fmaf(m, kLn2, tail);
            g.loss[token] = l;
            loss = l;
            counted = id >= 0;
        }
    }
    if (!g.ends || !g.total) return;
    if (lane == 0) sums[group] = loss, counts[group] = counted;
    __syncthreads();
    if (group == 0) {
        loss = sums[lane];
        counted = counts[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            loss += __shfl_xor_sync(kFull, loss, o);
            counted += __shfl_xor_sync(kFull, counted, o);
        }
        if (lane == 0) {
            g.sums[blockIdx.x + g.block0] = loss;
            g.counts[blockIdx.x + g.block0] = counted;
            __threadfence();
            is_last = atomicAdd(g.counter, 1) == g.blocks - 1;
        }
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    loss = 0.0;
    counted = 0;
    for (int i = threadIdx.x; i < g.blocks; i += blockDim.x) {
        loss += __ldcg(&g.sums[i]);
        counted += __ldcg(&g.counts[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        loss += __shfl_xor_sync(kFull, loss, o);
        counted += __shfl_xor_sync(kFull, counted, o);
    }
    if (lane == 0) sums[group] = loss, counts[group] = counted;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.0;
        counted = 0;
        for (int i = 0; i < 32; ++i) loss += sums[i], counted += counts[i];
        const int n = max(1, counted);
        g.total[0] = static_cast<float>(loss);
        g.total[1] = static_cast<float>(loss / n);
        g.total[2] = static_cast<float>(1.0 / n);
    }
}

// ----------------------------------------------------------- packed tokens

// Row i of dst is row order[i] of src (NULL: row i), for the tokens that are
// there; rows behind them, as far as a step of depth reaches, are zero.  With
// order, also what the tokens' ends need.
constexpr int kPackRows = 4;  // a block's, asked for together (every block has a warp at least)
template <bool AL>
__global__ void __launch_bounds__(kRowThreads) k_loss_pack(const __grid_constant__ PackArgs g)
{
    pdl_wait();
    pdl_launch_dependents();
    const int i0 = blockIdx.x * kPackRows, piece = piece_of<__nv_bfloat16>(blockIdx.y);
    const int count = g.count ? *g.count : g.rows;
    int64_t token[kPackRows];
#pragma unroll
    for (int r = 0; r < kPackRows; ++r) token[r] = g.order && i0 + r < g.rows ? g.order[i0 + r] : i0 + r;
    const int end = min(g.rows, count + 63);  // (rows behind the last are nobody's, and boxes fill them with zeros)
    Piece<__nv_bfloat16, AL> p[kPackRows];
    const bool inside = !AL && piece + 8 <= g.cols && i0 + kPackRows <= count;  // whole pieces of all rows: no branch between
    if (inside) {
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) p[r].q = load_any(g.src + token[r] * g.ld_src + piece, 16);
    }
#pragma unroll
    for (int r = 0; r < kPackRows; ++r) {
        const int i = i0 + r;
        if (!inside) p[r].q = make_uint4(0, 0, 0, 0);
        if (i >= count) continue;
        if (!inside) p[r].load(g.src + token[r] * g.ld_src, piece, g.cols);
    }
    if (g.order && piece < kPackRows * 8 && i0 + piece / 8 < count) {  // the first threads: what goes with a row
        const int r = piece / 8;
        const int64_t t = r == 0 ? token[0] : r == 1 ? token[1] : r == 2 ? token[2] : token[3];
        const float c = g.dloss[t * g.dloss_stride] * (g.scale ? *g.scale : 1.0f);
        g.lse_out[i0 + r] = g.lse[t];
        g.share_out[i0 + r] = c;
        g.coef_out[i0 + r] = c * expm1f(-g.loss[t]);
    }
#pragma unroll
    for (int r = 0; r < kPackRows; ++r)
        if (i0 + r < end && piece < g.cols)
            *reinterpret_cast<uint4 *>(g.dst + (i0 + r) * g.ld_dst + piece) = p[r].q;
}

// dx of token order[i]: the parts' sum, and the target's term.  Tokens without a
// target get zeros, those with an impossible one NaN.
constexpr int kFinishRows = 2;  // a block's, asked for together
template <bool AL, bool PARTS>
__global__ void __launch_bounds__(kRowThreads) k_loss_finish(const __grid_constant__ FinishArgs g)
{
    using T = __nv_bfloat16;
    constexpr int R = kFinishRows;
    pdl_wait();
    pdl_launch_dependents();
    const int i0 = blockIdx.x * R, piece = piece_of<T>(blockIdx.y), count = *g.count, status = *g.status;
    int token[R], key[R];
    float coef[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = min(i0 + r, static_cast<int>(g.tokens) - 1);
        token[r] = g.order[i];
        key[r] = g.key[i];
        coef[r] = g.coef[i];
    }
    const int parts = PARTS ? parts_of((count + kTile - 1) / kTile * ((g.cols + kTile - 1) / kTile), g.depth, g.splits, g.pairs)
                            : 1;
    T *dx[R];
    int c[R];
    bool there[R];
    Piece<T, AL> w[R];
    float acc[R][kVec<T>];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        dx[r] = g.dx + token[r] * g.ld_dx;
        c[r] = piece - skip_of_row<T, AL>(dx[r]);
        there[r] = i0 + r < count && c[r] < g.cols;
        if (there[r]) w[r].load(g.w + (g.gathered ? i0 + r : key[r]) * g.ld_w, c[r], g.cols);
    }
    auto load_part = [&](float(&v)[kVec<T>], int part, int r) {
        const float *from = g.part + (part * g.tokens + i0 + r) * g.ld_part;
        if (AL) {
            load_floats<T>(v, from, c[r]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) v[e] = c[r] + e >= 0 && c[r] + e < g.cols ? from[c[r] + e] : 0.0f;
        }
    };
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (there[r]) load_part(acc[r], 0, r);
    constexpr int kAhead = 4;  // parts asked for together
    for (int p0 = 1; p0 < parts; p0 += kAhead) {
        float v[kAhead][R][kVec<T>];
#pragma unroll
        for (int p = 0; p < kAhead; ++p)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (there[r] && p0 + p < parts) load_part(v[p][r], p0 + p, r);
#pragma unroll
        for (int p = 0; p < kAhead; ++p)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (there[r] && p0 + p < parts) {
#pragma unroll
                    for (int e = 0; e < kVec<T>; ++e) acc[r][e] += v[p][r][e];
                }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (i0 + r >= g.tokens || c[r] >= g.cols) continue;
        Piece<T, AL> out;
        if (there[r] && !status) {
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) out.v[e] = __float2bfloat16_rn(fmaf(coef[r], to_float(w[r].v[e]), acc[r][e]));
        } else {
            const bool wrong = status || id_at(g.ids, g.wide, token[r]) >= 0;
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) out.v[e] = __float2bfloat16_rn(wrong ? __int_as_float(0x7FC00000) : 0.0f);
        }
        out.store(dx[r], c[r], g.cols);
    }
}

}  // namespace dev

namespace {

// Pairs of blocks that the GPU holds at once, asked for once a device.
template <int OP>
cudaError_t pairs_at_once(int *pairs)
{
    static int known[64] = {};
    int device = 0;
    cudaError_t rc = cudaGetDevice(&device);
    if (rc != cudaSuccess) return rc;
    const int at = device & 63;
    if (!known[at]) {
        rc = cudaFuncSetAttribute(dev::k_product<OP>, cudaFuncAttributeMaxDynamicSharedMemorySize, dev::kProductBytes);
        if (rc != cudaSuccess) return rc;
        const int n = static_cast<int>(clusters_at_once(dev::k_product<OP>, dev::kProductThreads, dev::kProductBytes, 2));
        if (n <= 0) return cudaErrorInvalidConfiguration;
        known[at] = n;
    }
    *pairs = known[at];
    return cudaSuccess;
}

template <int OP>
cudaError_t product(const ProductArgs &g, const ProductMaps &maps, cudaStream_t s)
{
    int pairs;
    const cudaError_t rc = pairs_at_once<OP>(&pairs);
    if (rc != cudaSuccess) return rc;
    const int64_t items = static_cast<int64_t>((g.m + dev::kTile - 1) / dev::kTile) * ((g.n + dev::kTile - 1) / dev::kTile) *
                          g.splits;
    if (items == 0) return cudaSuccess;
    return launch<true>(dev::k_product<OP>, dim3(2 * static_cast<uint32_t>(std::min<int64_t>(items, pairs))),
                        dev::kProductThreads, dev::kProductBytes, 2, s, g, maps);
}

// Whether a forward pass is one of few tokens: x fits beside another block's.
bool is_few(uint64_t tokens, uint64_t cols)
{
    const uint64_t rows = tokens <= 1 ? 1 : 2;
    return tokens <= dev::kFewMost && rows * dev::few_pitch(static_cast<uint32_t>(cols)) <= 100 * 1024;
}
uint32_t few_blocks(uint64_t rows)
{
    return static_cast<uint32_t>(std::min<uint64_t>(dev::kFewBlocks, (rows + 2 * dev::kFewWarps - 1) / (2 * dev::kFewWarps)));
}
template <int TOKENS>
cudaError_t few_at(const ProductArgs &g, const FewArgs &f, bool aligned, cudaStream_t s)
{
    return launch<true>(aligned ? dev::k_logits_few<TOKENS, true> : dev::k_logits_few<TOKENS, false>,
                        dim3(few_blocks(g.n)), dev::kFewThreads, TOKENS * dev::few_pitch(g.k), 1, s, g, f);
}
cudaError_t few(const ProductArgs &g, const FewArgs &f, bool aligned, cudaStream_t s)
{
    return g.m <= 1 ? few_at<1>(g, f, aligned, s) : few_at<2>(g, f, aligned, s);
}

// Tensor cores' float32 sums drop what does not fit, always towards zero: over a depth of 4096 a logit of 12 comes out 5e-5
// too small, and losses of 0.03 are wrong by 4e-5 of their size.  So the sums of every 1024 of depth are added to the rest in
// registers (1.2e-5, and 9e-6 of such losses, as float32 products have), of every 512 where tokens are few (6e-6, 4e-6): there
// it costs nothing, with many up to 3%.  (256: 4 to 8%.)
uint32_t sum_steps(uint64_t tokens) { return (tokens > 1024 ? 1024 : 512) / dev::kDepth; }

// Rows of A's boxes.  Of few tokens no more is fetched than there is (rows behind them reach only themselves).
uint32_t a_rows(uint64_t tokens) { return tokens <= 8 ? 8 : tokens <= 32 ? 32 : dev::kHalfTile; }

cudaError_t pack(const PackArgs &g, bool aligned, cudaStream_t s)
{
    if (g.rows == 0) return cudaSuccess;
    uint32_t threads, slabs;
    row_shape(g.cols, 8, true, &threads, &slabs);
    const dim3 grid((g.rows + dev::kPackRows - 1) / dev::kPackRows, slabs);
    return aligned ? launch<true>(dev::k_loss_pack<true>, grid, threads, 0, 1, s, g)
                   : launch<true>(dev::k_loss_pack<false>, grid, threads, 0, 1, s, g);
}

// The values of g that are there at a time: 256 MB (above 2^19 tokens, which pass that with 256 columns: 256 columns).
constexpr uint64_t kGradValues = 1ull << 27;
constexpr uint64_t kPackValues = 1ull << 26;  // of W, where its rows have to be moved to 16-byte boundaries
// The tiles' maxima and sums, 8 bytes a token and 64 columns, within 256 MB: of so many tokens at most, fewer where the
// vocabulary is large (262,144 rows: 8192), but at no fewer than 2048, with fewer rows at a time (above 2^20) instead: each
// product of the forward pass reads its part of W once.
constexpr uint64_t kMergeChunk = 32768, kMergeLeast = 2048, kMergeParts = 1ull << 25;

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// Parts of the depth of dx's product, at most, so that few tokens still give every pair work (parts_of chooses): within
// 256 MB, where one of float32 [tokens, cols] is not more.  They are reserved whatever parts_of, which knows the
// tokens that have a target, will use (1000 x 10,007 x 1024: 64 of 4 MB, of which 4 to 10 are).
int dx_splits(uint64_t tokens, uint64_t cols)
{
    const uint64_t room = (1ull << 28) / std::max<uint64_t>(1, 4 * tokens * up(cols, 8));
    return static_cast<int>(std::max<uint64_t>(1, std::min<uint64_t>(64, room)));
}

// Where things are in d_work.  What lives from piece to piece comes first, and
// does not depend on a piece's size.
struct Layout {
    uint64_t bytes = 0;
    uint64_t take(uint64_t n)
    {
        const uint64_t at = bytes;
        bytes += up(n, 256);
        return at;
    }
};
struct ForwardLayout : Layout {
    uint64_t head, state, mine, sums, counts, x, part, w;
    uint64_t ld, chunk, piece;  // rows of packed matrices; tokens of a product; rows of W that are moved at a time
    ForwardLayout(uint64_t tokens, uint64_t cols, uint64_t rows, bool move)
    {
        ld = up(cols, 64);  // whole lines of 128 bytes: boxes of others touch two
        piece = move ? std::min(rows, std::max<uint64_t>(256, kPackValues / ld / 256 * 256)) : rows;
        chunk = std::min(tokens, kMergeChunk);
        const auto units_of = [](uint64_t n) { return up(n, dev::kUnit) / dev::kUnit; };
        // (what is reserved does not fall where rows grow: a smaller piece has to find room in a larger one's)
        const uint64_t parts = std::min(kMergeParts, chunk * units_of(piece));
        if (chunk * units_of(piece) > kMergeParts)
            chunk = std::min(chunk, std::max(kMergeLeast, kMergeParts / units_of(piece) / 256 * 256));
        if (chunk * units_of(piece) > kMergeParts) piece = kMergeParts / chunk * dev::kUnit / 256 * 256;
        const uint64_t blocks = up(tokens, dev::kMergeTokens) / dev::kMergeTokens;
        head = take(16);
        state = take(8 * tokens);
        mine = take(4 * tokens);
        sums = take(8 * blocks);
        counts = take(4 * blocks);
        x = take(move ? 2 * tokens * ld : 0);
        part = take(8 * (is_few(tokens, cols) ? std::max(parts, chunk * few_blocks(piece)) : parts));
        w = take(move ? 2 * piece * ld : 0);
    }
};
struct BackwardLayout : Layout {
    uint64_t head, key[2], order[2], first, lse, share, coef, x, extra, part, target, g, sums, w;
    uint64_t ld, ldf, piece, ld_g;  // rows of packed BF16 and of float32 matrices, rows of W at a time, rows of g
    int splits, depth;
    BackwardLayout(uint64_t tokens, uint64_t vocab, uint64_t cols, uint64_t rows, bool weight, bool move, bool pieces)
    {
        ld = up(cols, 64);
        ldf = up(cols, 8);
        splits = dx_splits(tokens, cols);
        uint64_t most = std::max<uint64_t>(256, kGradValues / std::max<uint64_t>(1, up(tokens, 256)) / 256 * 256);
        depth = static_cast<int>(up(std::min(vocab, most), dev::kDepth) / dev::kDepth);
        if (move) most = std::min(most, std::max<uint64_t>(256, kPackValues / ld / 256 * 256));
        piece = std::min(rows, most);
        ld_g = up(piece, 64);
        head = take(16);
        for (int i = 0; i < 2; ++i) {
            key[i] = take(4 * tokens);
            order[i] = take(4 * tokens);
        }
        first = take(weight ? 4 * vocab : 0);
        lse = take(4 * tokens);
        share = take(4 * tokens);
        coef = take(4 * tokens);
        x = take(2 * tokens * ld);
        extra = take(weight ? 4 * tokens * ldf : 0);
        part = take(4 * static_cast<uint64_t>(splits) * tokens * ldf);
        target = take(pieces ? 2 * tokens * ld : 0);
        // g takes the place of the partial sums of the targets' terms, which come before it
        g = take(std::max(2 * tokens * ld_g,
                          weight ? 8 * (up(tokens, LCT_EMBEDDING_CHUNK(tokens)) / LCT_EMBEDDING_CHUNK(tokens)) * LCT_EMBEDDING_PART(cols) : 0));
        w = take(move ? 2 * piece * ld : 0);
    }
};

// What both directions check.
lct_status check_batch(const lct_ids *ids, const uint16_t *d_x, uint64_t ld_x, uint64_t cols, const uint16_t *d_w,
                       uint64_t ld_w, uint64_t first, uint64_t rows, const void *d_work, Matrix *x, Matrix *w)
{
    const lct_status rc = check_ids(ids);
    if (rc != LCT_OK) return rc;
    if (cols == 0 || rows == 0 || first > ids->vocab || rows > ids->vocab - first) return LCT_ERR_INVALID_ARG;
    if (cols > LCT_VOCAB_MAX_COLS) return LCT_ERR_UNSUPPORTED;
    *x = Matrix{d_x, ld_x, cols, ids->tokens, 2};
    *w = Matrix{d_w, ld_w, cols, rows, 2};
    if (!matrix_ok(*x) || !matrix_ok(*w) || !d_work || reinterpret_cast<uintptr_t>(d_work) % 256) return LCT_ERR_INVALID_ARG;
    return LCT_OK;
}

template <typename T>
T *at(void *work, uint64_t offset)
{
    return reinterpret_cast<T *>(static_cast<char *>(work) + offset);
}
const __nv_bfloat16 *bf16(const uint16_t *p) { return reinterpret_cast<const __nv_bfloat16 *>(p); }
__nv_bfloat16 *bf16(uint16_t *p) { return reinterpret_cast<__nv_bfloat16 *>(p); }

}  // namespace
}  // namespace lct

using namespace lct;

extern "C" uint64_t lct_loss_work_bytes(uint64_t tokens, uint64_t vocab, uint64_t cols, uint64_t rows, int32_t flags)
{
    // of what the calls refuse, nothing is worked out
    if (!cols || cols > LCT_VOCAB_MAX_COLS || tokens > LCT_VOCAB_MAX_TOKENS || vocab > LCT_VOCAB_MAX || rows > vocab) return 0;
    const bool move = flags & LCT_LOSS_UNALIGNED;
    if (flags & LCT_LOSS_BACKWARD)
        return BackwardLayout(tokens, vocab, cols, rows, flags & LCT_LOSS_WEIGHT, move, rows < vocab).bytes;
    return ForwardLayout(tokens, cols, rows, move && !is_few(tokens, cols)).bytes;
}

namespace {

lct_status forward(const lct_ids *targets, const uint16_t *d_x, uint64_t ld_x, uint64_t cols, const uint16_t *d_w,
                   uint64_t ld_w, uint64_t first, uint64_t rows, float *d_loss, float *d_lse, float *d_total, void *d_work,
                   uint64_t work_bytes, bool stalled, void *stream)
{
    Matrix x, w;
    const lct_status ok = check_batch(targets, d_x, ld_x, cols, d_w, ld_w, first, rows, d_work, &x, &w);
    if (ok != LCT_OK) return ok;
    const uint64_t t = targets->tokens, id_size = targets->wide ? 8 : 4;
    const bool by_few = !stalled && is_few(t, cols), w_al = matrix_al(w) && cols % 8 == 0;
    const bool move = !by_few && (!matrix_al(x) || !matrix_al(w)), begins = first == 0, ends = first + rows == targets->vocab;
    const ForwardLayout l(t, cols, rows, move);
    if (work_bytes < l.bytes || (t && (!d_loss || !d_lse)) || reinterpret_cast<uintptr_t>(d_loss) % 4 ||
        reinterpret_cast<uintptr_t>(d_lse) % 4 || reinterpret_cast<uintptr_t>(d_total) % 4)
        return LCT_ERR_INVALID_ARG;
    const struct {
        const void *p;
        uint64_t n;
    } out[4] = {{d_loss, 4 * t}, {d_lse, 4 * t}, {d_total, 12}, {d_work, l.bytes}};
    for (int i = 0; i < 4; ++i) {
        if (!apart(x, out[i].p, out[i].n) || !apart(w, out[i].p, out[i].n) ||
            !apart(targets->d_ids, t * id_size, out[i].p, out[i].n))
            return LCT_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (!apart(out[i].p, out[i].n, out[j].p, out[j].n)) return LCT_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (t == 0) {
        if (!d_total || !ends) return LCT_OK;
        // sum and mean of no losses; nobody has a share
        return cudaMemsetAsync(d_total, 0, 12, s) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
    }
    const __nv_bfloat16 *xp = bf16(d_x);
    uint64_t ldx = ld_x;
    if (move && !matrix_al(x)) {
        xp = at<__nv_bfloat16>(d_work, l.x);
        ldx = l.ld;
        if (begins) {
            PackArgs p{};
            p.src = bf16(d_x);
            p.ld_src = static_cast<int64_t>(ld_x);
            p.dst = at<__nv_bfloat16>(d_work, l.x);
            p.ld_dst = static_cast<int64_t>(l.ld);
            p.rows = static_cast<int32_t>(t);
            p.cols = static_cast<int32_t>(cols);
            if (pack(p, false, s) != cudaSuccess) return LCT_ERR_CUDA;
        }
    }
    for (uint64_t r0 = 0; r0 < rows; r0 += l.piece) {
        const uint64_t n = std::min(l.piece, rows - r0);
        const __nv_bfloat16 *wp = bf16(d_w) + r0 * ld_w;
        uint64_t ldw = ld_w;
        if (move && !matrix_al(w)) {
            PackArgs p{};
            p.src = wp;
            p.ld_src = static_cast<int64_t>(ld_w);
            p.dst = at<__nv_bfloat16>(d_work, l.w);
            p.ld_dst = static_cast<int64_t>(l.ld);
            p.rows = static_cast<int32_t>(n);
            p.cols = static_cast<int32_t>(cols);
            if (pack(p, false, s) != cudaSuccess) return LCT_ERR_CUDA;
            wp = p.dst;
            ldw = l.ld;
        }
        for (uint64_t t0 = 0; t0 < t; t0 += l.chunk) {
            const uint64_t tn = std::min(l.chunk, t - t0);
            const void *ids = static_cast<const char *>(targets->d_ids) + t0 * id_size;
            ProductArgs g{};
            g.m = static_cast<int32_t>(tn);
            g.n = static_cast<int32_t>(n);
            g.k = static_cast<int32_t>(cols);
            g.status = at<int32_t>(d_work, l.head);
            g.stalled = stalled;
            g.splits = 1;
            g.begins = begins && r0 == 0 && t0 == 0;
            g.ids = ids;
            g.wide = targets->wide;
            g.row0 = static_cast<int64_t>(first + r0);
            g.part = at<float2>(d_work, l.part);
            g.mine = at<float>(d_work, l.mine) + t0;
            if (by_few) {
                const FewArgs f{xp, wp, static_cast<int64_t>(ldx), static_cast<int64_t>(ldw)};
                if (few(g, f, w_al, s) != cudaSuccess) return LCT_ERR_CUDA;
            } else {
                ProductMaps maps{};
                g.a_rows = a_rows(tn);
                g.sum_steps = static_cast<int32_t>(sum_steps(t));
                if (!box_map(&maps.a, xp + t0 * ldx, cols, tn, ldx, 0, g.a_rows) ||
                    !box_map(&maps.b, wp, cols, n, ldw, 0, dev::kHalfTile) || product<kLogits>(g, maps, s) != cudaSuccess)
                    return LCT_ERR_CUDA;
            }
            MergeArgs m{};
            m.part = g.part;
            m.state = at<float2>(d_work, l.state) + t0;
            m.mine = g.mine;
            m.ids = ids;
            m.wide = targets->wide;
            m.loss = d_loss + t0;
            m.lse = d_lse + t0;
            m.total = d_total;
            m.sums = at<double>(d_work, l.sums);
            m.counts = at<int32_t>(d_work, l.counts);
            m.status = g.status;
            m.counter = g.status + 1;
            m.tokens = static_cast<int64_t>(tn);
            m.vocab = static_cast<int64_t>(targets->vocab);
            m.slots = by_few ? static_cast<int32_t>(few_blocks(n)) : static_cast<int32_t>(up(n, dev::kUnit) / dev::kUnit);
            m.blocks = static_cast<int32_t>(up(t, dev::kMergeTokens) / dev::kMergeTokens);
            m.block0 = static_cast<int32_t>(t0 / dev::kMergeTokens);
            m.begins = begins && r0 == 0;
            m.ends = ends && r0 + n == rows;
            if (launch<true>(dev::k_loss_merge, dim3(static_cast<uint32_t>(up(tn, dev::kMergeTokens) / dev::kMergeTokens)), 1024,
                             0, 1, s, m) != cudaSuccess)
                return LCT_ERR_CUDA;
        }
    }
    return LCT_OK;
}

lct_status backward(const lct_ids *targets, const uint16_t *d_x, uint64_t ld_x, uint64_t cols, const uint16_t *d_w,
                    uint64_t ld_w, uint64_t first, uint64_t rows, const float *d_loss, const float *d_lse,
                    const float *d_dloss, uint64_t dloss_stride, const float *d_scale, uint16_t *d_dx, uint64_t ld_dx,
                    uint16_t *d_dw, uint64_t ld_dw, void *d_work, uint64_t work_bytes, bool stalled, void *stream)
{
    Matrix x, w;
    const lct_status ok = check_batch(targets, d_x, ld_x, cols, d_w, ld_w, first, rows, d_work, &x, &w);
    if (ok != LCT_OK) return ok;
    const uint64_t t = targets->tokens, v = targets->vocab, id_bytes = t * (targets->wide ? 8 : 4);
    const bool move = !matrix_al(x) || !matrix_al(w), begins = first == 0, ends = first + rows == v, pieces = rows < v;
    const BackwardLayout l(t, v, cols, rows, d_dw != nullptr, move, pieces);
    const Matrix dx{d_dx, ld_dx, cols, t, 2}, dw{d_dw, ld_dw, cols, d_dw ? rows : 0, 2};
    if (work_bytes < l.bytes || !matrix_ok(dx) || !matrix_ok(dw) || dloss_stride > 1) return LCT_ERR_INVALID_ARG;
    if (t && (!d_loss || !d_lse || !d_dloss)) return LCT_ERR_INVALID_ARG;
    const struct {
        const void *p;
        uint64_t n;
    } in[5] = {{targets->d_ids, id_bytes},
               {d_loss, 4 * t},
               {d_lse, 4 * t},
               {d_dloss, t ? 4 * ((t - 1) * dloss_stride + 1) : 0},
               {d_scale, 4}};
    for (int i = 1; i < 5; ++i)
        if (reinterpret_cast<uintptr_t>(in[i].p) % 4) return LCT_ERR_INVALID_ARG;
    if (!apart(dx, x) || !apart(dx, w) || !apart(dw, x) || !apart(dw, w) || !apart(dx, dw) || !apart(dx, d_work, l.bytes) ||
        !apart(dw, d_work, l.bytes) || !apart(x, d_work, l.bytes) || !apart(w, d_work, l.bytes))
        return LCT_ERR_INVALID_ARG;
    for (const auto &r : in)
        if (!apart(dx, r.p, r.n) || !apart(dw, r.p, r.n) || !apart(d_work, l.bytes, r.p, r.n)) return LCT_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (t == 0) {
        if (!d_dw) return LCT_OK;
        return cudaMemset2DAsync(d_dw, 2 * ld_dw, 0, 2 * cols, rows, s) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
    }
    int32_t *status = at<int32_t>(d_work, l.head), *count = status + 2;
    int32_t *key = at<int32_t>(d_work, l.key[0]), *order = at<int32_t>(d_work, l.order[0]);
    __nv_bfloat16 *xp = at<__nv_bfloat16>(d_work, l.x);
    const int64_t ld = static_cast<int64_t>(l.ld), ldf = static_cast<int64_t>(l.ldf);
    const int32_t tokens = static_cast<int32_t>(t), k = static_cast<int32_t>(cols);
    if (begins) {
        SortArgs o{};
        o.ids = targets->d_ids;
        o.wide = targets->wide;
        for (int i = 0; i < 2; ++i) {
            o.key[i] = at<int32_t>(d_work, l.key[i]);
            o.order[i] = at<int32_t>(d_work, l.order[i]);
        }
        int32_t *sums = at<int32_t>(d_work, l.first);
        if (d_dw) {  // no row of the vocabulary has a sum yet
            const int64_t all = static_cast<int64_t>(4 * v);
            o.fill.out = sums;
            o.fill.value = 0xFFFFFFFFu;
            o.fill.bytes = o.fill.ld_out = 4096;
            o.fill.rows = o.fill.early = (all + 4095) / 4096;
            o.fill.last = all - (o.fill.rows - 1) * 4096;
        }
        o.count = count;
        o.clear = status;
        o.tokens = tokens;
        o.vocab = static_cast<int32_t>(v);
        if (launch_sort_ids(o, s) != cudaSuccess) return LCT_ERR_CUDA;
        PackArgs p{};
        p.src = bf16(d_x);
        p.ld_src = static_cast<int64_t>(ld_x);
        p.dst = xp;
        p.ld_dst = ld;
        p.order = order;
        p.count = count;
        p.dloss = d_dloss;
        p.dloss_stride = static_cast<int64_t>(dloss_stride);
        p.scale = d_scale;
        p.loss = d_loss;
        p.lse = d_lse;
        p.lse_out = at<float>(d_work, l.lse);
        p.share_out = at<float>(d_work, l.share);
        p.coef_out = at<float>(d_work, l.coef);
        p.rows = tokens;
        p.cols = k;
        if (pack(p, matrix_al(x) && cols % 8 == 0, s) != cudaSuccess) return LCT_ERR_CUDA;
        if (d_dw) {
            SegmentArgs e{};
            e.src = xp;
            e.ld_src = ld;
            e.key = key;
            e.first = sums;
            e.count = count;
            e.coef = p.coef_out;
            e.out = at<float>(d_work, l.extra);
            e.ld_out = ldf;
            e.part = at<float>(d_work, l.g);
            e.scale = 1.0f;
            e.cols = k;
            e.tokens = tokens;
            e.compact = true;
            if (launch_segments(e, false, cols % 8 == 0, s) != cudaSuccess) return LCT_ERR_CUDA;
        }
    }
    if (pieces) {  // the targets' rows, as their pieces come
        LookupArgs u{};
        u.ids = key;
        u.table = d_w;
        u.out = at<__nv_bfloat16>(d_work, l.target);
        u.ld_table = static_cast<int64_t>(ld_w);
        u.ld_out = ld;
        u.row0 = static_cast<int64_t>(first);
        u.rows = static_cast<int64_t>(rows);
        u.vocab = static_cast<int64_t>(v);
        u.tokens = static_cast<int64_t>(t);
        u.cols = k;
        u.scale = 1.0f;
        if (launch_lookup(u, false, matrix_al(w) && cols % 8 == 0, s) != cudaSuccess) return LCT_ERR_CUDA;
    }
    const bool dw_boxes = matrix_al(dw);
    int pairs;
    if (pairs_at_once<kDx>(&pairs) != cudaSuccess) return LCT_ERR_CUDA;
    for (uint64_t r0 = 0; r0 < rows; r0 += l.piece) {
        const uint64_t n = std::min(l.piece, rows - r0);
        const __nv_bfloat16 *wp = bf16(d_w) + r0 * ld_w;
        uint64_t ldw = ld_w;
        if (!matrix_al(w)) {
            PackArgs p{};
            p.src = wp;
            p.ld_src = static_cast<int64_t>(ld_w);
            p.dst = at<__nv_bfloat16>(d_work, l.w);
            p.ld_dst = ld;
            p.rows = static_cast<int32_t>(n);
            p.cols = k;
            if (pack(p, false, s) != cudaSuccess) return LCT_ERR_CUDA;
            wp = p.dst;
            ldw = l.ld;
        }
        __nv_bfloat16 *gp = at<__nv_bfloat16>(d_work, l.g);
        ProductMaps maps{};
        ProductArgs g{};
        g.m = tokens;
        g.n = static_cast<int32_t>(n);
        g.k = k;
        g.count = count;
        g.status = status;
        g.stalled = stalled;
        g.splits = 1;
        g.row0 = static_cast<int64_t>(first + r0);
        g.target = key;
        g.lse = at<float>(d_work, l.lse);
        g.share = at<float>(d_work, l.share);
        g.boxes = true;
        g.a_rows = a_rows(t);
        if (!box_map(&maps.a, xp, cols, t, l.ld, 0, g.a_rows) || !box_map(&maps.b, wp, cols, n, ldw, 0, dev::kHalfTile) ||
            !box_map(&maps.c, gp, n, t, l.ld_g, 0, 32) || product<kSoftmax>(g, maps, s) != cudaSuccess)
            return LCT_ERR_CUDA;
        g.n = k;
        g.k = static_cast<int32_t>(n);
        g.splits = l.splits;
        g.depth = l.depth;
        g.pairs = pairs;
        g.add = !(begins && r0 == 0);
        if (!box_map(&maps.a, gp, n, t, l.ld_g, 0, g.a_rows) || !box_map(&maps.b, wp, cols, n, ldw, 0, dev::kDepth) ||
            !box_map32(&maps.c, at<float>(d_work, l.part), cols, t, l.ldf, l.splits) ||
            product<kDx>(g, maps, s) != cudaSuccess)
            return LCT_ERR_CUDA;
        if (!d_dw) continue;
        g.m = static_cast<int32_t>(n);
        g.k = tokens;
        g.splits = 1;
        g.extra = at<float>(d_work, l.extra);
        g.first = at<int32_t>(d_work, l.first);
        g.ld_extra = ldf;
        g.out = bf16(d_dw) + r0 * ld_dw;
        g.ld_out = static_cast<int64_t>(ld_dw);
        g.boxes = dw_boxes;
        if (!box_map(&maps.a, gp, n, t, l.ld_g, 0, dev::kDepth) || !box_map(&maps.b, xp, cols, t, l.ld, 0, dev::kDepth) ||
            (dw_boxes && !box_map(&maps.c, g.out, cols, n, ld_dw, 0, 32)) || product<kDw>(g, maps, s) != cudaSuccess)
            return LCT_ERR_CUDA;
    }
    if (!ends) return LCT_OK;
    FinishArgs f{};
    f.part = at<float>(d_work, l.part);
    f.ld_part = ldf;
    f.tokens = static_cast<int64_t>(t);
    f.splits = l.splits;
    f.depth = l.depth;
    f.pairs = pairs;
    f.key = key;
    f.order = order;
    f.count = count;
    f.status = status;
    f.coef = at<float>(d_work, l.coef);
    f.w = pieces ? at<__nv_bfloat16>(d_work, l.target) : bf16(d_w);
    f.ld_w = pieces ? ld : static_cast<int64_t>(ld_w);
    f.gathered = pieces;
    f.ids = targets->d_ids;
    f.wide = targets->wide;
    f.dx = bf16(d_dx);
    f.ld_dx = static_cast<int64_t>(ld_dx);
    f.cols = k;
    const bool al = cols % 8 == 0 && matrix_al(dx) && (pieces || matrix_al(w));
    uint32_t threads, slabs;
    row_shape(k, 8, al, &threads, &slabs);
    const dim3 grid((tokens + dev::kFinishRows - 1) / dev::kFinishRows, slabs);
    const auto kernel = f.splits > 1 ? (al ? dev::k_loss_finish<true, true> : dev::k_loss_finish<false, true>)
                                     : (al ? dev::k_loss_finish<true, false> : dev::k_loss_finish<false, false>);
    const cudaError_t rc = launch<true>(kernel, grid, threads, 0, 1, s, f);
    return rc == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
}

}  // namespace

#define LOSS_FORWARD(name, stalled)                                                                                     \
    extern "C" lct_status name(const lct_ids *targets, const uint16_t *d_x, uint64_t ld_x, uint64_t cols,               \
                               const uint16_t *d_w, uint64_t ld_w, uint64_t first, uint64_t rows, float *d_loss,        \
                               float *d_lse, float *d_total, void *d_work, uint64_t work_bytes, void *stream)           \
    {                                                                                                                   \
        return forward(targets, d_x, ld_x, cols, d_w, ld_w, first, rows, d_loss, d_lse, d_total, d_work, work_bytes,    \
                       stalled, stream);                                                                                \
    }
#define LOSS_BACKWARD(name, stalled)                                                                                    \
    extern "C" lct_status name(const lct_ids *targets, const uint16_t *d_x, uint64_t ld_x, uint64_t cols,               \
                               const uint16_t *d_w, uint64_t ld_w, uint64_t first, uint64_t rows, const float *d_loss,  \
                               const float *d_lse, const float *d_dloss, uint64_t dloss_stride, const float *d_scale,   \
                               uint16_t *d_dx, uint64_t ld_dx, uint16_t *d_dw, uint64_t ld_dw, void *d_work,            \
                               uint64_t work_bytes, void *stream)                                                       \
    {                                                                                                                   \
        return backward(targets, d_x, ld_x, cols, d_w, ld_w, first, rows, d_loss, d_lse, d_dloss, dloss_stride, d_scale, \
                        d_dx, ld_dx, d_dw, ld_dw, d_work, work_bytes, stalled, stream);                                 \
    }
LOSS_FORWARD(lct_loss_forward, false)
LOSS_BACKWARD(lct_loss_backward, false)
LOSS_FORWARD(lct_debug_loss_forward_timeout, true)
LOSS_BACKWARD(lct_debug_loss_backward_timeout, true)
