// Library-private declarations shared by the host entry points and the CUDA
// kernels of liblct.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/lct.h"

namespace lct {

constexpr int kStreams = LCT_STREAMS;
constexpr uint64_t kMaxN = 1ull << 40;
constexpr uint64_t kDefaultWaitNs = 1000000000ull;  // 1 s bound on any device wait

struct Geometry {
    uint32_t block;       // exponents per block
    uint32_t slot_words;  // 32-bit words per stream slot
};

// [EXP] "Compressing is easy": 65,536-value blocks in CLEAN, 32,768 in MEDIUM
// and HIGH.  Slot sizes: 800 bits in CLEAN (the 1.4382x bound of [EXP] "Here
// is the idealized arithmetic"); 512 and 640 bits in MEDIUM and HIGH.
inline bool level_geometry(int level, Geometry *g)
{
    switch (level) {
    case LCT_LEVEL_CLEAN: *g = {65536u, 25u}; return true;
    case LCT_LEVEL_MEDIUM: *g = {32768u, 16u}; return true;
    case LCT_LEVEL_HIGH: *g = {32768u, 20u}; return true;
    default: return false;
    }
}

uint32_t codebook_hash(const lct_codebook &cb);
bool codebook_valid(const lct_codebook &cb);

// The codebook as kernels receive it (by value, in kernel parameters).
struct DevCodebook {
    uint8_t len[256];
    uint8_t code[256];
    uint16_t dec[256];
    uint8_t esc_len;
    uint8_t esc_code;
    uint8_t zero_atom;  // exponent 0 <-> symbol 0, unshifted
    uint8_t pad;
    uint32_t hash;
};

// Device view of one compressed tensor.
struct DevTensor {
    lct_header *hdr;
    uint8_t *sf;
    uint32_t *slots;
    uint16_t *markers;
    uint64_t *blk_off;
    uint8_t *ovf;
    unsigned long long *work;  // per-block scan status words
    uint64_t ovf_cap;
    uint64_t n;
    uint32_t nblocks;
    int32_t level;
};

// Every argument block carries two multipliers, 32 and 4, that the decoders
// use for address arithmetic: as launch arguments they are not compile-time
// constants, so the multiply-adds stay on the FMA pipe instead of becoming
// shifts on the integer ALU pipe.
struct EncodeArgs {
    const uint16_t *x;
    DevTensor t;
    DevCodebook cb;
    int32_t median_exp;
    uint32_t pad;
    uint64_t wait_ns;
    uint32_t mul_row, mul_ent, mul_sf, pad_mul;  // 32, 4 and 0x01010000 (set_multipliers)
    uint32_t deferred, pad_def;  // block offsets computed after the writer (set by its launcher)
};

struct DecodeArgs {
    DevTensor t;
    uint16_t *y;          // value i of block first_block is y[i]
    DevCodebook cb;
    uint64_t wait_ns;
    uint32_t first_block;  // the launch decodes blocks first_block .. + grid size
    uint32_t pad;
    uint32_t mul_row, mul_ent, mul_sf, pad_mul;  // 32, 4 and 0x01010000 (set_multipliers)
    uint32_t deferred, pad_def;  // block offsets computed after the writer (set by its launcher)
};

// Weight updates of the fused one-pass kernel.
enum : uint32_t { OP_SGD = 0, OP_ADAMW = 1 };

struct UpdateArgs {
    DevTensor in[3];      // W, M, and V for AdamW
    DevTensor w_out;
    DevCodebook cb[3];
    float k[8];           // the step's constants (SGD: k[0] = eta)
    uint32_t op;          // OP_SGD or OP_ADAMW
    uint32_t nin;         // inputs used: 2 or 3
    uint32_t in_place;    // W_out's sign-fraction bytes are W_in's
    uint32_t pad;
    uint64_t wait_ns;
    uint32_t mul_row, mul_ent, mul_sf, pad_mul;  // 32, 4 and 0x01010000 (set_multipliers)
    uint32_t deferred, pad_def;  // block offsets computed after the writer (set by its launcher)
};

// Updates of the fused two-state kernel (two compressed tensors and a dense
// gradient in, both tensors out).
enum : uint32_t { OP2_MOMENTUM = 0, OP2_ADAM_MOMENTS = 1 };

struct MomentumArgs {
    DevTensor w_in, m_in, w_out, m_out;  // the two states (W and M, or AdamW's M and V)
    const uint16_t *g;  // dense BF16 gradient, n values
    DevCodebook cbw, cbm;
    float k[8];         // the step's constants (momentum: k[0] = eta, k[1] = mu)
    uint32_t op;        // OP2_MOMENTUM or OP2_ADAM_MOMENTS
    uint32_t in_place;  // an output shares its input's sign-fraction bytes
    uint64_t wait_ns;
    uint32_t mul_row, mul_ent, mul_sf, pad_mul;  // 32, 4 and 0x01010000 (set_multipliers)
    uint32_t deferred, pad_def;  // block offsets computed after the writer (set by its launcher)
};

template <typename Args>
inline void set_multipliers(Args &a)
{
    a.mul_row = 32;
    a.mul_ent = 4;
    a.mul_sf = 0x01010000u;
    a.pad_mul = 0;
    a.deferred = 0;
    a.pad_def = 0;
}

cudaError_t launch_encode(const EncodeArgs &a, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs &a, uint32_t nblocks, cudaStream_t s);
cudaError_t launch_update(const UpdateArgs &a, cudaStream_t s);
cudaError_t launch_momentum(const MomentumArgs &a, cudaStream_t s);
// Deferred placement (grids of at least four blocks per SM): a block with no
// overflow bytes publishes its count and leaves, blocks with bytes to place
// still wait for their exclusive prefix, and launch_block_offsets (after the
// writer) writes every block offset, ovf_used and the capacity check.
bool deferred_placement(uint32_t nblocks);
// Grids of at most two blocks per SM (the launch is latency-bound).
bool small_grid(uint32_t nblocks);
cudaError_t launch_block_offsets(const DevTensor &t, cudaStream_t s);
cudaError_t launch_block_offsets2(const DevTensor &t0, const DevTensor &t1, cudaStream_t s);  // same nblocks
cudaError_t launch_wait_probe(lct_header *hdr, unsigned long long *work, uint64_t wait_ns,
                              cudaStream_t s);


// Gradients of one norm or clipping call (host arrays of device addresses).
constexpr uint32_t kGradMaxParts = 608;  // partial sums, a double each; the clipping factor behind them
static_assert(8 * kGradMaxParts + 32 <= LCT_GRAD_WORK_BYTES, "");
struct GradArgs {
    const void *const *src;
    void *const *dst;  // NULL for a norm alone
    const uint64_t *n;
    const int32_t *dtype;
    uint64_t count;
    float max_norm;
    float *norm;   // device
    double *part;  // device, LCT_GRAD_WORK_BYTES
};
cudaError_t launch_grads(const GradArgs &a, bool clip, cudaStream_t s);

// The adapters' kernels.  `in` is x and `base`, `out` are y and the result
// (backward: dy, dx and the new dx).
struct AdapterArgs {
    const __nv_bfloat16 *a, *b;  // [adapters, rank, k], [adapters, n, rank]
    const float *scale;
    const int32_t *ranks;        // or NULL
    const int32_t *order, *starts;
    int32_t *tiles, *status;
    const __nv_bfloat16 *in, *base;
    __nv_bfloat16 *out;          // or NULL: no rows are wanted
    const __nv_bfloat16 *x;      // backward: the forward pass's x
    const float *kept;           // backward: its x A^T, [tokens, rank]
    float *keep;                 // forward: where to put that, or NULL
    __nv_bfloat16 *work;         // backward: s dy B and s x A^T as hi and lo, [2][tokens][2][rank16]
    __nv_bfloat16 *da, *db;
    int64_t ld_in, ld_base, ld_out, ld_x;
    int32_t adapters, rank, rank16, k, n, nin, nout, tokens, rows;
    bool al_a, al_b, al_in, al_base, al_out, al_x, al_db;  // rows begin at 16-byte boundaries
    bool sparse;                                            // backward: more adapters than tokens
    bool boxes_w;                                           // the weights come as boxes: set by the launcher
    bool stalled;                                           // a test: no products are made, so that waits run out
};
struct PlanArgs {
    const int32_t *index;
    int32_t *order, *starts, *tiles;
    int32_t tokens, adapters, rows;
};
cudaError_t launch_adapter(const AdapterArgs &a, bool back, cudaStream_t s);
cudaError_t launch_adapter_grad(const AdapterArgs &a, cudaStream_t s);
cudaError_t launch_adapter_plan(const PlanArgs &a, cudaStream_t s);

// A matrix of rows in memory, as a call gets it, with values of `size` bytes.
struct Matrix {
    const void *p;
    uint64_t ld, cols, rows, size;
};
inline uint64_t matrix_bytes(const Matrix &m) { return m.rows ? m.size * ((m.rows - 1) * m.ld + m.cols) : 0; }
// (Up to 2^24 rows: their extent is within 64 bits before it is compared.)
inline bool matrix_ok(const Matrix &m)
{
    return !m.rows || (m.p && reinterpret_cast<uintptr_t>(m.p) % m.size == 0 && m.ld >= m.cols && m.ld <= kMaxN &&
                       (m.rows - 1) * m.ld + m.cols <= kMaxN);
}
// Whether every row begins at a 16-byte boundary (and TMA's strides hold the distance between rows).
inline bool matrix_al(const Matrix &m)
{
    return !m.rows || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 &&
                       ((m.ld * m.size % 16 == 0 && m.ld < 1ull << 36) || m.rows == 1));
}
inline bool apart(const void *x, uint64_t xn, const void *p, uint64_t n)
{
    const uint64_t xl = reinterpret_cast<uint64_t>(x), pl = reinterpret_cast<uint64_t>(p);
    return !x || !p || !xn || !n || xl + xn <= pl || pl + n <= xl;
}
inline bool apart(const Matrix &m, const void *p, uint64_t n) { return apart(m.p, matrix_bytes(m), p, n); }
// Whether two matrices share no value: apart in memory, or column slices of rows with one stride that do not meet.
inline bool apart(const Matrix &x, const Matrix &y)
{
    if (!x.rows || !y.rows || apart(x.p, matrix_bytes(x), y.p, matrix_bytes(y))) return true;
    const uint64_t xl = reinterpret_cast<uint64_t>(x.p), yl = reinterpret_cast<uint64_t>(y.p), ld = x.ld * x.size;
    if (x.ld != y.ld || x.size != y.size || (xl ^ yl) % x.size) return false;
    const uint64_t d = yl >= xl ? (yl - xl) % ld : (ld - (xl - yl) % ld) % ld;
    return d >= x.cols * x.size && d + y.cols * y.size <= ld;
}

// Rows of a value, or of a base, the last `early` of them while ids are sorted.  In bytes.
struct FillArgs {
    void *out;                         // NULL: nothing
    const void *base;                  // or NULL
    int64_t rows, early, bytes, last;  // the last row may be shorter
    int64_t ld_out, ld_base;
    uint32_t value;
};
// Ids sorted: key and order [0] are the result, [1] scratch; how many are within the vocabulary.
struct SortArgs {
    const void *ids;
    int32_t *key[2], *order[2], *count;
    int32_t *clear;                    // two words that become zero, or NULL
    FillArgs fill;
    int32_t tokens, vocab, bits, passes;  // bits a pass and passes are set by the launcher
    bool wide;
};
struct LookupArgs {
    const void *ids, *table;
    void *out;
    int64_t ld_table, ld_out, row0, rows, vocab, tokens;  // the table's rows are row0 .. row0 + rows of vocab
    int32_t cols;
    float scale;
    bool wide;
};
// Sums of the rows of equal ids, in sorted order.
struct SegmentArgs {
    const void *src;          // row order[i] (NULL: row i) belongs to key[i]
    const int32_t *key, *order, *count;
    int32_t *first;           // compact: the row that is key's
    const float *coef;        // [i], or NULL: 1
    const void *base;         // or NULL
    void *out;                // row key[i]; compact: float32 rows, that of the key's first place
    float *part;              // [chunks][2][LCT_EMBEDDING_PART]
    int64_t ld_src, ld_base, ld_out;
    float scale;
    FillArgs fill;            // rows without tokens, or none
    int32_t cols, tokens;
    int32_t chunk, fill_rows; // set by the launcher, as are the next two
    uint32_t chunks, slabs;
    bool compact;
};
cudaError_t launch_sort_ids(SortArgs a, cudaStream_t s);
cudaError_t launch_lookup(const LookupArgs &a, bool wide, bool aligned, cudaStream_t s);  // wide: float32 values
cudaError_t launch_segments(const SegmentArgs &a, bool wide, bool aligned, cudaStream_t s);
lct_status check_ids(const lct_ids *ids);

}  // namespace lct
