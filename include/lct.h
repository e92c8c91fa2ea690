/*
 * lct.h -- C ABI of liblct.so: lossless BF16 tensor compression on the GPU
 * (exponent-Huffman coding with fixed-length streams) and the fused
 * compressed SGD step, for NVIDIA GB300 (sm_103a).
 *
 * The operations follow two pages describing LCT (Losslessly Compressed
 * Tensors), cited by title and paragraph:
 *   [ABS] "LCT: Losslessly Compressed Tensors with GPU friendly execution for
 *         Training" (Zhu, Sun, Lio, Yu), abstract page;
 *   [EXP] "LCT paper -- Lossless Huffman coding of BF16 training tensors --
 *         What does it mean?", explainer page; paragraphs are named by their
 *         opening words ("In bits", "Compressing is easy", "Training adds a
 *         second problem", "Here is the idealized arithmetic").
 *
 * Conventions shared by every entry point
 *   - Every function returns an lct_status and never throws.
 *   - The library never allocates device memory.  All device buffers are
 *     owned by the caller and named by plain device pointers ("d_" prefix);
 *     every other pointer is a host pointer.
 *   - GPU work is enqueued asynchronously on `stream` (a cudaStream_t passed
 *     as void*; NULL is the legacy default stream).  Nothing synchronises
 *     except lct_compressed_size() with a tensor.
 *   - Errors the host can see (NULL or misaligned pointers, size mismatches,
 *     bad levels, malformed codebooks, overlapping buffers) return at once
 *     and enqueue nothing.  Errors only the GPU can see (overflow capacity
 *     exceeded, corrupt stream data, an overflow-offset wait that ran out)
 *     are latched into the tensor's device header; read them back with
 *     lct_compressed_size().  Device-side checks never fault: every index
 *     into caller memory is bounds-checked and skipped on failure.
 *   - Device pointers must be 16-byte aligned.
 *   - Launches report CUDA launch errors as LCT_ERR_CUDA.
 */
#ifndef LCT_H
#define LCT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LCT_OK = 0,
    LCT_ERR_INVALID_ARG = 1,       /* host-side argument check failed */
    LCT_ERR_UNSUPPORTED = 2,       /* valid request the library does not implement */
    LCT_ERR_OVERFLOW_CAPACITY = 3, /* device: the overflow bytes did not fit d_ovf */
    LCT_ERR_CORRUPT = 4,           /* device: header, markers or offsets inconsistent */
    LCT_ERR_TIMEOUT = 5,           /* device: a wait for an earlier block's offset ran out */
    LCT_ERR_CUDA = 6               /* a CUDA runtime call failed */
} lct_status;

/* Exponent distribution models the user picks from ([EXP] "In bits"). */
typedef enum {
    LCT_MODEL_GAUSSIAN = 0, /* |x| half-normal, scale = sigma */
    LCT_MODEL_LAPLACE = 1,  /* |x| exponential, scale = b */
    LCT_MODEL_POWERLAW = 2  /* |x| Lomax (Pareto II), scale = s, shape = alpha */
} lct_model;

/* Block levels ([EXP] "Compressing is easy"): CLEAN blocks hold 65,536
 * exponents, MEDIUM and HIGH 32,768.  Each stream's slot is 800 bits in
 * CLEAN (3.125 bits/exponent; the pages' 1.4382x CLEAN bound,
 * [EXP] "Here is the idealized arithmetic"), 512 bits in MEDIUM and 640 bits
 * in HIGH (4 and 5 bits/exponent: sizes the pages do not print). */
typedef enum { LCT_LEVEL_CLEAN = 0, LCT_LEVEL_MEDIUM = 1, LCT_LEVEL_HIGH = 2 } lct_level;

#define LCT_STREAMS 256        /* streams per block, dealt round-robin */
#define LCT_MAX_CODE_BITS 8    /* code length cap ([EXP] "In bits") */
#define LCT_LITERAL_BITS 8     /* raw exponent after the escape prefix */
#define LCT_SHIFT_SAMPLES 4096 /* at most this many samples set the shift */
#define LCT_HEADER_BYTES 64
#define LCT_MAGIC 0x3154434Cu  /* "LCT1" */

/* A precomputed codebook ([EXP] "In bits": built ahead of time from the
 * chosen model, codes at most 8 bits, rare exponents under one escape prefix
 * followed by an 8-bit literal).  Plain host data, about 1 KB; it is copied
 * into kernel parameters on every call.
 *
 * Symbols are shifted exponents s = e - delta (delta from the tensor header).
 * Codes are canonical: ordered by (length, symbol), escape last among equal
 * lengths; code values are right-aligned in `len` bits, sent most significant
 * bit first. */
typedef struct {
    uint8_t len[256];     /* code length of symbol s (1..8), 0 = sent as escape */
    uint8_t code[256];    /* code of symbol s, right-aligned */
    uint16_t dec[256];    /* 8-bit window -> bits 0..8 symbol (256 = escape), bits 12..15 length */
    uint8_t esc_len;      /* escape prefix length (1..8) */
    uint8_t esc_code;     /* escape prefix, right-aligned */
    uint16_t nsym;        /* symbols with their own code */
    int32_t median_exp;   /* the model's median biased exponent (1..254) */
    int32_t model;        /* lct_model it was built from */
    uint32_t hash;        /* 32-bit FNV-1a of len, code, esc_len, esc_code, zero_atom */
    double scale, shape;  /* model parameters it was built from */
    double zero_frac;     /* point mass at zero it was built with (0 = none) */
    uint32_t zero_atom;   /* 1: exponent 0 always codes as symbol 0, unshifted;
                             a nonzero exponent the shift maps to symbol 0 escapes */
    uint32_t reserved;
} lct_codebook;

/* Device header, LCT_HEADER_BYTES at t->d_header.  Written by lct_encode and
 * lct_sgd_step_fused; read by lct_decode and lct_compressed_size. */
typedef struct {
    uint32_t magic;    /* LCT_MAGIC */
    uint32_t version;  /* 1 */
    uint64_t n;        /* BF16 values */
    int32_t level;     /* lct_level */
    int32_t delta;     /* scale shift: symbol = exponent - delta */
    uint32_t status;   /* first device-side error latched (an lct_status), 0 = none */
    uint32_t cb_hash;  /* codebook hash the streams were written with */
    uint64_t ovf_used; /* overflow bytes the last write needed (may exceed ovf_cap) */
    uint64_t ovf_cap;  /* capacity the last write was given */
    uint64_t reserved[2];
} lct_header;

/* A compressed tensor: caller-owned device regions (sizes from
 * lct_compressed_size).  Layout, with nblocks = ceil(n / block):
 *   d_sf       n bytes: sign in bit 7, fraction in bits 0..6, element order
 *              ([EXP] "In bits": the sign-fraction byte is stored as is);
 *   d_slots    nblocks * slot_words * 256 uint32, index [block][word][stream]:
 *              stream j of a block holds its positions i with i mod 256 = j
 *              ([EXP] "Compressing is easy": neighbours go to different
 *              streams), codes packed MSB-first from bit 31 of word 0, unused
 *              bits zero;
 *   d_markers  nblocks * 256 uint16: symbols held in each slot; the stream's
 *              later symbols are in the overflow (the spill-start marker);
 *   d_blk_off  nblocks + 1 uint64: exclusive prefix of the blocks' overflow
 *              byte counts; entry nblocks is the total;
 *   d_ovf      ovf_cap bytes: spilled exponents, uncompressed, in (block,
 *              stream, symbol) order; may be a slice of a buffer shared by
 *              many tensors ([EXP] "Here is the idealized arithmetic");
 *   d_work     work_bytes of scratch for the blocks' overflow-offset scan
 *              (not part of the compressed data; needed by writers only). */
typedef struct {
    uint64_t n;
    int32_t level;
    int32_t reserved;
    void *d_header;
    uint8_t *d_sf;
    uint32_t *d_slots;
    uint16_t *d_markers;
    uint64_t *d_blk_off;
    uint8_t *d_ovf;
    uint64_t ovf_cap;
    void *d_work;
} lct_tensor;

typedef struct {
    uint64_t n;
    uint64_t nblocks;
    uint32_t block;            /* exponents per block */
    uint32_t slot_words;       /* 32-bit words per stream slot */
    uint64_t header_bytes;
    uint64_t sf_bytes;
    uint64_t slot_bytes;
    uint64_t marker_bytes;
    uint64_t blk_off_bytes;
    uint64_t fixed_bytes;      /* header + sf + slots + markers + blk_off */
    uint64_t worst_ovf_bytes;  /* n: every exponent spilled */
    uint64_t work_bytes;       /* d_work scratch */
    /* filled only when a tensor is passed (after a stream synchronise) */
    uint64_t ovf_used;         /* overflow bytes the last write needed */
    uint32_t status;           /* latched device status (lct_status) */
    int32_t delta;             /* the tensor's scale shift */
} lct_sizes;

/* Build a codebook from a distribution model ([EXP] "In bits"; the paper's
 * "precomputed codebooks", [ABS]).  Host only, deterministic.
 *   model  lct_model; scale > 0 (sigma, b or s); shape = alpha > 0 for the
 *          power-law model, ignored otherwise.
 * Exponent bucket e holds |x| in [2^(e-127), 2^(e-126)) (e = 0: zeros and
 * subnormals; e = 254 open above; e = 255 weight 0).  Bucket masses are
 * scaled by 2^40 and rounded to integers; for k = 1..min(255, nonzero
 * buckets) the k heaviest buckets (ties: smaller exponent first) get codes
 * alongside an escape of the remaining weight (at least 1), lengths from
 * package-merge capped at 8 bits; the k with the least expected bits wins
 * (smallest k on a tie).  Errors: LCT_ERR_INVALID_ARG for a NULL `out` or
 * bad parameters. */
lct_status lct_codebook_build(int model, double scale, double shape, lct_codebook *out);

/* The same with a point mass at zero: a fraction zero_frac (0 <= zero_frac <
 * 1) of the values are exactly zero, as in ReLU/GELU activations, and the
 * rest follow the model.  Bucket masses are (1 - zero_frac) * p(e), plus
 * zero_frac at e = 0; the rest of the construction is lct_codebook_build's.
 * The pages note that the user supplies the distribution and that one which
 * does not fit the tensor raises storage ([EXP] "Read the 3.5x longer context
 * claim carefully"); zeros are a common misfit, since any shift moves them to
 * an unused symbol and they escape at 16 bits each.  The resulting codebook
 * has zero_atom = 1: exponent 0 (zeros and subnormals) always codes as symbol
 * 0 whatever the tensor's shift, and a nonzero exponent that the shift maps
 * onto symbol 0 is escaped.  The pages have no such model; its encoding is
 * decoded by lct_decode like any other.  Returns LCT_ERR_INVALID_ARG for bad
 * parameters. */
lct_status lct_codebook_build_zero_atom(int model, double scale, double shape, double zero_frac,
                                        lct_codebook *out);

/* Region sizes for an n-value tensor at `level`, and, when `t` is not NULL,
 * the state of a written tensor: synchronises `stream`, then reads the
 * device header into out->ovf_used / status / delta.
 * Compression ratio = 2n / (fixed_bytes + ovf_used).  Errors:
 * LCT_ERR_INVALID_ARG (NULL out, bad level, n > 2^40, t->n or t->level not
 * matching), LCT_ERR_CUDA. */
lct_status lct_compressed_size(uint64_t n, int level, const lct_tensor *t, void *stream,
                               lct_sizes *out);

/* Compress n BF16 values d_x (device, 16-byte aligned) into `t`
 * ([EXP] "In bits" and "Compressing is easy").  Enqueues:
 *   1. the scale shift: at most 4096 values sampled at floor(k*n/m); the lower
 *      median of their normal exponents (1..254) minus cb->median_exp,
 *      clamped to [-127, 127], 0 if none; written to the header;
 *   2. one pass per block: sign-fraction bytes out, each exponent coded as
 *      its symbol's code or escape + 8-bit raw exponent, packed into its
 *      stream's slot until the first code that does not fit (the marker);
 *      the rest of the stream spills to d_ovf; blocks' overflow offsets come
 *      from a single-pass scan over d_work.
 * If the overflow exceeds t->ovf_cap, blocks that do not fit write no
 * overflow bytes and LCT_ERR_OVERFLOW_CAPACITY is latched; header.ovf_used
 * tells the size needed.  d_x is not modified. */
lct_status lct_encode(const uint16_t *d_x, const lct_codebook *cb, const lct_tensor *t,
                      void *stream);

/* lct_encode for callers that cannot allocate device memory.  (The paper has
 * no counterpart: this is a convenience of this library.)
 *
 * lct_encode needs `t->d_work`, a little device scratch (8 bytes per block)
 * for the scan that places each block's overflow bytes.  Some callers cannot
 * allocate it: a caching allocator or out-of-memory handler that compresses
 * tensors to free space would have to re-enter the allocator, or fail for
 * lack of memory, to get scratch; other code must avoid cudaMalloc/cudaFree
 * because they can synchronise the device.  This variant allocates nothing:
 * its scratch is a fixed array of LCT_STATIC_SCRATCH_BLOCKS 8-byte words
 * (128 KiB) compiled into the library, which every GPU that loads the library
 * holds until the process exits.  `t->d_work` is ignored and may be NULL;
 * everything else is exactly as for lct_encode (same checks, same output,
 * bit for bit).
 *   - Tensors needing more than LCT_STATIC_SCRATCH_BLOCKS blocks (n above
 *     2^30 values in CLEAN, 2^29 in MEDIUM and HIGH) are rejected with
 *     LCT_ERR_UNSUPPORTED before anything is enqueued.
 *   - Every call looks up the array's device address on the current device
 *     (nothing is cached, so the address stays right after cudaDeviceReset).
 *     The first call on a device may load the library's device code there;
 *     make that first call before any stream capture.
 *   - All calls share the one array.  Each call clears the words it uses
 *     before using them, but calls whose GPU work overlaps -- on different
 *     streams, or from different threads -- race on the array and may produce
 *     wrong overflow offsets.  Serialise them.
 * Errors: as lct_encode, plus LCT_ERR_UNSUPPORTED (too large) and
 * LCT_ERR_CUDA (the device address could not be obtained). */
#define LCT_STATIC_SCRATCH_BLOCKS 16384
lct_status lct_encode_static_scratch(const uint16_t *d_x, const lct_codebook *cb, const lct_tensor *t,
                                     void *stream);

/* Reconstruct the n BF16 values of `t` into d_y (device, 16-byte aligned),
 * bit for bit ([EXP] "In bits": every value decodes exactly).  `cb` must be
 * the codebook the tensor was written with (checked on the device by hash).
 * Latches LCT_ERR_CORRUPT (bad magic, n, level or hash, a marker beyond its
 * stream, a slot whose codes run past it, offsets that disagree with the
 * markers) or LCT_ERR_OVERFLOW_CAPACITY (overflow never written); d_y is then
 * unspecified.  d_y must not overlap the tensor. */
lct_status lct_decode(const lct_tensor *t, const lct_codebook *cb, uint16_t *d_y, void *stream);

/* Decode only blocks first_block .. first_block + nblocks - 1 of `t` into d_y
 * (device, 16-byte aligned): value i of block first_block goes to d_y[i], so
 * d_y holds min(nblocks * block, n - first_block * block) values.  This is
 * the piece for decoding a compressed matmul operand tile by tile into a
 * small dense buffer that a GEMM reads ([EXP] "Read the 3.5x longer context
 * claim carefully": decoding inside matmul kernels is named as future work;
 * decoding a tile at a time ahead of a library GEMM keeps only one tile
 * dense).  Blocks are independent given the stored shift and offsets.
 * nblocks = 0 enqueues nothing.  Errors as lct_decode (latched in t's
 * header), plus LCT_ERR_INVALID_ARG for a range past the last block. */
lct_status lct_decode_blocks(const lct_tensor *t, const lct_codebook *cb, uint64_t first_block, uint64_t nblocks,
                             uint16_t *d_y, void *stream);

/* One fused SGD step W <- W - eta*M on compressed W and M ([EXP] "Training
 * adds a second problem": read the compressed inputs, compute, write the new
 * bytes in one pass).  Per value, in float32: p = round(eta*m),
 * r = round(w - p) (two roundings, no fused multiply-add), then BF16 by
 * round-to-nearest-even (subnormals kept, NaN -> 0x7FC0).  The new W is coded
 * with cbW and W_in's stored shift (the codebook stays fixed).
 * W_in, M and W_out must have the same n and level.  W_out may share
 * d_header, d_sf, d_slots, d_markers and d_blk_off with W_in (in-place
 * update) but its d_ovf and d_work must not overlap W_in's or M's overflow,
 * and W_out must not overlap M.  M is read only. */
lct_status lct_sgd_step_fused(const lct_tensor *W_in, const lct_codebook *cbW, const lct_tensor *M,
                              const lct_codebook *cbM, float eta, const lct_tensor *W_out,
                              void *stream);

/* One fused SGD-with-momentum step on compressed W and M with a dense BF16
 * gradient d_g (n values, 16-byte aligned):
 *   M' = bf16(round(round(mu*m) + g)),   W' = bf16(round(w - round(eta*M')))
 * The pages name the momentum buffer of SGD with momentum as optimizer state
 * that LCT keeps compressed ([EXP] "Jargon", entry "Optimizer state"; [ABS])
 * and ask for a single-pass update of compressed tensors ([EXP] "Training
 * adds a second problem"); they print no update rule, so this is the
 * heavy-ball form without dampening or Nesterov term.  Every float32 product
 * and sum is rounded on its own (no fused multiply-add); the weight step uses
 * M' as stored (BF16); rounding to BF16 is round-to-nearest-even with
 * subnormals kept and NaN -> 0x7FC0.  W' is coded with cbW and W_in's stored
 * shift, M' with cbM and M_in's stored shift.
 * All four tensors must have the same n and level.  Each output may share
 * d_header, d_sf, d_slots, d_markers and d_blk_off with its own input (in
 * place) but not partly overlap them; its d_ovf and d_work must be apart from
 * every input region; W' and M' must not overlap each other, W' must not
 * overlap M_in, M' must not overlap W_in, and d_g must not overlap either
 * output.  Each output latches its own status (capacity, corrupt input,
 * timeout); a corrupt input or a timeout is latched in both. */
lct_status lct_sgd_momentum_step_fused(const lct_tensor *W_in, const lct_codebook *cbW, const lct_tensor *M_in,
                                       const lct_codebook *cbM, const uint16_t *d_g, float eta, float mu,
                                       const lct_tensor *W_out, const lct_tensor *M_out, void *stream);

/* Hyper-parameters of one AdamW step (step >= 1 counts the steps taken,
 * this one included). */
typedef struct {
    double lr;
    double beta1, beta2;   /* in [0, 1) */
    double eps;            /* > 0 */
    double weight_decay;   /* decoupled: W <- W - lr*weight_decay*W */
    uint64_t step;
} lct_adamw_params;

/* One fused AdamW step on compressed W, M (first moment) and V (second
 * moment) with a dense BF16 gradient d_g (n values, 16-byte aligned).  The
 * pages name optimizer state -- buffers the size of the weights that the
 * optimizer keeps -- among the tensors LCT stores compressed ([EXP] "Jargon",
 * entry "Optimizer state"; [ABS]) and ask for updates that read and write
 * compressed tensors in one pass ([EXP] "Training adds a second problem");
 * they print no optimizer, so this is AdamW with decoupled weight decay.
 * With float constants rounded once from the parameters in double,
 *   b1 = beta1, c1 = 1 - beta1, b2 = beta2, c2 = 1 - beta2,
 *   a = lr / (1 - beta1^step), r = 1 / sqrt(1 - beta2^step), e = eps,
 *   d = lr * weight_decay,
 * every value is updated with each float32 operation rounded on its own (no
 * fused multiply-add; sqrt and division correctly rounded):
 *   M' = bf16(b1*m + c1*g)
 *   V' = bf16(b2*v + c2*(g*g))
 *   W' = bf16((w - d*w) - (a*M') / (sqrt(V')*r + e))
 * where the weight update takes M' and V' as stored (BF16); rounding to BF16
 * is round-to-nearest-even with subnormals kept and NaN -> 0x7FC0.  Each
 * output is coded with its input's codebook and stored shift.  Two passes:
 * one kernel writes M' and V', a second one W' (reading M' and V').
 * All six tensors must have the same n and level.  Each output may share
 * d_header, d_sf, d_slots, d_markers and d_blk_off with its own input (in
 * place) but not partly overlap them; its d_ovf and d_work must be apart from
 * every input region; an output must not overlap another output or another
 * tensor's input, and d_g must not overlap any output.  Each output latches
 * its own status; LCT_ERR_INVALID_ARG for bad parameters. */
lct_status lct_adamw_step_fused(const lct_tensor *W_in, const lct_codebook *cbW, const lct_tensor *M_in,
                                const lct_codebook *cbM, const lct_tensor *V_in, const lct_codebook *cbV,
                                const uint16_t *d_g, const lct_adamw_params *p, const lct_tensor *W_out,
                                const lct_tensor *M_out, const lct_tensor *V_out, void *stream);

/* ---- gradients of many tensors: their global norm, and clipping -------- */

typedef enum { LCT_DTYPE_BF16 = 0, LCT_DTYPE_F32 = 1 } lct_dtype;

#define LCT_GRAD_WORK_BYTES 4896 /* device scratch of the two calls below */

/* The global 2-norm of `count` gradients, *d_norm = sqrt(sum of g^2): the
 * dense gradients that the fused steps take, or any other list.  (The pages
 * have no counterpart.)  d_g, n and dtype are host arrays of `count` entries:
 * device address (aligned to its values, so slices of a bucket are fine),
 * values (0 is fine, the address is then not looked at) and lct_dtype, which
 * may differ between tensors.  They are read before the call returns.
 * d_work is LCT_GRAD_WORK_BYTES of scratch.  Partial sums are held in double
 * and added in a fixed order: the result does not change from run to run, no
 * square overflows or underflows, and only a norm above float's range is
 * returned as infinity.  A NaN or an infinity among the values gives NaN or
 * infinity.  count = 0 gives 0.
 * Errors: LCT_ERR_INVALID_ARG (NULL or misaligned pointers, n > 2^40, d_norm
 * or d_work over one another or over a gradient), LCT_ERR_UNSUPPORTED
 * (another dtype), LCT_ERR_CUDA. */
lct_status lct_grad_norm(const void *const *d_g, const uint64_t *n, const int32_t *dtype, uint64_t count,
                         float *d_norm, void *d_work, void *stream);

/* The same norm into *d_norm, and every gradient scaled by
 *   c = min(1, max_norm / (norm + 1e-6))
 * into d_out[i] (n[i] values of d_g[i]'s type, rounded once, to nearest even).
 * d_out[i] is d_g[i] itself (in place) or apart from every gradient and every
 * other output.  With c = 1 gradients in place are not touched.  A norm above
 * float's range, which *d_norm gives as infinity, still clips to max_norm.  c
 * is NaN where a gradient is NaN, and 0 where one is infinite (an infinity
 * times 0 is NaN, a finite value 0): read *d_norm before a step to skip it.
 * Errors: as lct_grad_norm, and LCT_ERR_INVALID_ARG for max_norm that is not
 * positive and finite, or for overlapping tensors (d_norm and d_work among
 * them). */
lct_status lct_grad_clip(const void *const *d_g, void *const *d_out, const uint64_t *n, const int32_t *dtype,
                         uint64_t count, float max_norm, float *d_norm, void *d_work, void *stream);

/* ---- low-rank adapters of many requests beside a shared projection ------ */

#define LCT_ADAPTER_TILE 128           /* tokens in a tile of a plan */
#define LCT_ADAPTER_MAX_RANK 128
#define LCT_ADAPTER_MAX 16384          /* adapters in a bank */
#define LCT_ADAPTER_MAX_TOKENS (1 << 24)
#define LCT_ADAPTER_MAX_COLS (1 << 20) /* columns of x and of y */
/* rows of a plan's tile table (at least one) */
#define LCT_ADAPTER_TILE_ROWS(tokens, adapters)                                                            \
    ((tokens) == 0 ? 1ull                                                                                  \
                   : ((uint64_t)(tokens) + LCT_ADAPTER_TILE - 1) / LCT_ADAPTER_TILE +                      \
                         ((uint64_t)(adapters) + 1 < (uint64_t)(tokens) ? (uint64_t)(adapters) + 1         \
                                                                        : (uint64_t)(tokens)))
/* scratch of lct_adapter_backward */
#define LCT_ADAPTER_WORK_BYTES(tokens, rank) (8ull * (tokens) * (((rank) + 15ull) / 16 * 16))

/* A bank of adapters for one projection of k to n columns (caller-owned
 * device memory, BF16, row-major): adapter a adds s_a (x A_a^T) B_a^T.  It uses
 * the first d_ranks[a] (clamped to 0..rank) rows of A_a and columns of B_a; the
 * others are not read.  d_ranks NULL: all of them. */
typedef struct {
    const uint16_t *d_a;     /* [adapters][rank][k] */
    const uint16_t *d_b;     /* [adapters][n][rank] */
    const float *d_scale;    /* [adapters] */
    const int32_t *d_ranks;  /* [adapters] or NULL */
    uint64_t adapters, rank, k, n;
} lct_adapters;

/* The grouping of a batch's tokens by adapter, from lct_adapter_plan: made
 * once for a batch and used for every projection in it.  Entries are checked
 * against `tokens` and `adapters` where they are used: tables that are not a
 * plan's reach nothing out of bounds, latch LCT_ERR_CORRUPT in the plan's
 * status where that shows, and give unspecified results. */
typedef struct {
    const int32_t *d_order;  /* [tokens]: tokens in stable order of their adapter, those without one last */
    const int32_t *d_starts; /* [adapters + 2]: where each adapter's tokens begin; without one; tokens */
    int32_t *d_tiles;        /* [LCT_ADAPTER_TILE_ROWS][4], 16-byte aligned: adapter (-1: none), first place
                                in the order, tokens (1..128, 0: unused row), 0; the first row's fourth
                                value is the plan's status (an lct_status) */
    uint64_t tokens, adapters;
} lct_token_plan;

/* Fill the three tables of a plan from each token's adapter, d_index[tokens]
 * (-1: none).  (The pages have no counterpart.)  An index outside -1 ..
 * adapters - 1 counts as none and latches LCT_ERR_INVALID_ARG in the plan's
 * status.  Errors: LCT_ERR_INVALID_ARG (NULL or misaligned pointers, no
 * adapters, overlapping tables), LCT_ERR_UNSUPPORTED (more adapters or tokens
 * than the limits above), LCT_ERR_CUDA. */
lct_status lct_adapter_plan(const int32_t *d_index, uint64_t tokens, uint64_t adapters, int32_t *d_order,
                            int32_t *d_starts, int32_t *d_tiles, void *stream);

/* out = y + s_a (x A_a^T) B_a^T for every token, out = y where it has no
 * adapter: what many requests' adapters add to y, the shared projection of
 * the same x.  x [tokens, k], y and out [tokens, n] are BF16 with rows ld_*
 * values apart; out may be y itself.  Rows that begin at 16-byte boundaries
 * are the fast case; of others whole aligned 16-byte pieces are fetched, what
 * lies before a row's first value among it.  The sums are float32, the narrow
 * product is carried to the second one with 16 bits, and out is rounded once.
 * d_xa, if not NULL, gets x A_a^T [tokens, rank] in float32 (0 where an adapter
 * has no such rank) for lct_adapter_backward.  Infinities and NaN in x stay in
 * their rows and follow the formula, whatever ranks an adapter leaves unused;
 * an infinite B_a (backward, for dx_out: A_a) may give NaN where the formula
 * gives an infinity, as the narrow product's two parts may have opposite signs.
 * A wait that ran out on the device latches LCT_ERR_TIMEOUT in the plan's
 * status.  Errors: LCT_ERR_INVALID_ARG (NULL or misaligned pointers, strides
 * below the widths, a plan for another number of adapters, an output that
 * overlaps another operand), LCT_ERR_UNSUPPORTED (rank above
 * LCT_ADAPTER_MAX_RANK or another limit), LCT_ERR_CUDA. */
lct_status lct_adapter_forward(const lct_adapters *bank, const lct_token_plan *plan, const uint16_t *d_x,
                               uint64_t ld_x, const uint16_t *d_y, uint64_t ld_y, uint16_t *d_out, uint64_t ld_out,
                               float *d_xa, void *stream);

/* The gradients of lct_adapter_forward for dy, the gradient of out (which is
 * also that of y): with d = s_a dy B_a,
 *   dx_out = dx + d A_a        (dx: the shared projection's part; dx_out may be dx itself)
 *   dA_a = sum over a's tokens of d^T x
 *   dB_a = sum over a's tokens of s_a dy^T (x A_a^T)
 * in BF16, each rounded once; gradients of unused ranks and adapters are 0.
 * x and d_xa are the forward pass's.  d_dx_out NULL leaves dx out; d_da and
 * d_db NULL (both) leave the bank's gradients out, and x, d_xa and d_work are
 * then not looked at.  d_work: LCT_ADAPTER_WORK_BYTES of scratch, 16-byte
 * aligned.  Sums over tokens are added in a fixed order.  Errors as
 * lct_adapter_forward. */
lct_status lct_adapter_backward(const lct_adapters *bank, const lct_token_plan *plan, const uint16_t *d_dy,
                                uint64_t ld_dy, const uint16_t *d_x, uint64_t ld_x, const float *d_xa,
                                const uint16_t *d_dx, uint64_t ld_dx, uint16_t *d_dx_out, uint64_t ld_dx_out,
                                uint16_t *d_da, uint16_t *d_db, void *d_work, void *stream);

/* ---- the vocabulary's two ends: the lookup, and the loss ----------------- */

#define LCT_VOCAB_MAX (1 << 24)          /* rows of the vocabulary's matrix */
#define LCT_VOCAB_MAX_COLS (1 << 16)
#define LCT_VOCAB_MAX_TOKENS (1 << 24)
#define LCT_EMBEDDING_CHUNK(tokens) ((tokens) <= 8192 ? 8 : 32) /* sorted tokens that one block adds */
#define LCT_EMBEDDING_PART(cols) (((uint64_t)(cols) + 14) / 8 * 8) /* values of a partial sum */
/* scratch of lct_embedding_grad */
#define LCT_EMBEDDING_WORK_BYTES(tokens, cols)                                                             \
    (16ull + 64ull * (((uint64_t)(tokens) + 3) / 4) +                                                      \
     8ull * (((uint64_t)(tokens) + LCT_EMBEDDING_CHUNK(tokens) - 1) / LCT_EMBEDDING_CHUNK(tokens)) *                  \
         LCT_EMBEDDING_PART(cols))

/* A batch's ids: a row of the vocabulary's matrix for each token.  A negative
 * id is none (padding, a token without a target). */
typedef struct {
    const void *d_ids; /* [tokens], int32 or (wide) int64 */
    int32_t wide;      /* 0 or 1 */
    uint64_t tokens, vocab;
} lct_ids;

/* out_i = scale * table[id_i] for every token, rounded once; a row of zeros for
 * a token without an id, and of NaN for an id of vocab or more.  (The pages have
 * no counterpart.)  d_table holds rows `first` .. first + rows of the matrix
 * [vocab, cols], ld_table values apart, of `dtype`, which is out's too; tokens
 * of other rows are left as they are, so that a compressed matrix can be decoded
 * and looked up a piece at a time.  Rows of whole 16-byte pieces at 16-byte
 * boundaries are the fast case; of others whole aligned pieces are fetched, what
 * lies before a row's first value and behind its last one among it.  Errors: LCT_ERR_INVALID_ARG (NULL or misaligned pointers, strides
 * below cols, rows outside the vocabulary, out over another operand),
 * LCT_ERR_UNSUPPORTED (another dtype, a size above the limits), LCT_ERR_CUDA. */
lct_status lct_embedding(const lct_ids *ids, const void *d_table, uint64_t ld_table, int32_t dtype, uint64_t first,
                         uint64_t rows, uint64_t cols, float scale, void *d_out, uint64_t ld_out, void *stream);

/* The gradient of lct_embedding for dy [tokens, cols], the gradient of its out:
 *   out_v = base_v + scale * sum of dy_i over the tokens with id_i = v
 * for every v of the vocabulary: the dense gradient that the fused steps take
 * (with ld_out = cols).  base may be NULL (zero) or out itself, whose rows
 * without tokens are then not touched: a matrix that is also the loss's
 * projection adds the lookup's gradient to that one's.  Sums are float32, added
 * in an order that depends on the ids alone (the same bits every time), and
 * rounded once.  Ids outside the vocabulary add nothing.  d_work:
 * LCT_EMBEDDING_WORK_BYTES of scratch, 16-byte aligned.  Errors as
 * lct_embedding. */
lct_status lct_embedding_grad(const lct_ids *ids, const void *d_dy, uint64_t ld_dy, int32_t dtype, uint64_t cols,
                              float scale, const void *d_base, uint64_t ld_base, void *d_out, uint64_t ld_out,
                              void *d_work, void *stream);

/* What lct_loss_work_bytes is asked for. */
#define LCT_LOSS_BACKWARD 1
#define LCT_LOSS_WEIGHT 2    /* backward: with the weight's gradient */
#define LCT_LOSS_UNALIGNED 4 /* a row of x or of the weight does not begin at a 16-byte boundary */

/* Bytes of scratch (256-byte aligned) of the two calls below for pieces of at
 * most `rows` rows of the vocabulary: one piece (rows = vocab), or several.  0 for
 * sizes that the calls refuse.  The forward pass takes at most 256 MB and a few
 * words a token; the backward pass, for g and for dx's sums, at most 256 MB each
 * (512 bytes a token, or as much as a float32 dx, where that is more), a copy of
 * x, and with the weight's gradient another in float32 and a word for each row of
 * the vocabulary.  Neither grows with tokens times vocab.  Rows that have
 * to be copied to 16-byte boundaries add a copy of x (forward) and 128 MB or 256
 * rows of the weight; several pieces one of the targets' rows. */
uint64_t lct_loss_work_bytes(uint64_t tokens, uint64_t vocab, uint64_t cols, uint64_t rows, int32_t flags);

/* The cross entropy of a projection onto the vocabulary, which keeps no logits:
 *   lse_i = log sum over v of exp(x_i W_v),   loss_i = lse_i - x_i W_{t_i}
 * in float32.  (The pages have no counterpart.)  x [tokens, cols] and W are
 * BF16; products add in float32.  A token without a target (t_i < 0) has loss 0;
 * a target of vocab or more gives NaN, and so does an infinite logit.
 * d_w holds rows `first` .. first + rows of W [vocab, cols].  The whole W can be
 * given in one call (first 0, rows = vocab), or in pieces, in order, with the
 * same batch, results and d_work: what they have in common lives there from call
 * to call.  d_loss and d_lse are written by the last piece's call.
 * d_total, if not NULL, gets three floats: the sum of the losses, their mean over
 * the tokens with a target, and 1 over the number of those (no token: sum and
 * mean 0).  Rows at 16-byte boundaries are the fast case; others are copied to
 * such in d_work first.  A wait that ran out on the device makes every loss NaN
 * and leaves LCT_ERR_TIMEOUT in d_work's first word.  Errors:
 * LCT_ERR_INVALID_ARG (NULL or misaligned pointers, strides below cols, a piece
 * outside the vocabulary, too little scratch, an output over another operand),
 * LCT_ERR_UNSUPPORTED (a size above the limits), LCT_ERR_CUDA. */
lct_status lct_loss_forward(const lct_ids *targets, const uint16_t *d_x, uint64_t ld_x, uint64_t cols,
                            const uint16_t *d_w, uint64_t ld_w, uint64_t first, uint64_t rows, float *d_loss,
                            float *d_lse, float *d_total, void *d_work, uint64_t work_bytes, void *stream);

/* The gradients of lct_loss_forward: with c_i = d_dloss[i * dloss_stride] *
 * *d_scale (dloss_stride 0 or 1; d_scale NULL: 1), the gradient of loss_i, and
 *   g_iv = c_i (exp(x_i W_v - lse_i) - [v = t_i]),
 *   dx = g W  [tokens, cols],   dW = g^T x  (this piece's rows; d_dw NULL: left out)
 * in BF16.  Logits are computed again, g is held in BF16 for a bounded part of
 * the vocabulary at a time but for its targets' entries, which go into both
 * results in float32.  A token without a target has dx 0 and adds nothing to
 * dW, whatever its x holds; one with an impossible target has dx NaN and adds
 * nothing.  Pieces as in the forward pass (d_dw NULL for all or none); d_dx is
 * written by the last one's call.  Sums are added in an order that depends on the
 * targets alone: the same bits every time.  A wait that ran out on the device
 * leaves LCT_ERR_TIMEOUT in d_work's first word and makes dx NaN, and so the
 * rows of dW that its piece had not finished by then and those of later pieces.
 * Errors as lct_loss_forward. */
lct_status lct_loss_backward(const lct_ids *targets, const uint16_t *d_x, uint64_t ld_x, uint64_t cols,
                             const uint16_t *d_w, uint64_t ld_w, uint64_t first, uint64_t rows, const float *d_loss,
                             const float *d_lse, const float *d_dloss, uint64_t dloss_stride, const float *d_scale,
                             uint16_t *d_dx, uint64_t ld_dx, uint16_t *d_dw, uint64_t ld_dw, void *d_work,
                             uint64_t work_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* LCT_H */
