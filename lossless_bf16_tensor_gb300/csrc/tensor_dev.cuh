// What the kernels with tensor-core products share (sm_103a): operand
// descriptors and products of tcgen05, TMEM, boxes of matrices (TMA), bounded
// waits at mbarriers; and on the host a launch with its attributes and the maps
// of boxes.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>

#include "codec_dev.cuh"

namespace lct {
namespace dev {

// ---------------------------------------------------------------- tcgen05

// A row-swizzled tile: rows of 128 bytes, the 16-byte piece c of row r at
// piece c ^ (r & 7) (the 128-byte swizzle that TMEM operands are read with).
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t piece)
{
    return row * 128 + ((piece ^ (row & 7)) << 4);
}

// Shared-memory matrix descriptor of such a tile at a 1024-byte boundary plus
// an offset.  Rows come in groups of eight, 1024 bytes apart; `atoms` is the
// distance between 64-column tiles where the operand's rows run along the
// memory's columns.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t atoms)
{
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(atoms >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction word: float32 sums of BF16 products, M = 128, N columns; an
// operand is "across" when its rows run along the columns of its tile.
__device__ __forceinline__ uint32_t mma_word(uint32_t n, bool a_across, bool b_across)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_across ? 1u << 15 : 0u) | (b_across ? 1u << 16 : 0u) |
           ((n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t word, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// One thread of the warp, as the compiler knows: products take their operands
// from uniform registers, which a plain `lane == 0` makes it build thread by
// thread (650 cycles for four products, where this takes 100).
__device__ __forceinline__ bool elect()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// `bar` gets one arrival when the products issued so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t *at, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Eight columns of this lane's row (lane 32 w + l of the warp w of a quarter).
__device__ __forceinline__ void tmem_load8(uint32_t addr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------- shared memory, boxes

__device__ __forceinline__ void store16(uint32_t dst, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t src)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(src)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    return at;
}
// Writes before it, of this block's or of a peer's memory, are seen by products after it.
__device__ __forceinline__ void fence_proxy_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// A box of a row-major matrix into a row-swizzled tile; what lies outside is
// zero.  x begins a 16-byte piece.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void fetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}


// ------------------------------------------------------------------- waits

// Waits at a barrier, for at most about a second by the SM's clock (a wait
// that passes takes microseconds).  After a wait that ran out a thread waits no
// more and tells nobody anything, and it starts no box and no product: what it
// started last has had that second to end.
constexpr uint32_t kWaitClocks = 1800000000u;
__device__ __forceinline__ bool try_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
struct Waiter {
    bool dead = false;
    template <typename Ready>
    __device__ __forceinline__ void until(Ready ready)
    {
        if (dead || ready()) return;
        const uint32_t t0 = static_cast<uint32_t>(clock());
#pragma unroll 1
        while (!ready())
            if (static_cast<uint32_t>(clock()) - t0 > kWaitClocks) {
                dead = true;
                break;
            }
    }
    __device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity)  // for this block's own warps
    {
        until([&] { return mbar_try(bar, parity); });
    }
    __device__ __forceinline__ void wait_both(uint64_t *a, uint32_t a_parity, uint64_t *b, uint32_t b_parity)
    {
        until([&] {
            const bool x = mbar_try(a, a_parity), y = mbar_try(b, b_parity);
            return x && y;
        });
    }
    __device__ __forceinline__ void wait_cluster(uint64_t *bar, uint32_t parity)  // for the cluster's
    {
        until([&] { return try_cluster(smem_addr(bar), parity); });
    }
};

}  // namespace dev

// What a kernel may have of dynamic shared memory, asked for before a launch that takes more than 32 KB.  It is a
// property of the kernel and not of the launch: where the sizes of a call choose how much is taken, another thread's
// smaller launch in between would lower it again.  So it is the same for all of them.  (Static shared memory, here
// below 10 KB, comes on top.)
constexpr uint32_t kSharedMost = 200 * 1024;

template <bool DEPENDENT = false, typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, uint32_t threads, uint32_t smem, uint32_t cluster, cudaStream_t s,
                   A... args)
{
    if (smem > 32 * 1024) {  // above what every kernel may have
        const cudaError_t rc = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    smem < kSharedMost ? kSharedMost : smem);
        if (rc != cudaSuccess) return rc;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = DEPENDENT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A box map of [planes][rows][cols] BF16 (planes 0: a plain matrix) for boxes
// of 64 columns by `box` rows in the 128-byte swizzle.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}
inline bool box_map(CUtensorMap *m, const void *p, uint64_t cols, uint64_t rows, uint64_t ld, uint64_t planes, uint32_t box)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    if (rows == 1) ld = (cols + 7) / 8 * 8;  // the stride of a single row means nothing, but has to be one
    const cuuint64_t dims[3] = {cols, rows, planes}, strides[2] = {2 * ld, 2 * ld * rows};
    const cuuint32_t size[3] = {64, box, 1}, step[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes ? 3 : 2, const_cast<void *>(p), dims, strides, size, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for float32 (planes > 0) and boxes of 32 columns by 32 rows.
inline bool box_map32(CUtensorMap *m, const float *p, uint64_t cols, uint64_t rows, uint64_t ld, uint64_t planes)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {cols, rows, planes}, strides[2] = {4 * ld, 4 * ld * rows};
    const cuuint32_t size[3] = {32, 32, 1}, step[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float *>(p), dims, strides, size, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How many clusters of a size the GPU holds at once (0: none, or an error).
template <typename... P>
uint32_t clusters_at_once(void (*kernel)(P...), uint32_t threads, uint32_t smem, uint32_t cluster)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();  // a size that does not fit is no error of the caller's
        return 0;
    }
    return n > 0 ? static_cast<uint32_t>(n) : 0;
}

}  // namespace lct
