// Rows of a matrix as blocks of threads read and write them, and the ids that
// choose rows.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "codec_dev.cuh"

namespace lct {
namespace dev {

__device__ __forceinline__ int64_t id_at(const void *ids, bool wide, int64_t i)
{
    return wide ? static_cast<const int64_t *>(ids)[i] : static_cast<const int32_t *>(ids)[i];
}

// ------------------------------------------------- pieces of a row, by a block

// A thread's values of a row: 16 bytes side by side, or (rows at any address)
// every kRowThreads-th value, which a warp still reads and writes in one piece.
constexpr int kRowThreads = 256;
template <typename T, bool AL>
struct RowPiece {
    static constexpr int kVec = AL ? 16 / sizeof(T) : 4;
    static __device__ __forceinline__ int col(int slab, int e)
    {
        const int n = blockDim.x;
        return AL ? (slab * n + static_cast<int>(threadIdx.x)) * kVec + e : (slab * kVec + e) * n + static_cast<int>(threadIdx.x);
    }
};
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v)
{
    if constexpr (std::is_same<T, float>::value)
        return v;
    else
        return __float2bfloat16_rn(v);
}
template <typename T, bool AL>
struct Piece {
    using P = RowPiece<T, AL>;
    union {
        uint4 q;
        T v[P::kVec];
    };
    __device__ __forceinline__ Piece() {}
    __device__ __forceinline__ void load(const T *row, int slab, int cols)
    {
        if (AL) {
            const int c = P::col(slab, 0);
            q = c < cols ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < P::kVec; ++e) v[e] = P::col(slab, e) < cols ? row[P::col(slab, e)] : from_float<T>(0.0f);
        }
    }
    __device__ __forceinline__ void store(T *row, int slab, int cols) const
    {
        if (AL) {
            const int c = P::col(slab, 0);
            if (c < cols) *reinterpret_cast<uint4 *>(row + c) = q;
        } else {
#pragma unroll
            for (int e = 0; e < P::kVec; ++e)
                if (P::col(slab, e) < cols) row[P::col(slab, e)] = v[e];
        }
    }
};

// A thread's float32 values that go with a piece, in a row of such that begins at a 16-byte boundary where pieces do.
template <typename T, bool AL>
struct FloatPiece {
    using P = RowPiece<T, AL>;
    static __device__ __forceinline__ void load(float (&v)[P::kVec], const float *row, int slab, int cols)
    {
        if constexpr (AL) {
            const int c = P::col(slab, 0);
#pragma unroll
            for (int e = 0; e < P::kVec; e += 4) {
                const float4 q = c < cols ? *reinterpret_cast<const float4 *>(row + c + e) : make_float4(0, 0, 0, 0);
                v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < P::kVec; ++e) v[e] = P::col(slab, e) < cols ? row[P::col(slab, e)] : 0.0f;
        }
    }
    static __device__ __forceinline__ void store(const float (&v)[P::kVec], float *row, int slab, int cols)
    {
        if constexpr (AL) {
            const int c = P::col(slab, 0);
#pragma unroll
            for (int e = 0; e < P::kVec; e += 4)
                if (c < cols) *reinterpret_cast<float4 *>(row + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < P::kVec; ++e)
                if (P::col(slab, e) < cols) row[P::col(slab, e)] = v[e];
        }
    }
};

}  // namespace dev

// Threads of a block and slabs of a row for `vec` values a thread.
inline void row_shape(int cols, int vec, uint32_t *threads, uint32_t *slabs)
{
    const uint32_t pieces = (static_cast<uint32_t>(cols) + vec - 1) / vec;
    const uint32_t t = (pieces + 31) / 32 * 32;
    *threads = t < static_cast<uint32_t>(dev::kRowThreads) ? t : dev::kRowThreads;
    *slabs = (pieces + *threads - 1) / *threads;
}

}  // namespace lct
