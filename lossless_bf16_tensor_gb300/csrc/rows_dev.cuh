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

// A thread's values of a row: 16 bytes side by side, which begin at a 16-byte
// boundary of the row that is written.  Where rows begin at any address, a row's
// first piece begins `skip` values before the row.
constexpr int kRowThreads = 256;
template <typename T>
constexpr int kVec = 16 / sizeof(T);
template <typename T>
__device__ __forceinline__ int piece_of(int slab)
{
    return (slab * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * kVec<T>;
}
template <typename T, bool AL>
__device__ __forceinline__ int skip_of_row(const T *row)
{
    return AL ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}
// The 16 bytes from byte `s` on (even, below 16) of two pieces.
__device__ __forceinline__ uint4 shift16(const uint4 &x, const uint4 &y, uint32_t s)
{
    const bool eight = s & 8, four = s & 4;
    const uint32_t a0 = eight ? x.z : x.x, a1 = eight ? x.w : x.y, a2 = eight ? y.x : x.z, a3 = eight ? y.y : x.w,
                   a4 = eight ? y.z : y.x, a5 = eight ? y.w : y.y;
    const uint32_t b0 = four ? a1 : a0, b1 = four ? a2 : a1, b2 = four ? a3 : a2, b3 = four ? a4 : a3, b4 = four ? a5 : a4;
    const uint32_t bits = (s & 2) * 8;
    return make_uint4(__funnelshift_r(b0, b1, bits), __funnelshift_r(b1, b2, bits), __funnelshift_r(b2, b3, bits),
                      __funnelshift_r(b3, b4, bits));
}
// Up to 16 bytes from any even address: the aligned pieces that hold them (which lie in the tensor's allocation), joined.
__device__ __forceinline__ uint4 load_any(const void *p, uint32_t bytes)
{
    const uint32_t s = reinterpret_cast<uintptr_t>(p) & 15;
    const uint4 *a = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) - s);
    // (the second is read in any case, the first again where it holds all: a branch would keep reads from being batched)
    const uint4 x = a[0], y = a[s + bytes > 16];
    return shift16(x, y, s);
}
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
// AL: rows begin at 16-byte boundaries and are whole pieces long.
template <typename T, bool AL>
struct Piece {
    union {
        uint4 q;
        T v[kVec<T>];
    };
    __device__ __forceinline__ Piece() {}
    // Values c .. of a row; those outside it are zero.
    __device__ __forceinline__ void load(const T *row, int c, int cols)
    {
        if (AL) {
            q = c < cols ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
            return;
        }
        if (c >= 0 && c + kVec<T> <= cols) {
            q = load_any(row + c, 16);
        } else {
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) v[e] = c + e >= 0 && c + e < cols ? row[c + e] : from_float<T>(0.0f);
        }
    }
    // Into a row with a boundary at value c.
    __device__ __forceinline__ void store(T *row, int c, int cols) const
    {
        if (AL ? c < cols : c >= 0 && c + kVec<T> <= cols) {
            *reinterpret_cast<uint4 *>(row + c) = q;
        } else if (!AL) {
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e)
                if (c + e >= 0 && c + e < cols) row[c + e] = v[e];
        }
    }
};

// The float32 values of a thread's piece, at their place in a row of such that has room for whole pieces.
template <typename T>
__device__ __forceinline__ void load_floats(float (&v)[kVec<T>], const float *row, int piece)
{
#pragma unroll
    for (int e = 0; e < kVec<T>; e += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(row + piece + e);
        v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
    }
}
template <typename T>
__device__ __forceinline__ void store_floats(const float (&v)[kVec<T>], float *row, int piece)
{
#pragma unroll
    for (int e = 0; e < kVec<T>; e += 4)
        *reinterpret_cast<float4 *>(row + piece + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
}

}  // namespace dev

// Threads of a block and slabs of a row for `vec` values a thread; a row at any address may begin inside a piece.
inline void row_shape(int cols, int vec, bool aligned, uint32_t *threads, uint32_t *slabs)
{
    const uint32_t pieces = (static_cast<uint32_t>(cols) + (aligned ? 0 : vec - 1) + vec - 1) / vec;
    const uint32_t t = (pieces + 31) / 32 * 32;
    *threads = t < static_cast<uint32_t>(dev::kRowThreads) ? t : dev::kRowThreads;
    *slabs = (pieces + *threads - 1) / *threads;
}

}  // namespace lct
