// Global gradient norm over many tensors, and clipping by it.
//
//   |G| = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (|G| + 1e-6)),  g' = c * g
//
// A norm reads every gradient once (2 or 4 bytes a value, two operations a
// value), so HBM bounds it.  Clipping reads them a second time, since c is
// known only when the whole sum is, and writes them once.
//
// The tensors' addresses travel as kernel parameters, so a call copies no
// table to the device and keeps nothing between calls.  The tensors are cut
// into units of 256 16-byte vectors, counted from the aligned address at or
// below a tensor's first value, and every block takes an equal contiguous
// range of units, whatever the tensors' sizes: one binary search a block
// finds its first tensor.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include <cuda_bf16.h>

#include "internal.h"

namespace lct {
namespace dev {

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 8;  // vectors a thread holds at once

// One tensor of a launch.  n counts values; bit 63 says they are float32.
struct GradEntry {
    unsigned long long src, dst, n;
};

template <int CAP>
struct GradTable {
    GradEntry e[CAP];
    uint32_t first[CAP + 1];  // units before tensor i; entry `count` is their total
    uint32_t count;
};

constexpr unsigned long long kF32Bit = 1ull << 63;

struct Span {
    unsigned long long src, dst;  // aligned down to 16 bytes
    unsigned long long lo, hi;    // bytes of the tensor, counted from src
    unsigned long long nvec;
    bool f32;
    bool same_phase;              // dst lies like src within a vector
};

__device__ __forceinline__ Span span_of(const GradEntry &e)
{
    Span s;
    s.f32 = (e.n & kF32Bit) != 0;
    const unsigned long long n = e.n & ~kF32Bit;
    s.lo = e.src & 15ull;
    s.hi = s.lo + n * (s.f32 ? 4 : 2);
    s.src = e.src - s.lo;
    s.same_phase = ((e.src ^ e.dst) & 15ull) == 0;
    s.dst = e.dst - s.lo;
    s.nvec = (s.hi + 15) / 16;
    return s;
}

// Vector v of a tensor; a vector at the tensor's first or last bytes is put
// together from its own values, the rest of it zero.
__device__ __forceinline__ uint4 load_vec(const Span &s, unsigned long long v)
{
    const unsigned long long at = v * 16;
    if (at >= s.lo && at + 16 <= s.hi) return *reinterpret_cast<const uint4 *>(s.src + at);
    uint32_t w[4] = {0, 0, 0, 0};
    if (s.f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + 4 * i >= s.lo && at + 4 * i < s.hi) w[i] = *reinterpret_cast<const uint32_t *>(s.src + at + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + 2 * i >= s.lo && at + 2 * i < s.hi)
                w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(s.src + at + 2 * i))
                            << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <typename T>
__device__ __forceinline__ T squares(const uint4 &v, bool f32, T acc)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (f32) {
            const T a = static_cast<T>(__uint_as_float(w[i]));
            acc = acc + a * a;
        } else {
            const T a = static_cast<T>(bf_lo(w[i])), b = static_cast<T>(bf_hi(w[i]));
            acc = acc + a * a;
            acc = acc + b * b;
        }
    }
    return acc;
}

// The sum of squares of a thread's vectors.  A float sum of at most 64
// squares is within 64 * 2^-24 of them in the worst order; it is used where
// it lies well inside float's range, and anything else (an overflow, squares
// that underflow, infinities and NaN) is summed again in double from the
// registers.  A sum of zeros alone stays zero.
__device__ __forceinline__ double sum_vectors(const uint4 (&v)[kGradUnroll], bool f32)
{
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kGradUnroll; ++i) {
        s[i & 3] = squares<float>(v[i], f32, s[i & 3]);
        any |= v[i].x | v[i].y | v[i].z | v[i].w;
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    if (t > 0x1p-60f && t < 0x1p120f) return static_cast<double>(t);
    double d = 0.0;
    if (any & (f32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) {
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i) d = squares<double>(v[i], f32, d);
    }
    return d;
}

template <int CAP>
__device__ __forceinline__ uint32_t find_entry(const GradTable<CAP> &t, uint32_t unit)
{
    uint32_t lo = 0, hi = t.count;  // the last i with first[i] <= unit and some units
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (t.first[mid] <= unit)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Block sum of one double a thread, in a fixed order; every thread gets it.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += sh[i];
    __syncthreads();
    return t;
}

__device__ __forceinline__ uint32_t range_at(uint32_t units, uint32_t block, uint32_t blocks)
{
    return static_cast<uint32_t>(static_cast<unsigned long long>(units) * block / blocks);
}

template <int CAP>
__device__ __forceinline__ double sum_units(const GradTable<CAP> &t, uint32_t lo, uint32_t hi)
{
    double acc = 0.0;
    uint32_t e = lo < hi ? find_entry(t, lo) : 0;
    for (uint32_t u = lo; u < hi;) {
        while (u >= t.first[e + 1]) ++e;
        const Span s = span_of(t.e[e]);
        const uint32_t end = min(hi, t.first[e + 1]), base = t.first[e];
        for (; u < end; u += kGradUnroll) {
            const uint32_t count = min(end - u, static_cast<uint32_t>(kGradUnroll));
            const unsigned long long v0 = static_cast<unsigned long long>(u - base) * kGradThreads + threadIdx.x;
            uint4 v[kGradUnroll];
#pragma unroll
            for (int i = 0; i < kGradUnroll; ++i) {
                const unsigned long long at = v0 + static_cast<unsigned long long>(i) * kGradThreads;
                v[i] = i < count && at < s.nvec ? load_vec(s, at) : make_uint4(0, 0, 0, 0);
            }
            acc += sum_vectors(v, s.f32);
        }
        u = end;
    }
    return acc;
}

// Partial sums of one launch's tensors, one a block.  `add` is set on a later
// launch over more tensors, which adds to the first one's partial sums.
template <int CAP>
__global__ void __launch_bounds__(kGradThreads) k_grad_sum(const __grid_constant__ GradTable<CAP> t, double *part,
                                                           uint32_t add)
{
    __shared__ double sh[kGradThreads / 32];
    const uint32_t units = t.first[t.count];
    const double acc = sum_units(t, range_at(units, blockIdx.x, gridDim.x), range_at(units, blockIdx.x + 1, gridDim.x));
    const double total = block_sum<kGradThreads>(acc, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = (add ? part[blockIdx.x] : 0.0) + total;
}

__device__ __forceinline__ double total_of(const double *part, uint32_t parts, double *sh)
{
    double a = 0.0;
    for (uint32_t i = threadIdx.x; i < parts; i += kGradThreads) a += part[i];
    return block_sum<kGradThreads>(a, sh);
}

__global__ void __launch_bounds__(kGradThreads) k_grad_norm(const double *part, uint32_t parts, float *norm)
{
    __shared__ double sh[kGradThreads / 32];
    const double total = total_of(part, parts, sh);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(total));
}

// g' = (g * pre) * mul.  The factor is taken in double from the double norm,
// so a norm above float's range still clips; a factor too small for a normal
// float is split in two.
struct Factor {
    float pre, mul;
    bool one;
};

__device__ __forceinline__ Factor factor_of(double total, float max_norm)
{
    double c = static_cast<double>(max_norm) / (sqrt(total) + 1e-6);
    if (c > 1.0) c = 1.0;  // NaN stays
    Factor f;
    f.one = c == 1.0;
    f.pre = c < 0x1p-100 ? 0x1p-64f : 1.0f;
    f.mul = static_cast<float>(c < 0x1p-100 ? c * 0x1p64 : c);
    return f;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint4 scale_vec(const uint4 &v, bool f32, const Factor &f)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = f32 ? __float_as_uint((__uint_as_float(w[i]) * f.pre) * f.mul)
                   : pack_bf16((bf_lo(w[i]) * f.pre) * f.mul, (bf_hi(w[i]) * f.pre) * f.mul);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_vec(const Span &s, unsigned long long v, const uint4 &x)
{
    const unsigned long long at = v * 16;
    if (s.same_phase && at >= s.lo && at + 16 <= s.hi) {
        *reinterpret_cast<uint4 *>(s.dst + at) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (s.f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + 4 * i >= s.lo && at + 4 * i < s.hi) *reinterpret_cast<uint32_t *>(s.dst + at + 4 * i) = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + 2 * i >= s.lo && at + 2 * i < s.hi)
                *reinterpret_cast<uint16_t *>(s.dst + at + 2 * i) = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

// The scaling pass over units lo..hi, last unit first: what the summing pass
// read last is what L2 still holds.
template <int CAP>
__device__ __forceinline__ void scale_units(const GradTable<CAP> &t, uint32_t lo, uint32_t hi, const Factor &f)
{
    uint32_t e = lo < hi ? find_entry(t, hi - 1) : 0;
    for (uint32_t end = hi; end > lo;) {
        while (t.first[e] >= end) --e;
        const Span s = span_of(t.e[e]);
        const uint32_t base = t.first[e], begin = max(lo, base);
        const bool skip = f.one && t.e[e].src == t.e[e].dst;
        while (!skip && end > begin) {
            const uint32_t count = min(end - begin, static_cast<uint32_t>(kGradUnroll));
            const uint32_t u = end - count;
            const unsigned long long v0 = static_cast<unsigned long long>(u - base) * kGradThreads + threadIdx.x;
            uint4 v[kGradUnroll];
#pragma unroll
            for (int i = 0; i < kGradUnroll; ++i) {
                const unsigned long long at = v0 + static_cast<unsigned long long>(i) * kGradThreads;
                if (i < count && at < s.nvec) v[i] = load_vec(s, at);
            }
#pragma unroll
            for (int i = 0; i < kGradUnroll; ++i) {
                const unsigned long long at = v0 + static_cast<unsigned long long>(i) * kGradThreads;
                if (i < count && at < s.nvec) store_vec(s, at, scale_vec(v[i], s.f32, f));
            }
            end = u;
        }
        end = begin;
    }
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) k_grad_scale(const __grid_constant__ GradTable<CAP> t,
                                                             const double *part, uint32_t parts, float max_norm,
                                                             float *norm)
{
    __shared__ double sh[kGradThreads / 32];
    const double total = total_of(part, parts, sh);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(sqrt(total));
    const Factor f = factor_of(total, max_norm);
    const uint32_t units = t.first[t.count];
    scale_units(t, range_at(units, blockIdx.x, gridDim.x), range_at(units, blockIdx.x + 1, gridDim.x), f);
}

}  // namespace dev

namespace {

using dev::GradEntry;
using dev::GradTable;

constexpr int kCapSmall = 64, kCapLarge = 1024;

uint64_t units_of(uint64_t src, uint64_t bytes)
{
    if (!bytes) return 0;
    const uint64_t vecs = ((src & 15) + bytes + 15) / 16;
    return (vecs + dev::kGradThreads - 1) / dev::kGradThreads;
}

// Fills a table with as many tensors as it takes, from `at` on; returns the
// first one that is left.
template <int CAP>
uint64_t fill_table(const GradArgs &a, uint64_t at, GradTable<CAP> *t)
{
    uint32_t k = 0, units = 0;
    for (; at < a.count && k < CAP; ++at) {
        if (!a.n[at]) continue;
        const uint64_t bytes = a.n[at] * (a.dtype[at] == LCT_DTYPE_F32 ? 4 : 2);
        const uint64_t src = reinterpret_cast<uint64_t>(a.src[at]);
        const uint64_t u = units_of(src, bytes);
        if (k > 0 && u > 0x7FFFFFFFull - units) break;
        t->e[k].src = src;
        t->e[k].dst = a.dst ? reinterpret_cast<uint64_t>(a.dst[at]) : src;
        t->e[k].n = a.n[at] | (a.dtype[at] == LCT_DTYPE_F32 ? dev::kF32Bit : 0);
        t->first[k] = units;
        units += static_cast<uint32_t>(u);
        ++k;
    }
    t->first[k] = units;
    t->count = k;
    return at;
}

uint32_t grad_grid(uint32_t units)
{
    const uint32_t want = (units + 1) / 2;  // at least two units a block
    return std::max(1u, std::min(want, static_cast<uint32_t>(kGradMaxParts)));
}

template <int CAP>
cudaError_t run_tables(const GradArgs &a, bool clip, cudaStream_t s)
{
    GradTable<CAP> t;
    uint32_t parts = 0;
    cudaError_t rc;
    uint64_t at = 0;
    do {
        at = fill_table(a, at, &t);
        // a later launch adds to the first one's partial sums, so it has no more blocks than that
        const uint32_t grid = parts ? parts : (at < a.count ? kGradMaxParts : grad_grid(t.first[t.count]));
        dev::k_grad_sum<CAP><<<grid, dev::kGradThreads, 0, s>>>(t, a.part, parts ? 1u : 0u);
        if ((rc = cudaGetLastError()) != cudaSuccess) return rc;
        parts = grid;
    } while (at < a.count);
    if (!clip) {
        dev::k_grad_norm<<<1, dev::kGradThreads, 0, s>>>(a.part, parts, a.norm);
        return cudaGetLastError();
    }
    at = 0;
    bool first = true;
    do {
        at = fill_table(a, at, &t);
        const uint32_t grid = at < a.count || !first ? kGradMaxParts : grad_grid(t.first[t.count]);
        dev::k_grad_scale<CAP><<<grid, dev::kGradThreads, 0, s>>>(t, a.part, parts, a.max_norm,
                                                                  first ? a.norm : nullptr);
        if ((rc = cudaGetLastError()) != cudaSuccess) return rc;
        first = false;
    } while (at < a.count);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_grads(const GradArgs &a, bool clip, cudaStream_t s)
{
    return a.count <= kCapSmall ? run_tables<kCapSmall>(a, clip, s) : run_tables<kCapLarge>(a, clip, s);
}

namespace {

// No output may touch another output, and none may touch a gradient but its
// own, in place.
bool grads_apart(const GradArgs &a)
{
    struct R {
        uintptr_t lo, hi;
        uint64_t tensor;
        int kind;  // 0 gradient, 1 output, 2 both (in place)
    };
    std::vector<R> r;
    r.reserve(2 * a.count);
    for (uint64_t i = 0; i < a.count; ++i) {
        if (!a.n[i]) continue;
        const uint64_t bytes = a.n[i] * (a.dtype[i] == LCT_DTYPE_F32 ? 4 : 2);
        const uintptr_t g = reinterpret_cast<uintptr_t>(a.src[i]), o = reinterpret_cast<uintptr_t>(a.dst[i]);
        if (g == o)
            r.push_back({g, g + bytes, i, 2});
        else {
            r.push_back({g, g + bytes, i, 0});
            r.push_back({o, o + bytes, i, 1});
        }
    }
    std::sort(r.begin(), r.end(), [](const R &x, const R &y) { return x.lo < y.lo; });
    uintptr_t any_hi = 0, out_hi = 0;  // furthest end of any range, and of an output, so far
    for (const R &x : r) {
        if (x.kind ? x.lo < any_hi : x.lo < out_hi) return false;
        any_hi = std::max(any_hi, x.hi);
        if (x.kind) out_hi = std::max(out_hi, x.hi);
    }
    return true;
}

lct_status check_grads(GradArgs *a, bool clip)
{
    if (!a->norm || (reinterpret_cast<uintptr_t>(a->norm) & 3u)) return LCT_ERR_INVALID_ARG;
    if (!a->part || (reinterpret_cast<uintptr_t>(a->part) & 15u)) return LCT_ERR_INVALID_ARG;
    if (a->count && (!a->src || !a->n || !a->dtype || (clip && !a->dst))) return LCT_ERR_INVALID_ARG;
    for (uint64_t i = 0; i < a->count; ++i) {
        if (a->dtype[i] != LCT_DTYPE_BF16 && a->dtype[i] != LCT_DTYPE_F32) return LCT_ERR_UNSUPPORTED;
        if (a->n[i] > kMaxN) return LCT_ERR_INVALID_ARG;
        if (!a->n[i]) continue;
        const uintptr_t mask = a->dtype[i] == LCT_DTYPE_F32 ? 3u : 1u;
        if (!a->src[i] || (reinterpret_cast<uintptr_t>(a->src[i]) & mask)) return LCT_ERR_INVALID_ARG;
        if (clip && (!a->dst[i] || (reinterpret_cast<uintptr_t>(a->dst[i]) & mask))) return LCT_ERR_INVALID_ARG;
    }
    return LCT_OK;
}

}  // namespace
}  // namespace lct

using namespace lct;

extern "C" lct_status lct_grad_norm(const void *const *d_g, const uint64_t *n, const int32_t *dtype, uint64_t count,
                                    float *d_norm, void *d_work, void *stream)
{
    GradArgs a{d_g, nullptr, n, dtype, count, 0.0f, d_norm, static_cast<double *>(d_work)};
    const lct_status rc = check_grads(&a, false);
    if (rc != LCT_OK) return rc;
    return launch_grads(a, false, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
}

extern "C" lct_status lct_grad_clip(const void *const *d_g, void *const *d_out, const uint64_t *n,
                                    const int32_t *dtype, uint64_t count, float max_norm, float *d_norm, void *d_work,
                                    void *stream)
{
    GradArgs a{d_g, d_out, n, dtype, count, max_norm, d_norm, static_cast<double *>(d_work)};
    const lct_status rc = check_grads(&a, true);
    if (rc != LCT_OK) return rc;
    if (!(max_norm > 0.0f) || !std::isfinite(max_norm)) return LCT_ERR_INVALID_ARG;
    if (!grads_apart(a)) return LCT_ERR_INVALID_ARG;
    return launch_grads(a, true, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LCT_OK : LCT_ERR_CUDA;
}
