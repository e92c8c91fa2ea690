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
// range of units, whatever the tensors' sizes.  The host says with which
// tensor a block begins: a search by the block would be a chain of reads of
// parameters that no cache holds yet.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <vector>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "internal.h"

namespace lct {
namespace dev {

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 8;  // vectors a thread holds at once
constexpr int kGradBlocksPerSm = 4;
constexpr int kGradCluster = 8;

// One tensor of a launch.  n counts values; bit 63 says they are float32.
struct GradEntry {
    unsigned long long src, dst, n;
};

template <int CAP>
struct GradTable {
    GradEntry e[CAP];
    uint32_t first[CAP + 1];  // units before tensor i; entry `count` is their total
    uint32_t count;
    uint16_t start[kGradMaxParts];  // the tensor that holds block i's first unit
};

constexpr unsigned long long kF32Bit = 1ull << 63;

struct Span {
    unsigned long long src, dst;  // aligned down to 16 bytes
    unsigned long long hi;        // the tensor's bytes are lo..hi, counted from src
    uint32_t lo;
    bool f32;
    bool same_phase, in_place;    // dst lies like src within a vector, or is src
};

__device__ __forceinline__ Span span_of(const GradEntry &e)
{
    Span s;
    s.f32 = (e.n & kF32Bit) != 0;
    const unsigned long long n = e.n & ~kF32Bit;
    s.lo = static_cast<uint32_t>(e.src & 15ull);
    s.hi = s.lo + n * (s.f32 ? 4 : 2);
    s.src = e.src - s.lo;
    s.same_phase = ((e.src ^ e.dst) & 15ull) == 0;
    s.in_place = e.src == e.dst;
    s.dst = e.dst - s.lo;
    return s;
}

// The vector at byte `at` of a tensor; one at the tensor's first or last bytes
// is put together from its own values, the rest of it zero.
template <bool WHOLE>
__device__ __forceinline__ uint4 load_vec(const Span &s, unsigned long long at)
{
    if (WHOLE || (at >= s.lo && at + 16 <= s.hi)) return *reinterpret_cast<const uint4 *>(s.src + at);
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

// The sum of squares of a thread's vectors; bit i of f32 says that vector i
// holds float32 values.  A float sum of at most 64 squares is within 64 *
// 2^-24 of them in the worst order; it is used where it lies well inside
// float's range, and anything else (an overflow, squares that underflow,
// infinities and NaN) is summed again in double from the registers.  A sum of
// zeros alone stays zero.
__device__ __forceinline__ double sum_vectors(const uint4 (&v)[kGradUnroll], uint32_t f32)
{
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kGradUnroll; ++i) {
        s[i & 3] = squares<float>(v[i], (f32 >> i) & 1, s[i & 3]);
        any |= v[i].x | v[i].y | v[i].z | v[i].w;
    }
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
    if (t > 0x1p-60f && t < 0x1p120f) return static_cast<double>(t);
    double d = 0.0;
    if (any) {
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i) d = squares<double>(v[i], (f32 >> i) & 1, d);
    }
    return d;
}

// Block sum of one double a thread, in a fixed order; the first warp gets it.
// A double addition takes a warp 16 cycles of a pipe that the SM has one of, so
// that one warp adds, and little: with eight warps adding and taking roots each
// block took 6 us for what is 0.3 us of work.
__device__ __forceinline__ double block_sum(double v, double *sh)
{
    sh[threadIdx.x] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x < 32) {
#pragma unroll
        for (int i = 0; i < kGradThreads / 32; ++i) t += sh[i * 32 + threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    return t;
}

__host__ __device__ __forceinline__ uint32_t range_at(uint32_t units, uint32_t block, uint32_t blocks)
{
    return static_cast<uint32_t>(static_cast<unsigned long long>(units) * block / blocks);
}

// The tensor that holds a unit: the last one that begins at it or before.
template <int CAP>
__device__ __forceinline__ uint32_t find_entry(const GradTable<CAP> &t, uint32_t unit)
{
    uint32_t lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (t.first[mid] <= unit)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Calls `with(i, span, byte, whole)` for this thread's vector of each of up to
// eight units u0..u1 of a launch that is there, e being the tensor of u0; byte
// is the vector's place in the span.  Eight units inside one tensor, whose
// vectors are all whole, are the case that is to be fast (`whole` is then true
// at compile time: with the checks of a tensor's edges in it, the scaling pass
// was bound by issuing instructions).  Units that several
// tensors share (a list of small ones) have an address each, so that their
// loads are in flight together.
template <int CAP, typename With>
__device__ __forceinline__ void each_unit(const GradTable<CAP> &t, uint32_t u0, uint32_t u1, uint32_t e, With with)
{
    const Span s = span_of(t.e[e]);
    const unsigned long long b0 = static_cast<unsigned long long>(u0 - t.first[e]) * (kGradThreads * 16);
    if (u0 + kGradUnroll <= min(u1, t.first[e + 1]) && b0 >= s.lo && b0 + kGradUnroll * kGradThreads * 16 <= s.hi) {
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i)
            with(i, s, b0 + threadIdx.x * 16 + i * (kGradThreads * 16), std::true_type{});
    } else {
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i) {
            if (u0 + i >= u1) continue;
            while (u0 + i >= t.first[e + 1]) ++e;
            const Span edge = span_of(t.e[e]);
            const unsigned long long at =
                (static_cast<unsigned long long>(u0 + i - t.first[e]) * kGradThreads + threadIdx.x) * 16;
            if (at < edge.hi) with(i, edge, at, std::false_type{});
        }
    }
}

template <int CAP>
__device__ __forceinline__ double sum_units(const GradTable<CAP> &t, uint32_t lo, uint32_t hi)
{
    double acc = 0.0;
    uint32_t e = t.start[blockIdx.x];
    for (uint32_t u = lo; u < hi; u += kGradUnroll) {
        while (u >= t.first[e + 1]) ++e;
        uint4 v[kGradUnroll];
        uint32_t f32 = 0;
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i) v[i] = make_uint4(0, 0, 0, 0);
        each_unit(t, u, hi, e, [&](int i, const Span &s, unsigned long long at, auto whole) {
            v[i] = load_vec<whole.value>(s, at);
            f32 |= static_cast<uint32_t>(s.f32) << i;
        });
        acc += sum_vectors(v, f32);
    }
    return acc;
}

// Partial sums of one launch's tensors, one a block.  `add` is set on a later
// launch over more tensors, which adds to the first one's partial sums.  324 MB
// in 290 tensors take 53 us with the norm's launch, 6.1 TB/s, 91% of a copy's
// rate; 1216 or 2432 blocks, or five or six an SM, were slower than these 608.
template <int CAP>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm)
    k_grad_sum(const __grid_constant__ GradTable<CAP> t, double *part, uint32_t add)
{
    __shared__ double sh[kGradThreads];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t units = t.first[t.count];
    const double acc = sum_units(t, range_at(units, blockIdx.x, gridDim.x), range_at(units, blockIdx.x + 1, gridDim.x));
    const double total = block_sum(acc, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = (add ? part[blockIdx.x] : 0.0) + total;
}

// The root of a total as root * 2^exp with root in [1, 2), in float: the
// total's exponent made even, its fraction rounded to float (2^-24) and the
// root of that (2^-24 again).  Zero, infinity and NaN pass with exp = 0.
struct Root {
    float root;
    int exp;
};
__device__ __forceinline__ Root root_of(double total)
{
    if (!(total > 0.0 && total < __longlong_as_double(0x7FF0000000000000ll)))
        return {static_cast<float>(total), 0};
    // sums of squares of float32 values are normal doubles
    const long long bits = __double_as_longlong(total);
    const int e = static_cast<int>(bits >> 52) - 1023, odd = e & 1;
    const double m = __longlong_as_double((bits & 0x000FFFFFFFFFFFFFll) | (static_cast<long long>(1023 + odd) << 52));
    return {sqrtf(static_cast<float>(m)), (e - odd) / 2};
}
__device__ __forceinline__ float norm_of(const Root &r) { return r.exp > 127 ? INFINITY : ldexpf(r.root, r.exp); }

// g' = (g * pre) * mul.  pre is a power of two, 1 unless the factor lies below
// float's normal range: then mul is the smallest normal power of two times the
// factor's fraction, so that no bit of the factor is lost and only the last
// product rounds (g * pre is exact wherever that product is not zero).  A
// factor below 2^-274, whose results lie below 2^-146, gives zeros.
struct Factor {
    float pre, mul;
    bool one;
};

__device__ __forceinline__ Factor factor_of(const Root &r, float max_norm)
{
    Factor f = {1.0f, 0.0f, false};
    const float n = norm_of(r) + 1e-6f;
    const float c = max_norm / n;
    // a norm above float's range (r.exp > 127, beside which 1e-6 is nothing) lies above every max_norm
    if (r.exp <= 127 && !(c < 0x1p-126f && n < INFINITY)) {
        f.mul = c > 1.0f ? 1.0f : c;  // NaN stays; an infinite norm gives 0
        f.one = f.mul == 1.0f;
        return f;
    }
    int en = r.exp, em, ec;
    const float root = r.exp > 127 ? r.root : frexpf(n, &en);
    const float m = frexpf(frexpf(max_norm, &em) / root, &ec);
    const int e = ec + em - en;  // the factor is m * 2^e, m in [0.5, 1)
    f.pre = e < -125 ? ldexpf(1.0f, e + 125) : 1.0f;
    f.mul = ldexpf(m, max(e, -125));
    return f;
}

// The norm, and where `factor` is given that too, from all partial sums (which
// a thread reads at once: one warp that read them one after another took 6 us).
__global__ void __launch_bounds__(kGradThreads)
    k_grad_norm(const double *part, uint32_t parts, float *norm, float max_norm, Factor *factor)
{
    constexpr int kEach = (kGradMaxParts + kGradThreads - 1) / kGradThreads;
    __shared__ double sh[kGradThreads];
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    double p[kEach], mine = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t at = threadIdx.x + i * kGradThreads;
        p[i] = at < parts ? part[at] : 0.0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) mine += p[i];
    const double total = block_sum(mine, sh);
    if (threadIdx.x == 0) {
        const Root r = root_of(total);
        *norm = norm_of(r);
        if (factor) *factor = factor_of(r, max_norm);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint4 scale_vec(const uint4 &v, bool f32, const Factor &f)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (f.pre == 1.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = f32 ? __float_as_uint(__uint_as_float(w[i]) * f.mul)
                       : pack_bf16(bf_lo(w[i]) * f.mul, bf_hi(w[i]) * f.mul);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = f32 ? __float_as_uint((__uint_as_float(w[i]) * f.pre) * f.mul)
                       : pack_bf16((bf_lo(w[i]) * f.pre) * f.mul, (bf_hi(w[i]) * f.pre) * f.mul);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool WHOLE>
__device__ __forceinline__ void store_vec(const Span &s, unsigned long long at, const uint4 &x)
{
    if (s.same_phase && (WHOLE || (at >= s.lo && at + 16 <= s.hi))) {
        __stcs(reinterpret_cast<uint4 *>(s.dst + at), x);  // not to push out of L2 what is still to be read
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

// Scales units u0..u1 (at most eight), which v holds.
template <int CAP>
__device__ __forceinline__ void load_units(const GradTable<CAP> &t, uint32_t u0, uint32_t u1, uint32_t e, bool one,
                                           uint4 (&v)[kGradUnroll])
{
    each_unit(t, u0, u1, e, [&](int i, const Span &s, unsigned long long at, auto whole) {
        if (!(one && s.in_place)) v[i] = load_vec<whole.value>(s, at);
    });
}
template <int CAP>
__device__ __forceinline__ void scale_units(const GradTable<CAP> &t, uint32_t u0, uint32_t u1, uint32_t e,
                                            const uint4 (&v)[kGradUnroll], const Factor &f)
{
    each_unit(t, u0, u1, e, [&](int i, const Span &s, unsigned long long at, auto whole) {
        if (f.one && s.in_place) return;  // a factor of 1 changes nothing
        store_vec<whole.value>(s, at, scale_vec(v[i], s.f32, f));
    });
}

// The scaling pass, a block for every eight units, last unit first: what the
// summing pass read last is what L2 still holds.  Many short blocks, as each
// one first loads all it has and then stores it: blocks that stay and step
// through their share fall into step with each other, and DRAM then turns
// between reading and writing (norm and clipping of 162 million BF16 values
// took 181 us so, 162 us by short blocks; since the first blocks also load
// before the factor is there and the norm's last step is one round trip, 155
// us: 3 x 324 MB of traffic at 6.3 TB/s, some of it from L2).
template <int CAP>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm)
    k_grad_scale(const __grid_constant__ GradTable<CAP> t, const Factor *factor)
{
    const uint32_t units = t.first[t.count];
    const uint32_t u0 = (gridDim.x - 1 - blockIdx.x) * kGradUnroll, u1 = min(units, u0 + kGradUnroll);
    const uint32_t e = find_entry(t, u0);
    uint4 v[kGradUnroll];
    // the first blocks start while the factor is computed, and load meanwhile: nobody writes gradients there
    const bool early = blockIdx.x < kGradMaxParts;
    if (early) load_units(t, u0, u1, e, false, v);
    cudaGridDependencySynchronize();
    const Factor f = *factor;
    if (!early) load_units(t, u0, u1, e, f.one, v);
    scale_units(t, u0, u1, e, v, f);
}

// Norm and, for CLIP, scaling in one launch of one cluster: a few units, where
// a second launch would cost as much as the work (the norm of 14 tensors of
// 65,536 values in all: 4.5 us, most of it the launch and two meetings).
template <int CAP, bool CLIP>
__global__ void __launch_bounds__(kGradThreads) k_grad_cluster(const __grid_constant__ GradTable<CAP> t,
                                                               float max_norm, float *norm)
{
    namespace cg = cooperative_groups;
    __shared__ double sh[kGradThreads];
    __shared__ double mine;
    __shared__ Factor shared;
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t units = t.first[t.count];
    const uint32_t lo = range_at(units, blockIdx.x, gridDim.x), hi = range_at(units, blockIdx.x + 1, gridDim.x);
    const double acc = block_sum(sum_units(t, lo, hi), sh);
    if (threadIdx.x == 0) mine = acc;
    cluster.sync();
    if (threadIdx.x < 32) {
        double total = threadIdx.x < kGradCluster ? *cluster.map_shared_rank(&mine, threadIdx.x) : 0.0;
#pragma unroll
        for (int o = kGradCluster / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        if (threadIdx.x == 0) {
            const Root r = root_of(total);
            if (blockIdx.x == 0) *norm = norm_of(r);
            if (CLIP) shared = factor_of(r, max_norm);
        }
    }
    cluster.sync();  // no block leaves while its sum is read
    if (CLIP) {
        const Factor f = shared;
        for (uint32_t u = lo; u < hi; u += kGradUnroll) {
            const uint32_t e = find_entry(t, u);
            uint4 v[kGradUnroll];
            load_units(t, u, hi, e, f.one, v);
            scale_units(t, u, hi, e, v, f);
        }
    }
}

}  // namespace dev

namespace {

using dev::GradEntry;
using dev::GradTable;

constexpr int kCapSmall = 64, kCapMiddle = 384, kCapLarge = 1024;
constexpr uint32_t kClusterUnits = 64;

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

// Says with which tensor each block of a grid begins.
template <int CAP>
void set_starts(GradTable<CAP> *t, uint32_t grid)
{
    uint32_t e = 0;
    for (uint32_t b = 0; b < grid; ++b) {
        const uint32_t u = dev::range_at(t->first[t->count], b, grid);
        while (e + 1 < t->count && u >= t->first[e + 1]) ++e;
        t->start[b] = static_cast<uint16_t>(e);
    }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), uint32_t grid, uint32_t threads, uint32_t cluster, bool dependent,
                   cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (cluster > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    } else if (dependent) {  // its blocks may start while the launch before it ends, and wait for it themselves
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int CAP>
cudaError_t run_tables(const GradArgs &a, bool clip, cudaStream_t s)
{
    GradTable<CAP> t;
    uint32_t parts = 0, tables = 0;
    cudaError_t rc;
    uint64_t at = 0;
    do {
        at = fill_table(a, at, &t);
        const uint32_t units = t.first[t.count];
        if (!parts && at == a.count && units <= kClusterUnits) {
            set_starts(&t, dev::kGradCluster);
            return clip ? launch(dev::k_grad_cluster<CAP, true>, dev::kGradCluster, dev::kGradThreads, dev::kGradCluster, false, s, t,
                                 a.max_norm, a.norm)
                        : launch(dev::k_grad_cluster<CAP, false>, dev::kGradCluster, dev::kGradThreads, dev::kGradCluster, false, s, t,
                                 a.max_norm, a.norm);
        }
        // a later launch adds to the first one's partial sums, so it has as many blocks as that
        const uint32_t grid = parts ? parts : (at < a.count ? kGradMaxParts : grad_grid(units));
        set_starts(&t, grid);
        if ((rc = launch(dev::k_grad_sum<CAP>, grid, dev::kGradThreads, 1, parts != 0, s, t, a.part, parts ? 1u : 0u)) != cudaSuccess)
            return rc;
        parts = grid;
        ++tables;
    } while (at < a.count);
    dev::Factor *factor = clip ? reinterpret_cast<dev::Factor *>(a.part + kGradMaxParts) : nullptr;
    rc = launch(dev::k_grad_norm, 1, dev::kGradThreads, 1, true, s, static_cast<const double *>(a.part), parts, a.norm, a.max_norm,
                factor);
    if (!clip || rc != cudaSuccess) return rc;
    at = 0;
    for (bool first = true; first || at < a.count; first = false) {
        if (tables > 1)
            at = fill_table(a, at, &t);
        else
            at = a.count;  // a single table still lies in t
        const uint32_t units = t.first[t.count];
        if (!units) continue;
        rc = launch(dev::k_grad_scale<CAP>, (units + dev::kGradUnroll - 1) / dev::kGradUnroll, dev::kGradThreads, 1, first,
                    s, t, static_cast<const dev::Factor *>(factor));
        if (rc != cudaSuccess) return rc;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_grads(const GradArgs &a, bool clip, cudaStream_t s)
{
    if (a.count <= kCapSmall) return run_tables<kCapSmall>(a, clip, s);
    return a.count <= kCapMiddle ? run_tables<kCapMiddle>(a, clip, s) : run_tables<kCapLarge>(a, clip, s);
}

namespace {

// No output may touch another output, and none may touch a gradient but its
// own, in place.  Buckets come in the order of their addresses, so sorting is
// mostly a look that finds them sorted.
bool grads_apart(const GradArgs &a)
{
    struct R {
        uintptr_t lo, hi;
    };
    std::vector<R> out, in;  // outputs (with the gradients in place), and the other gradients
    out.reserve(a.count);
    for (uint64_t i = 0; i < a.count; ++i) {
        if (!a.n[i]) continue;
        const uint64_t bytes = a.n[i] * (a.dtype[i] == LCT_DTYPE_F32 ? 4 : 2);
        const uintptr_t g = reinterpret_cast<uintptr_t>(a.src[i]), o = reinterpret_cast<uintptr_t>(a.dst[i]);
        out.push_back({o, o + bytes});
        if (g != o) in.push_back({g, g + bytes});
    }
    const auto less = [](const R &x, const R &y) { return x.lo < y.lo; };
    for (auto *v : {&out, &in})
        if (!std::is_sorted(v->begin(), v->end(), less)) std::sort(v->begin(), v->end(), less);
    for (size_t i = 1; i < out.size(); ++i)
        if (out[i].lo < out[i - 1].hi) return false;
    // gradients may overlap one another, so each is held against the outputs on its own
    size_t k = 0;
    for (const R &x : in) {
        while (k < out.size() && out[k].hi <= x.lo) ++k;
        if (k < out.size() && out[k].lo < x.hi) return false;
    }
    return true;
}

// Whether n bytes at p and m bytes at q share none.
bool apart(const void *p, uint64_t n, const void *q, uint64_t m)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return x + n <= y || y + m <= x;
}

lct_status check_grads(GradArgs *a, bool clip)
{
    if (!a->norm || (reinterpret_cast<uintptr_t>(a->norm) & 3u)) return LCT_ERR_INVALID_ARG;
    if (!a->part || (reinterpret_cast<uintptr_t>(a->part) & 15u)) return LCT_ERR_INVALID_ARG;
    if (!apart(a->norm, 4, a->part, LCT_GRAD_WORK_BYTES)) return LCT_ERR_INVALID_ARG;
    if (a->count && (!a->src || !a->n || !a->dtype || (clip && !a->dst))) return LCT_ERR_INVALID_ARG;
    for (uint64_t i = 0; i < a->count; ++i) {
        if (a->dtype[i] != LCT_DTYPE_BF16 && a->dtype[i] != LCT_DTYPE_F32) return LCT_ERR_UNSUPPORTED;
        if (a->n[i] > kMaxN) return LCT_ERR_INVALID_ARG;
        if (!a->n[i]) continue;
        const uintptr_t mask = a->dtype[i] == LCT_DTYPE_F32 ? 3u : 1u;
        if (!a->src[i] || (reinterpret_cast<uintptr_t>(a->src[i]) & mask)) return LCT_ERR_INVALID_ARG;
        if (clip && (!a->dst[i] || (reinterpret_cast<uintptr_t>(a->dst[i]) & mask))) return LCT_ERR_INVALID_ARG;
        // the norm and the scratch are written while gradients are still read
        const uint64_t bytes = a->n[i] * (mask + 1);
        for (const void *p : {a->src[i], clip ? static_cast<const void *>(a->dst[i]) : a->src[i]})
            if (!apart(p, bytes, a->norm, 4) || !apart(p, bytes, a->part, LCT_GRAD_WORK_BYTES))
                return LCT_ERR_INVALID_ARG;
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
