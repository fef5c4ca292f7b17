// clip.hip -- the global norm over many gradients, and the clipped gradients.
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),
//   out = c g
// Memory bound: every gradient is read for the sum, and read and written for the
// product.  A block owns a chunk of one tensor; which one it finds in the table
// that travels as the kernel's argument, so a call needs no table in device memory
// and a captured call replays by itself.  Squares are summed in fp64 (values of
// any size, any count; the units for it idle otherwise) in a fixed order: threads,
// waves, blocks.
#include "device_common.h"
#include "kernels_block.h"

namespace moe_lora {
namespace {

constexpr int kThreads = 256;

// The chunk of block `block` : tensor index, first element and elements.
__device__ __forceinline__ int find_tensor(const ClipTable &t, int block)
{
    int lo = 0, hi = t.count - 1;   // the last tensor whose first block is not past `block`
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.t[mid].first <= block)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <int F32>
struct Element;
template <>
struct Element<0> {
    using type = uint16_t;
    static __device__ float load(const uint16_t *p) { return bf16_bits_to_float(*p); }
    static __device__ void store(uint16_t *p, float v) { *p = (uint16_t)float_to_bf16_bits(v); }
};
template <>
struct Element<1> {
    using type = float;
    static __device__ float load(const float *p) { return *p; }
    static __device__ void store(float *p, float v) { *p = v; }
};

// Values of a 16-byte word.
template <int F32>
__device__ __forceinline__ void unpack(u32x4 v, float (&f)[F32 ? 4 : 8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32 != 0) {
            f[i] = __uint_as_float(v[i]);
        } else {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
}

template <int F32>
__device__ __forceinline__ u32x4 pack(const float (&f)[F32 ? 4 : 8])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32 != 0)
            v[i] = __float_as_uint(f[i]);
        else
            v[i] = float_to_bf16_bits(f[2 * i]) | (float_to_bf16_bits(f[2 * i + 1]) << 16);
    }
    return v;
}

// Elements of p before its first 16-byte boundary, at most n.
template <int F32>
__device__ __forceinline__ int head_of(const void *p, int n)
{
    constexpr int kSize = F32 ? 4 : 2;
    const int head = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / kSize;
    return head < n ? head : n;
}

template <int F32>
__device__ __forceinline__ double chunk_squares(const void *data, int64_t at, int n)
{
    using E = Element<F32>;
    constexpr int kPer = F32 ? 4 : 8;
    const auto *p = static_cast<const typename E::type *>(data) + at;
    const int head = head_of<F32>(p, n), words = (n - head) / kPer, tail = head + words * kPer;
    double s = 0.0;
    if ((int)threadIdx.x < head) {
        const double v = E::load(p + threadIdx.x);
        s = v * v;
    }
    if ((int)threadIdx.x < n - tail) {
        const double v = E::load(p + tail + threadIdx.x);
        s = fma(v, v, s);
    }
#pragma unroll 4
    for (int w = threadIdx.x; w < words; w += kThreads) {
        float f[kPer];
        unpack<F32>(load16(p + head + w * kPer), f);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            s = fma((double)f[i], (double)f[i], s);
    }
    return s;
}

__device__ __forceinline__ float scaled(float v, ClipFactor c) { return v * c.power * c.rest; }

// STREAM is a template argument: of two stores under a branch the compiler makes one,
// without the hint.
template <int F32, bool STREAM>
__device__ __forceinline__ void chunk_scale(const void *data, void *out, int64_t at, int n, ClipFactor c)
{
    using E = Element<F32>;
    constexpr int kPer = F32 ? 4 : 8;
    const auto *p = static_cast<const typename E::type *>(data) + at;
    auto *o = static_cast<typename E::type *>(out) + at;
    if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) {
        for (int i = threadIdx.x; i < n; i += kThreads)   // 16-byte boundaries differ
            E::store(o + i, scaled(E::load(p + i), c));
        return;
    }
    const int head = head_of<F32>(p, n), words = (n - head) / kPer, tail = head + words * kPer;
    if ((int)threadIdx.x < head)
        E::store(o + threadIdx.x, scaled(E::load(p + threadIdx.x), c));
    if ((int)threadIdx.x < n - tail)
        E::store(o + tail + threadIdx.x, scaled(E::load(p + tail + threadIdx.x), c));
#pragma unroll 4
    for (int w = threadIdx.x; w < words; w += kThreads) {
        float f[kPer];
        unpack<F32>(load16(p + head + w * kPer), f);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            f[i] = scaled(f[i], c);
        if constexpr (STREAM)
            store16_stream(o + head + w * kPer, pack<F32>(f));
        else
            store16(o + head + w * kPer, pack<F32>(f));
    }
}

__device__ __forceinline__ double wave_sum(double s)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        s += __shfl_xor(s, off);
    return s;
}

__global__ __launch_bounds__(kThreads) void clip_squares_kernel(ClipTable t, double *partial)
{
    __shared__ double part[kThreads / kWave];
    const int i = find_tensor(t, blockIdx.x);
    const int64_t at = (int64_t)((int)blockIdx.x - t.t[i].first) * t.chunk;
    const int64_t left = t.t[i].n - at;
    const int n = left < t.chunk ? (int)left : t.chunk;
    double s = t.t[i].fp32 ? chunk_squares<1>(t.t[i].data, at, n) : chunk_squares<0>(t.t[i].data, at, n);
    s = wave_sum(s);
    if ((threadIdx.x & (kWave - 1)) == 0)
        part[wave_id()] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / kWave; ++w)
            s += part[w];
        partial[blockIdx.x] = s;
    }
}

// Sum of all partial sums by THREADS threads, the same bits in every block, and the norm
// and the factor that come of it.
template <int THREADS>
__device__ __forceinline__ ClipFactor factor_of(const ClipSums &c, float *norm)
{
    __shared__ double part[THREADS / kWave];
    double s = 0.0;
#pragma unroll 4
    for (int64_t b = threadIdx.x; b < c.blocks; b += THREADS)
        s += c.partial[b];
    s = wave_sum(s);
    if ((threadIdx.x & (kWave - 1)) == 0)
        part[wave_id()] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w)
        s += part[w];
    const double total = sqrt(s);
    *norm = (float)total;
    // a norm that is not finite (as the caller sees it): leave the values as they are
    const double f = (double)c.max_norm / (total + 1e-6);
    if (!(*norm < __builtin_inff() && f < 1.0))
        return ClipFactor{1.0f, 1.0f};
    // below the normal range half of the exponent goes into the power (values of 1e36 scaled
    // to a norm of 1e-3 would lose the factor's bits)
    const int e = f > 0.0 && f < 0x1p-126 ? ilogb(f) / 2 : 0;
    return ClipFactor{(float)ldexp(1.0, e), (float)ldexp(f, -e)};
}

constexpr int kNormThreads = 1024;

__global__ __launch_bounds__(kNormThreads) void clip_norm_kernel(ClipSums c)
{
    float norm;
    const ClipFactor f = factor_of<kNormThreads>(c, &norm);
    if (threadIdx.x == 0) {
        *c.norm = norm;
        *c.factor = f;
    }
}

// FEW: the blocks sum the partial sums themselves (up to 4096, 32 KB from the cache) and
// save a launch: 5 tensors of 0.3 M elements 7.6 us in kernels, 14.3 with it (and chunks
// of 32768).
template <bool FEW, bool STREAM>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipTable t, ClipSums c, int first_table)
{
    ClipFactor f;
    if constexpr (FEW) {
        float norm;
        f = factor_of<kThreads>(c, &norm);
        if (first_table && blockIdx.x == 0 && threadIdx.x == 0)
            *c.norm = norm;
    } else {
        f = *c.factor;
    }
    const int i = find_tensor(t, blockIdx.x);
    if (f.power * f.rest == 1.0f && t.t[i].out == t.t[i].data)
        return;
    const int64_t at = (int64_t)((int)blockIdx.x - t.t[i].first) * t.chunk;
    const int64_t left = t.t[i].n - at;
    const int n = left < t.chunk ? (int)left : t.chunk;
    if (t.t[i].fp32)
        chunk_scale<1, STREAM>(t.t[i].data, t.t[i].out, at, n, f);
    else
        chunk_scale<0, STREAM>(t.t[i].data, t.t[i].out, at, n, f);
}

} // namespace

hipError_t launch_clip_squares(const ClipTable &t, double *partial, hipStream_t s)
{
    hipLaunchKernelGGL(clip_squares_kernel, dim3(t.blocks), dim3(kThreads), 0, s, t, partial);
    return hipGetLastError();
}

hipError_t launch_clip_norm(const ClipSums &c, hipStream_t s)
{
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(kNormThreads), 0, s, c);
    return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable &t, const ClipSums &c, bool first_table, hipStream_t s)
{
    const dim3 grid(t.blocks), block(kThreads);
    if (c.blocks <= kClipFew) {
        if (t.stream)
            hipLaunchKernelGGL((clip_scale_kernel<true, true>), grid, block, 0, s, t, c, first_table);
        else
            hipLaunchKernelGGL((clip_scale_kernel<true, false>), grid, block, 0, s, t, c, first_table);
    } else if (t.stream) {
        hipLaunchKernelGGL((clip_scale_kernel<false, true>), grid, block, 0, s, t, c, 0);
    } else {
        hipLaunchKernelGGL((clip_scale_kernel<false, false>), grid, block, 0, s, t, c, 0);
    }
    return hipGetLastError();
}

} // namespace moe_lora
