// pack_w4.hip -- quantising expert weights to 4 bits and laying them out.
//
// Both run once, when weights are loaded: one thread per output piece (pack) or
// per group and column (quantise), neighbouring threads on neighbouring columns.
// 128 experts, hidden 2048, inter 768: packing w13 (201 MB in and out) takes 106
// us.  Quantising it takes 800 us, four times its bytes: it loads the 805 MB of
// weights twice, for the range and for the codes, 2 bytes a thread and row.
#include "device_common.h"
#include "kernels_w4.h"
#include "w4_layout.h"

namespace moe_lora {
namespace {

// Items are walked with a grid stride: weights of many experts have more words
// than one launch may have threads.
constexpr unsigned kMaxBlocks = 1u << 16;

__device__ __forceinline__ size_t first_item() { return (size_t)blockIdx.x * 256 + threadIdx.x; }
__device__ __forceinline__ size_t item_stride() { return (size_t)gridDim.x * 256; }

// One thread per 16 bytes of packed codes, the load of one lane: 8 K rows of
// one column of two tiles and two chunks.  (A thread per 4-byte word left the
// words of a line to two blocks, and the lines were written 2.6 times.)
__global__ __launch_bounds__(256) void pack_w4_codes_kernel(PackW4Args a)
{
    const W4Layout l = w4_layout(a.E_l, a.K, a.N, a.group, a.zeros != nullptr);
    for (size_t f = first_item(); f < l.scales / 16; f += item_stride()) {
        const int lane = (int)(f & 63);
        const int half = (int)(f >> 6) & 1;
        size_t rest = f >> 7;
        const int u = (int)(rest % l.k_units);
        rest /= l.k_units;
        const int slab = (int)(rest % l.n_slabs);
        const int e = (int)(rest / l.n_slabs);
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = w4_column(slab, half * 2 + (i >> 1), lane & 15, a.I);
            const int k0 = u * kW4UnitK + (i & 1) * 32 + (lane >> 4) * 8;
            uint32_t w = 0;
            if (k0 < a.K) {  // K % 32 == 0: the 8 rows are all inside or all padding
                const uint8_t *src = a.codes + ((size_t)e * (a.K / 2) + k0 / 2) * a.N + col;
#pragma unroll
                for (int r = 0; r < 8; r += 2) {
                    const uint32_t two = src[(size_t)(r / 2) * a.N];
                    const int b0 = w4_nibble_bit(r), b1 = w4_nibble_bit(r + 1);
                    const uint32_t lo = two & 15u, hi = two >> 4;
                    w |= (lo << b0) | (b0 > 28 ? lo >> (32 - b0) : 0u);
                    w |= (hi << b1) | (b1 > 28 ? hi >> (32 - b1) : 0u);
                }
            }
            v[i] = w;
        }
        reinterpret_cast<u32x4 *>(a.dst)[f] = v;
    }
}

// One thread per (expert, slab, group, column): its scale and zero point.
__global__ __launch_bounds__(256) void pack_w4_scales_kernel(PackW4Args a)
{
    const W4Layout l = w4_layout(a.E_l, a.K, a.N, a.group, a.zeros != nullptr);
    const size_t items = (size_t)a.E_l * l.n_slabs * l.n_groups * 64;
    for (size_t f = first_item(); f < items; f += item_stride()) {
        const int c = (int)(f >> 2) & 15, tile = (int)(f & 3);
        size_t rest = f >> 6;
        const int g = (int)(rest % l.n_groups);
        rest /= l.n_groups;
        const int slab = (int)(rest % l.n_slabs);
        const int e = (int)(rest / l.n_slabs);
        const size_t src = ((size_t)e * l.n_groups + g) * a.N + w4_column(slab, tile, c, a.I);
        reinterpret_cast<uint16_t *>(a.dst + l.scales)[f] = a.scales[src];
        if (a.zeros)
            a.dst[l.zeros + f] = 16 + (a.zeros[src] & 15);
    }
}

// Round-to-nearest 4-bit codes, one thread per (expert, group, column).
// Without zero points: s = bf16(max|w| / 7), q = round(w / s) + 8.  With:
// the range [min(w, 0), max(w, 0)] is cut into 15 steps, s = bf16(range / 15),
// z = round(-min / s), q = round(w / s) + z.  Codes and zero points are
// clamped to 0..15 (a NaN weight gives some code in range); an all-zero group
// has s = 0 and stands for zeros.
__global__ __launch_bounds__(256) void quantize_w4_kernel(QuantizeW4Args a)
{
    const int n_groups = (a.K + a.group - 1) / a.group;
    const size_t items = (size_t)a.E_l * n_groups * a.N;
    for (size_t f = first_item(); f < items; f += item_stride()) {
        const int n = (int)(f % a.N);
        size_t rest = f / a.N;
        const int g = (int)(rest % n_groups);
        const int e = (int)(rest / n_groups);
        const int k0 = g * a.group, k1 = min(a.K, k0 + a.group);
        const uint16_t *src = a.src + (size_t)e * a.K * a.N + n;
        float lo = 0.0f, hi = 0.0f;
        for (int k = k0; k < k1; ++k) {
            const float w = bf16_bits_to_float(src[(size_t)k * a.N]);
            lo = fminf(lo, w);
            hi = fmaxf(hi, w);
        }
        // the largest step is max|w| / 7 or (hi - lo) / 15, rounded to bf16; the
        // codes divide by the rounded step, so rounding the step moves no weight
        // by more than the clamp at the ends allows
        const float step = a.zeros ? hi / 15.0f - lo / 15.0f : fmaxf(hi, -lo) / 7.0f;
        const uint32_t bits = float_to_bf16_bits(step);
        const float s = bf16_bits_to_float(bits);
        const bool usable = s > 0.0f && s < INFINITY;
        const float z = !a.zeros ? 8.0f
                                 : usable ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 0.0f;
        a.scales[f] = (uint16_t)bits;
        if (a.zeros)
            a.zeros[f] = (uint8_t)z;
        uint8_t *dst = a.codes + ((size_t)e * (a.K / 2) + k0 / 2) * a.N + n;
        for (int k = k0; k < k1; k += 2) {
            uint32_t q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float w = bf16_bits_to_float(src[(size_t)(k + i) * a.N]);
                const float v = usable ? rintf(w / s) + z : z;
                q[i] = (uint32_t)fminf(fmaxf(v, 0.0f), 15.0f);
            }
            dst[(size_t)((k - k0) / 2) * a.N] = (uint8_t)(q[0] | (q[1] << 4));
        }
    }
}

unsigned blocks_of(size_t items)
{
    const size_t b = (items + 255) / 256;
    return b < kMaxBlocks ? (unsigned)b : kMaxBlocks;
}

} // namespace

hipError_t launch_pack_w4(const PackW4Args &a, hipStream_t s)
{
    const W4Layout l = w4_layout(a.E_l, a.K, a.N, a.group, a.zeros != nullptr);
    hipLaunchKernelGGL(pack_w4_codes_kernel, dim3(blocks_of(l.scales / 16)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(pack_w4_scales_kernel,
                       dim3(blocks_of((size_t)a.E_l * l.n_slabs * l.n_groups * 64)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_quantize_w4(const QuantizeW4Args &a, hipStream_t s)
{
    const size_t items = (size_t)a.E_l * ((a.K + a.group - 1) / a.group) * a.N;
    hipLaunchKernelGGL(quantize_w4_kernel, dim3(blocks_of(items)), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe_lora
