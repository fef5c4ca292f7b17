// finalize_f32.hip -- routing-weighted sum of fp32 expert outputs.
//
// out[t] = scale * sum_j w[t, j] * y[p(t, j)], j ascending, slots with p = -1
// skipped, fp32 sum, one bf16 rounding: finalize.hip's sum for expert outputs
// that were not rounded before.  With 4-bit weights the down product writes
// fp32 rows, so the layer output carries the rounding of the activations and
// its own, not a third one per slot; the rows cost twice the bytes.  2048 tokens
// top-8, hidden 2048: 142 MB in 22.6 us (the rows partly from the last-level
// cache, where the down product left them); a few tokens 2.3..4 us, a launch.
#include "device_common.h"
#include "kernels_w4.h"

namespace moe_lora {
namespace {

__global__ __launch_bounds__(256) void finalize_f32_kernel(FinalizeF32Args a)
{
    const int t = blockIdx.x;
    const int col0 = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (col0 >= a.H)
        return;
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    // slots in groups of 8: every index and row load of a group is issued
    // before any is used
    constexpr int kG = 8;
    for (int j0 = 0; j0 < a.k; j0 += kG) {
        int p[kG];
        float w[kG];
#pragma unroll
        for (int i = 0; i < kG; ++i) {
            const int j = min(j0 + i, a.k - 1);
            p[i] = j0 + i < a.k ? a.exp2perm[(size_t)t * a.k + j] : -1;
            w[i] = a.weights[(size_t)t * a.k + j];
        }
        f32x4 v[kG];
#pragma unroll
        for (int i = 0; i < kG; ++i)  // slots that are not local read row 0, unused
            v[i] = *reinterpret_cast<const f32x4 *>(a.Y + (size_t)max(p[i], 0) * a.H + col0);
#pragma unroll
        for (int i = 0; i < kG; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float s = fmaf(w[i], v[i][e], acc[e]);
                acc[e] = p[i] >= 0 ? s : acc[e];
            }
        }
    }
    uint2 o;
    o.x = float_to_bf16_bits(a.scale * acc[0]) | (float_to_bf16_bits(a.scale * acc[1]) << 16);
    o.y = float_to_bf16_bits(a.scale * acc[2]) | (float_to_bf16_bits(a.scale * acc[3]) << 16);
    *reinterpret_cast<uint2 *>(a.out + (size_t)t * a.H + col0) = o;
}

} // namespace

hipError_t launch_finalize_f32(const FinalizeF32Args &a, hipStream_t s)
{
    if (a.T <= 0)
        return hipSuccess;
    const int col_blocks = (a.H + 1023) / 1024;
    constexpr int kMaxTokens = 1 << 23;  // a launch may have 2^32 - 1 threads in x
    for (int t0 = 0; t0 < a.T; t0 += kMaxTokens) {
        FinalizeF32Args b = a;
        b.exp2perm += (size_t)t0 * a.k;
        b.weights += (size_t)t0 * a.k;
        b.out += (size_t)t0 * a.H;
        hipLaunchKernelGGL(finalize_f32_kernel, dim3(min(kMaxTokens, a.T - t0), col_blocks), dim3(256), 0, s, b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace moe_lora
