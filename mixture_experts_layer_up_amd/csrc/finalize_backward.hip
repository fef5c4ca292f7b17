// finalize_backward.hip -- gradients of the routing-weighted finalize.
//
// out[t] = scale sum_j w[t, j] y[p(t, j)] gives
//   dy[p(t, j)] = scale w[t, j] dout[t]       (bf16, one rounding)
//   dw[t, j]    = scale <dout[t], y[p(t, j)]> (fp32 sums; 0 for slots with p = -1)
// One wave per slot: it reads its expert-output row and its token's gradient
// row once, writes one gradient row, and reduces its dot product over the
// lanes in a fixed order.  The slots of a token are neighbours, so its
// gradient row comes from cache for all but the first.  Memory bound: 2 H
// bytes read and 2 H written per slot, 2 H read per token.  8192 tokens top-8,
// hidden 2048: 571 MB in 111 us, 5.1 TB/s, the rate of a large copy.
#include "device_common.h"
#include "kernels_router.h"

namespace moe_lora {
namespace {

constexpr int kSlotsPerBlock = 4;

__global__ __launch_bounds__(256) void finalize_backward_kernel(FinalizeBackwardArgs a)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int x = blockIdx.x * kSlotsPerBlock + wave_id();
    if (x >= a.n)
        return;
    const int t = x / a.k;
    const int p = a.exp2perm[x];
    if (p < 0 || p >= a.n) {
        if (lane == 0 && a.d_weights)
            a.d_weights[x] = 0.0f;
        return;
    }
    const float w = a.d_Y ? a.scale * a.weights[x] : 0.0f;
    const uint16_t *d_row = a.d_out + (size_t)t * a.H;
    const uint16_t *y_row = a.Y + (size_t)p * a.H;
    uint16_t *o_row = a.d_Y + (size_t)p * a.H;
    float dot = 0.0f;
#pragma unroll 4
    for (int c = lane * 8; c < a.H; c += kWave * 8) {
        const u32x4 d = load16(d_row + c);
        const u32x4 y = a.d_weights ? load16_stream(y_row + c) : zero16();
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float d0 = bf16_bits_to_float(d[i] & 0xffffu), d1 = bf16_bits_to_float(d[i] >> 16);
            dot = fmaf(d0, bf16_bits_to_float(y[i] & 0xffffu), dot);
            dot = fmaf(d1, bf16_bits_to_float(y[i] >> 16), dot);
            o[i] = float_to_bf16_bits(w * d0) | (float_to_bf16_bits(w * d1) << 16);
        }
        if (a.d_Y)
            store16_stream(o_row + c, o);
    }
    if (a.d_weights) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            dot += __shfl_xor(dot, off);
        if (lane == 0)
            a.d_weights[x] = a.scale * dot;
    }
}

} // namespace

hipError_t launch_finalize_backward(const FinalizeBackwardArgs &a, hipStream_t s)
{
    if (a.n <= 0)
        return hipSuccess;
    hipLaunchKernelGGL(finalize_backward_kernel, dim3((a.n + kSlotsPerBlock - 1) / kSlotsPerBlock),
                       dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe_lora
