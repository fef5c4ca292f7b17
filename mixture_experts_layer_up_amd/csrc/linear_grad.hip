// linear_grad.hip -- what the products' gradients need beside the products: the
// gradient through the activation with its column sums, and padded weight copies.
#include "device_common.h"
#include "kernels_block.h"
#include "moe_lora.h"

namespace moe_lora {
namespace {

// act'(z) of gelu and silu.
__device__ __forceinline__ float activation_slope(int act, float z)
{
    float p, inner;   // of z sigmoid(u(z)): p + z p (1 - p) u'
    if (act == MOE_LORA_ACT_GELU) {
        constexpr float c = 2.0f * 0.79788456080286535588f;
        const float zz = z * z;
        p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-c * 1.44269504088896340736f *
                                                               fmaf(0.044715f * zz, z, z)));
        inner = c * fmaf(3.0f * 0.044715f, zz, 1.0f);
    } else {
        p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.44269504088896340736f));
        inner = 1.0f;
    }
    const float q = p * (1.0f - p);
    // past where the sigmoid is 0 or 1 in fp32 the second term is 0 (z inner may be infinite)
    return q == 0.0f ? p : fmaf(z * q, inner, p);
}

// d act'(z), not swiglu.  relu: 0 where z <= 0, whatever d is (0 times an infinity is not).
__device__ __forceinline__ float through_activation(int act, float d, float z)
{
    if (act == MOE_LORA_ACT_NONE)
        return d;
    if (act == MOE_LORA_ACT_RELU)
        return z > 0.0f ? d : 0.0f;
    return d * activation_slope(act, z);
}

__device__ __forceinline__ void store_four(uint16_t *o, const float (&v)[4])
{
    *reinterpret_cast<uint2 *>(o) = uint2{float_to_bf16_bits(v[0]) | (float_to_bf16_bits(v[1]) << 16),
                                          float_to_bf16_bits(v[2]) | (float_to_bf16_bits(v[3]) << 16)};
}

// What rounding to bf16 leaves of each value (exact); nothing of what has no finite rounding.
__device__ __forceinline__ void rest_of_four(float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float first = bf16_bits_to_float(float_to_bf16_bits(v[i]));
        v[i] = __builtin_fabsf(first) < __builtin_inff() ? v[i] - first : 0.0f;
    }
}

constexpr int kTX = 32, kTY = 8;   // threads of a block: 4 columns each, rows

// Block (strip, column group): dz of its rows, and the sums of its columns over them.
// Bound by memory: d_out and preact in, dz out.
//
// dz of a bf16 gradient is rounded to bf16 for the products: one more rounding of what
// has been rounded so before (with it d_x and d_w are off by 0.0024 of their 2-norm, with
// their own rounding alone by 0.0017).  An fp32 gradient has no such rounding yet, and keeps
// 16 bits as the sum of two bf16 values; the products then take twice the steps.  Both ways:
// 8192 rows, 2048 terms, 128 columns with d_bias 35 and 49 us; 2 x 768 columns, swiglu, 123
// and 213, too much for bits that a bf16 gradient does not have.
__global__ __launch_bounds__(kTX *kTY) void act_grad_kernel(ActGradArgs a, int wide)
{
    __shared__ float part[kTY][kTX * 4 * 2];
    const int tx = threadIdx.x % kTX, ty = threadIdx.x / kTX;
    const int n = (blockIdx.y * kTX + tx) * 4;
    const int64_t per = (a.M + a.blocks - 1) / a.blocks;
    const int64_t first = blockIdx.x * per, last = first + per < a.M ? first + per : a.M;
    const bool gated = a.act == MOE_LORA_ACT_SWIGLU;
    const int W = a.sets * a.N;
    float sum[4] = {}, sum_up[4] = {};
    if (n < a.half) {
        for (int64_t m = first + ty; m < last; m += kTY) {
            float d[4] = {}, z[4] = {}, up[4] = {};
            if (wide && n < a.N) {   // N % 4 == 0: all four columns exist, or none (padding)
                if (a.fp32) {
                    const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.d_out) + m * a.N + n);
                    d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.d_out) + m * a.N + n);
                    d[0] = __uint_as_float(v.x << 16), d[1] = __uint_as_float(v.x & 0xffff0000u);
                    d[2] = __uint_as_float(v.y << 16), d[3] = __uint_as_float(v.y & 0xffff0000u);
                }
                if (a.preact) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(a.preact + m * W + n);
                    z[0] = __uint_as_float(v.x << 16), z[1] = __uint_as_float(v.x & 0xffff0000u);
                    z[2] = __uint_as_float(v.y << 16), z[3] = __uint_as_float(v.y & 0xffff0000u);
                    if (gated) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(a.preact + m * W + a.N + n);
                        up[0] = __uint_as_float(u.x << 16), up[1] = __uint_as_float(u.x & 0xffff0000u);
                        up[2] = __uint_as_float(u.y << 16), up[3] = __uint_as_float(u.y & 0xffff0000u);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (n + i >= a.N)
                        continue;
                    d[i] = a.fp32 ? static_cast<const float *>(a.d_out)[m * a.N + n + i]
                                  : bf16_bits_to_float(static_cast<const uint16_t *>(a.d_out)[m * a.N + n + i]);
                    if (a.preact) {
                        z[i] = bf16_bits_to_float(a.preact[m * W + n + i]);
                        if (gated)
                            up[i] = bf16_bits_to_float(a.preact[m * W + a.N + n + i]);
                    }
                }
            }
            float dup[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (gated) {
                    dup[i] = d[i] * silu_f32(z[i]);
                    // the slope first: up slope alone may pass the range where d brings it back
                    d[i] = d[i] * activation_slope(MOE_LORA_ACT_SILU, z[i]) * up[i];
                    sum_up[i] += dup[i];
                } else {
                    d[i] = through_activation(a.act, d[i], z[i]);
                }
                sum[i] += d[i];
            }
            if (a.dz) {   // columns past N are zeros
                uint16_t *o = a.dz + m * ((int64_t)a.sets * a.half) + n;
                store_four(o, d);
                if (gated)
                    store_four(o + a.half, dup);
                if (a.part) {
                    rest_of_four(d);
                    store_four(o + a.part, d);
                    if (gated) {
                        rest_of_four(dup);
                        store_four(o + a.part + a.half, dup);
                    }
                }
            }
        }
    }
    if (!a.partial)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        part[ty][tx * 4 + i] = sum[i];
        part[ty][kTX * 4 + tx * 4 + i] = sum_up[i];
    }
    __syncthreads();
    const int column = threadIdx.x % (kTX * 4), set = threadIdx.x / (kTX * 4);
    const int at = blockIdx.y * kTX * 4 + column;
    if (set < a.sets && at < a.N) {
        float s = 0.0f;
#pragma unroll
        for (int y = 0; y < kTY; ++y)
            s += part[y][set * kTX * 4 + column];
        a.partial[(size_t)blockIdx.x * W + set * a.N + at] = s;
    }
}

__global__ __launch_bounds__(256) void pad_columns_kernel(const uint16_t *w, uint16_t *out, int64_t K, int N,
                                                          int half, int sets)
{
    const int64_t total = K * sets * half;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < total; x += (int64_t)gridDim.x * 256) {
        const int64_t r = x / half;   // row k, set
        const int n = (int)(x - r * half);
        out[x] = n < N ? w[r * N + n] : 0;
    }
}

} // namespace

// Strips of rows: a row a thread as far as 256 strips go (1000 x 1024 values with four
// rows a thread, one after the other: 8.8 us instead of 5.6; 512 strips of 8192 rows
// cost more in the joining than they save).
int act_grad_blocks(int64_t M)
{
    const int64_t strips = (M + kTY - 1) / kTY;
    return strips < 1 ? 1 : strips < 256 ? (int)strips : 256;
}

hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s)
{
    auto at = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const int wide = a.N % 4 == 0 && at(a.d_out, a.fp32 ? 16 : 8) && at(a.preact, 8);
    hipLaunchKernelGGL(act_grad_kernel, dim3(a.blocks, (a.half + kTX * 4 - 1) / (kTX * 4)), dim3(kTX * kTY), 0,
                       s, a, wide);
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess || !a.d_bias || a.partial == a.d_bias)
        return rc;
    return launch_column_sums(a.partial, a.blocks, 1, a.sets * a.N, &a.d_bias, s);
}

hipError_t launch_pad_columns(const uint16_t *w, uint16_t *out, int64_t K, int N, int half, int sets,
                              hipStream_t s)
{
    const int64_t blocks = (K * sets * half + 255) / 256;
    hipLaunchKernelGGL(pad_columns_kernel, dim3(blocks < 1 << 16 ? blocks : 1 << 16), dim3(256), 0, s, w, out, K,
                       N, half, sets);
    return hipGetLastError();
}

} // namespace moe_lora
