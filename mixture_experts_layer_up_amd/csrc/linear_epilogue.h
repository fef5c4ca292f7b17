// linear_epilogue.h -- what the products do to a sum before they store it.
#pragma once

#include "device_common.h"
#include "kernels_block.h"
#include "moe_lora.h"

namespace moe_lora {
namespace {

// Activation of one value (not swiglu).  The exponential and the reciprocal are
// the hardware's, within about one fp32 ulp each; NaN stays NaN.
__device__ __forceinline__ float activate(int act, float z)
{
    if (act == MOE_LORA_ACT_RELU)
        return z <= 0.0f ? 0.0f : z;
    if (act == MOE_LORA_ACT_GELU) {
        constexpr float k = 2.0f * 0.79788456080286535588f * 1.44269504088896340736f;
        const float e = __builtin_amdgcn_exp2f(-k * fmaf(0.044715f * z * z, z, z));
        return z * __builtin_amdgcn_rcpf(1.0f + e);
    }
    if (act == MOE_LORA_ACT_SILU)
        return silu_f32(z);
    return z;
}

// Column of the stored row for column c of the weight as read; -1: padding.
__device__ __forceinline__ int stored_column(const Epilogue &e, int c)
{
    const int set = c >= e.half ? 1 : 0;
    const int n = c - set * e.half;
    return n < e.N && set < e.sets ? set * e.N + n : -1;
}

// One output: z is the sum of its column (of the gate's column for swiglu, `up`
// that of the up column), n < N the output column.
__device__ __forceinline__ void finish_one(const Epilogue &e, int64_t m, int n, float z, float up)
{
    const int64_t at = m * e.N + n;
    if (e.act == MOE_LORA_ACT_SWIGLU) {
        if (e.bias) {
            z += e.bias[n];
            up += e.bias[e.N + n];
        }
        if (e.preact) {
            e.preact[2 * m * e.N + n] = (uint16_t)float_to_bf16_bits(z);
            e.preact[(2 * m + 1) * e.N + n] = (uint16_t)float_to_bf16_bits(up);
        }
        z = silu_f32(z) * up;
    } else {
        if (e.bias)
            z += e.bias[n];
        if (e.preact)
            e.preact[at] = (uint16_t)float_to_bf16_bits(z);
        z = activate(e.act, z);
    }
    if (e.residual)
        z += bf16_bits_to_float(e.residual[at]);
    if (e.fp32)
        static_cast<float *>(e.out)[at] = z;
    else
        static_cast<uint16_t *>(e.out)[at] = (uint16_t)float_to_bf16_bits(z);
}

__device__ __forceinline__ uint2 pack4(const float (&f)[4])
{
    return uint2{float_to_bf16_bits(f[0]) | (float_to_bf16_bits(f[1]) << 16),
                 float_to_bf16_bits(f[2]) | (float_to_bf16_bits(f[3]) << 16)};
}

// Four outputs n .. n + 3 of row m, n a multiple of 4.  Where N is a multiple of 4
// and the pointers allow it (`wide`).
__device__ __forceinline__ void finish_four(const Epilogue &e, int64_t m, int n, float (&z)[4], float (&up)[4])
{
    if (e.padded) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = stored_column(e, n + i);
            if (c >= 0)
                static_cast<uint16_t *>(e.out)[m * e.sets * e.N + c] = (uint16_t)float_to_bf16_bits(z[i]);
        }
        return;
    }
    if (n >= e.N)
        return;
    if (!e.wide) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < e.N)
                finish_one(e, m, n + i, z[i], up[i]);
        return;
    }
    const int64_t at = m * e.N + n;
    const bool gated = e.act == MOE_LORA_ACT_SWIGLU;
    if (e.bias) {
        const float4 b = *reinterpret_cast<const float4 *>(e.bias + n);
        z[0] += b.x, z[1] += b.y, z[2] += b.z, z[3] += b.w;
        if (gated) {
            const float4 u = *reinterpret_cast<const float4 *>(e.bias + e.N + n);
            up[0] += u.x, up[1] += u.y, up[2] += u.z, up[3] += u.w;
        }
    }
    if (e.preact) {
        *reinterpret_cast<uint2 *>(e.preact + (gated ? 2 * m * e.N + n : at)) = pack4(z);
        if (gated)
            *reinterpret_cast<uint2 *>(e.preact + (2 * m + 1) * e.N + n) = pack4(up);
    }
    if (gated) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            z[i] = silu_f32(z[i]) * up[i];
    } else if (e.act != MOE_LORA_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            z[i] = activate(e.act, z[i]);
    }
    if (e.residual) {
        const uint2 r = *reinterpret_cast<const uint2 *>(e.residual + at);
        z[0] += bf16_bits_to_float(r.x & 0xffffu), z[1] += bf16_bits_to_float(r.x >> 16);
        z[2] += bf16_bits_to_float(r.y & 0xffffu), z[3] += bf16_bits_to_float(r.y >> 16);
    }
    if (e.fp32)
        *reinterpret_cast<float4 *>(static_cast<float *>(e.out) + at) = float4{z[0], z[1], z[2], z[3]};
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(e.out) + at) = pack4(z);
}

} // namespace
} // namespace moe_lora
