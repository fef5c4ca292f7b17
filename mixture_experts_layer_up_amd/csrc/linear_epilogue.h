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

// finish_one where the row and the column of the product exist.
__device__ __forceinline__ void finish_element(const Epilogue &e, int M, int64_t m, int c, float z, float up)
{
    if (m >= M)
        return;
    if (e.padded) {
        const int at = stored_column(e, c);
        if (at >= 0)
            static_cast<uint16_t *>(e.out)[m * e.sets * e.N + at] = (uint16_t)float_to_bf16_bits(z);
    } else if (c < e.N) {
        finish_one(e, m, c, z, up);
    }
}

__device__ __forceinline__ u32x4 pack_eight(const float (&f)[8])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = float_to_bf16_bits(f[2 * i]) | (float_to_bf16_bits(f[2 * i + 1]) << 16);
    return v;
}

// Eight outputs n .. n + 7 of row m, 16 bytes at a time: `wide` (N and n are multiples
// of 8), n < N.
__device__ __forceinline__ void finish_eight(const Epilogue &e, int64_t m, int n, float (&z)[8], float (&up)[8])
{
    const int64_t at = m * e.N + n;
    const bool gated = e.act == MOE_LORA_ACT_SWIGLU;
    if (e.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += e.bias[n + i];
        if (gated) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                up[i] += e.bias[e.N + n + i];
        }
    }
    if (e.preact) {
        store16(e.preact + (gated ? 2 * m * e.N + n : at), pack_eight(z));
        if (gated)
            store16(e.preact + (2 * m + 1) * e.N + n, pack_eight(up));
    }
    if (gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = silu_f32(z[i]) * up[i];
    } else if (e.act == MOE_LORA_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = activate(MOE_LORA_ACT_RELU, z[i]);
    } else if (e.act == MOE_LORA_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = activate(MOE_LORA_ACT_GELU, z[i]);
    } else if (e.act == MOE_LORA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = silu_f32(z[i]);
    }
    if (e.residual) {
        const u32x4 r = load16(e.residual + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[2 * i] += __uint_as_float(r[i] << 16);
            z[2 * i + 1] += __uint_as_float(r[i] & 0xffff0000u);
        }
    }
    if (e.fp32) {
        float *o = static_cast<float *>(e.out) + at;
        *reinterpret_cast<f32x4 *>(o) = f32x4{z[0], z[1], z[2], z[3]};
        *reinterpret_cast<f32x4 *>(o + 4) = f32x4{z[4], z[5], z[6], z[7]};
    } else {
        store16(static_cast<uint16_t *>(e.out) + at, pack_eight(z));
    }
}

} // namespace
} // namespace moe_lora
