// block_norm.hip -- the norms before and after a block with its gate and the
// residual sum, and their gradients.
//
//   b = y s (o + w_post),  s = rsqrt(mean(y^2) + eps)     (b = y without w_post)
//   r = alpha x + g b
//   z = r p (o + w_pre),   p = rsqrt(mean(r^2) + eps)
// and, with q = dz (o + w_pre), rh = r p, yh = y s, D the gradient of r:
//   D = dr + p (q - rh mean(q rh))        dx = alpha D       dw_pre = sum_t dz rh
//   h = g D (o + w_post)                  dw_post = sum_t g D yh
//   dy = s (h - yh mean(h yh))            dg = sum D b over the row or over t
// A row is held in the registers of TPR threads, 8 NV values each, so every
// array is read and written once.  The gradients recompute both rsqrt from the
// row (no statistics are kept between the passes): the sums ride along with
// those of q rh.
#include "device_common.h"
#include "kernels_block.h"
#include "moe_lora.h"

#include <type_traits>

namespace moe_lora {
namespace {

// Sums of N values over the TPR threads of a row, the same bits in every thread.
// Up to a wave: butterflies.  More: one value per wave through LDS; `scratch`
// holds N floats per wave of the block, two halves used in turn so that one
// barrier an exchange is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *scratch)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int off = (TPR < kWave ? TPR : kWave) / 2; off >= 1; off >>= 1)
            v[i] += __shfl_xor(v[i], off);
    if constexpr (TPR > kWave) {
        constexpr int kWaves = TPR / kWave;
        const int wave = wave_id();
        if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                scratch[wave * N + i] = v[i];
        }
        lds_barrier();
        const int first = wave / kWaves * kWaves;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                s += scratch[(first + w) * N + i];
            v[i] = s;
        }
    }
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = float_to_bf16_bits(f[2 * i]) | (float_to_bf16_bits(f[2 * i + 1]) << 16);
    return v;
}

constexpr int kBlock = 256;      // threads of a forward block (TPR where that is more)
constexpr int kGradBlock = 1024; // threads of a gradient block
constexpr int kMostBlocks = 1 << 20;  // a launch's threads stay below 2^32

template <int TPR, int NV>
__global__ __launch_bounds__(TPR > kBlock ? TPR : kBlock) void block_norm_kernel(NormArgs a)
{
    constexpr int kThreads = TPR > kBlock ? TPR : kBlock;
    constexpr int kRows = kThreads / TPR;
    __shared__ float scratch[3][kThreads / kWave];
    const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)gridDim.x * kRows) {
        const bool live = t0 + mine < a.T;   // all threads meet the barriers
        const size_t t = live ? t0 + mine : 0, row = t * a.H;
        float r[NV][8], y[NV][8];
        float sum[1] = {0.0f};
        u32x4 xv[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            const bool in = live && c < a.H;
            xv[v] = a.x && in ? load16(a.x + row + c) : zero16();
            unpack8(a.y && in ? load16(a.y + row + c) : zero16(), y[v]);
        }
        float g = a.gate_kind == MOE_LORA_GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.0f;
        if (a.w_post) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[0] = fmaf(y[v][i], y[v][i], sum[0]);
            row_sums<TPR>(sum, scratch[turn]);
            turn = turn == 2 ? 0 : turn + 1;
            g *= rsqrtf(sum[0] / a.H + a.eps);
        }
        sum[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            float x[8], w[8], gc[8];
            unpack8(xv[v], x);
            unpack8(a.w_post && c < a.H ? load16(a.w_post + c) : zero16(), w);
            unpack8(a.gate_kind == MOE_LORA_GATE_CHANNEL && c < a.H
                        ? load16(static_cast<const uint16_t *>(a.gate) + c) : zero16(), gc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float b = g * y[v][i];
                if (a.w_post)
                    b *= a.offset + w[i];
                if (a.gate_kind == MOE_LORA_GATE_CHANNEL)
                    b *= gc[i];
                r[v][i] = a.x ? (a.y ? fmaf(a.alpha, x[i], b) : a.alpha * x[i]) : b;
                sum[0] = fmaf(r[v][i], r[v][i], sum[0]);
            }
            if (a.r && live && c < a.H)
                store16(a.r + row + c, pack8(r[v]));
        }
        if (!a.z)
            continue;
        row_sums<TPR>(sum, scratch[turn]);
        turn = turn == 2 ? 0 : turn + 1;
        const float p = rsqrtf(sum[0] / a.H + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            if (live && c < a.H) {
                float w[8];
                unpack8(load16(a.w_pre + c), w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[v][i] *= p * (a.offset + w[i]);
                store16(a.z + row + c, pack8(r[v]));
            }
        }
    }
}

// Blocks walk the rows; the column sums of a thread's 8 NV columns stay in its
// registers over all its rows, are joined over the block's rows at a time
// through LDS at the end, and over the blocks by launch_column_sums.
template <int TPR, int NV>
__global__ __launch_bounds__(kGradBlock) void block_norm_backward_kernel(NormGradArgs a)
{
    constexpr int kRows = kGradBlock / TPR;
    constexpr int kColumns = TPR * 8;    // of one v
    __shared__ float scratch[3][kGradBlock / kWave * 3];
    __shared__ float columns[kRows][kColumns];
    const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
    const float inv_h = 1.0f / a.H;
    float s_post[NV][8] = {}, s_pre[NV][8] = {}, s_gate[NV][8] = {};
    const bool need_y = a.w_post || a.gate_at >= 0 || a.d_token;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)a.blocks * kRows) {
        const bool live = t0 + mine < a.T;
        const size_t t = live ? t0 + mine : 0, row = t * a.H;
        u32x4 rv[NV], yv[NV], dv[NV], zv[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            const bool in = live && c < a.H;
            rv[v] = a.dz && in ? load16(a.r + row + c) : zero16();
            zv[v] = a.dz && in ? load16(a.dz + row + c) : zero16();
            yv[v] = need_y && in ? load16(a.y + row + c) : zero16();
            dv[v] = a.dr && in ? load16(a.dr + row + c) : zero16();
        }
        const float gt = a.gate_kind == MOE_LORA_GATE_TOKEN
                             ? static_cast<const float *>(a.gate)[t] : 1.0f;
        float sums[3] = {0.0f, 0.0f, 0.0f};   // r^2, q r, y^2
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            float r[8], z[8], y[8], w[8];
            unpack8(rv[v], r);
            unpack8(zv[v], z);
            unpack8(yv[v], y);
            unpack8(a.dz && c < a.H ? load16(a.w_pre + c) : zero16(), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[0] = fmaf(r[i], r[i], sums[0]);
                sums[1] = fmaf(z[i] * (a.offset + w[i]), r[i], sums[1]);
                sums[2] = fmaf(y[i], y[i], sums[2]);
            }
        }
        row_sums<TPR>(sums, scratch[turn]);
        turn = turn == 2 ? 0 : turn + 1;
        const float p = rsqrtf(sums[0] * inv_h + a.eps);
        const float mean_q = sums[1] * p * inv_h;       // mean of q rh
        const float s = a.w_post ? rsqrtf(sums[2] * inv_h + a.eps) : 1.0f;
        float D[NV][8];
        float more[2] = {0.0f, 0.0f};                   // h yh, D b
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            const bool in = c < a.H;
            float r[8], z[8], y[8], wq[8], wp[8], gc[8];
            unpack8(rv[v], r);
            unpack8(zv[v], z);
            unpack8(yv[v], y);
            unpack8(dv[v], D[v]);
            unpack8(a.dz && in ? load16(a.w_pre + c) : zero16(), wq);
            unpack8(a.w_post && in ? load16(a.w_post + c) : zero16(), wp);
            unpack8(a.gate_kind == MOE_LORA_GATE_CHANNEL && in
                        ? load16(static_cast<const uint16_t *>(a.gate) + c) : zero16(), gc);
            float dx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (a.dz) {
                    const float rh = r[i] * p;
                    D[v][i] += p * (z[i] * (a.offset + wq[i]) - rh * mean_q);
                    s_pre[v][i] = fmaf(z[i], rh, s_pre[v][i]);
                }
                dx[i] = a.alpha * D[v][i];
                const float yh = y[i] * s;
                const float w = a.w_post ? a.offset + wp[i] : 1.0f;
                const float db = D[v][i] * (a.gate_kind == MOE_LORA_GATE_CHANNEL ? gc[i] : gt);
                more[0] = fmaf(db * w, yh, more[0]);
                more[1] = fmaf(D[v][i], yh * w, more[1]);
                s_post[v][i] = fmaf(db, yh, s_post[v][i]);
                s_gate[v][i] = fmaf(D[v][i], yh * w, s_gate[v][i]);
                D[v][i] = db * w;                       // h from here on
            }
            if (a.dx && live && in)
                store16(a.dx + row + c, pack8(dx));
        }
        if (a.w_post || a.d_token) {
            row_sums<TPR>(more, scratch[turn]);
            turn = turn == 2 ? 0 : turn + 1;
            if (a.d_token && live && lane == 0)
                a.d_token[t] = more[1];
        }
        if (a.dy && live) {
            const float mean_h = a.w_post ? more[0] * inv_h : 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * 8;
                float y[8], dy[8];
                unpack8(yv[v], y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dy[i] = a.w_post ? s * (D[v][i] - y[i] * s * mean_h) : D[v][i];
                if (c < a.H)
                    store16(a.dy + row + c, pack8(dy));
            }
        }
    }
    float *out = a.partial + (size_t)blockIdx.x * a.sums * a.H;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        const int at = which == 0 ? a.post_at : which == 1 ? a.pre_at : a.gate_at;
        if (at < 0)
            continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                columns[mine][lane * 8 + i] = which == 0 ? s_post[v][i] : which == 1 ? s_pre[v][i] : s_gate[v][i];
            __syncthreads();
            for (int c = threadIdx.x; c < kColumns; c += kGradBlock) {
                float total = 0.0f;
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    total += columns[k][c];
                if (v * kColumns + c < a.H)
                    out[(size_t)at * a.H + v * kColumns + c] = total;
            }
            __syncthreads();
        }
    }
}

// Calls f with the threads of a row and the vectors of a thread that hold H values.
template <class F>
hipError_t for_width(int H, F f)
{
    const int v = (H + 7) / 8;
    if (v <= 64)
        return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (v <= 128)
        return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    if (v <= 256)
        return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
    if (v <= 512)
        return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
    if (v <= 1024)
        return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 1>());
    if (v <= 2048)
        return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
    if (v <= 4096)
        return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 8>());
}

int threads_per_row(int H) { return H <= 1024 ? 64 : H <= 4096 ? 256 : 1024; }

} // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t s)
{
    if (a.T <= 0)
        return hipSuccess;
    return for_width(a.H, [&](auto tpr, auto nv) {
        constexpr int kThreads = tpr() > kBlock ? tpr() : kBlock;
        constexpr int kRows = kThreads / tpr();
        const int need = (a.T + kRows - 1) / kRows;
        hipLaunchKernelGGL((block_norm_kernel<tpr(), nv()>), dim3(need < kMostBlocks ? need : kMostBlocks),
                           dim3(kThreads), 0, s, a);
        return hipGetLastError();
    });
}

// One block per CU at most: each writes one row of column sums.
int norm_grad_blocks(int T, int H)
{
    const int rows = kGradBlock / threads_per_row(H);
    const int need = (T + rows - 1) / rows;
    return need < 1 ? 1 : need < 256 ? need : 256;
}

hipError_t launch_block_norm_backward(const NormGradArgs &a, hipStream_t s)
{
    return for_width(a.H, [&](auto tpr, auto nv) {
        hipLaunchKernelGGL((block_norm_backward_kernel<tpr(), nv()>), dim3(a.blocks), dim3(kGradBlock), 0,
                           s, a);
        return hipGetLastError();
    });
}

} // namespace moe_lora
