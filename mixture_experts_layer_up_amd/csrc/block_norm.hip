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
// array is read and written once.  The gradients take both rsqrt from the row again:
// no statistics are kept between the passes.
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
// threads of a gradient block: about 512, whole rows
template <int TPR>
constexpr int kGradBlock = 512 / TPR * TPR;
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
        const bool live = t0 + mine < a.T;   // every thread meets the barriers
        const size_t t = live ? t0 + mine : 0, row = t * a.H;
        int at = lane * 8;
        if constexpr (NV > 4)   // addresses are found in their turn, not kept for all rows
            asm("" : "+v"(at));
        float r[NV][8];
        float sum[1] = {0.0f};
        u32x4 xv[NV], yv[NV];   // as they are until their turn: 64 values a thread fit its registers so
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR * 8 + at;
            const bool in = live && c < a.H;
            xv[v] = a.x && in ? load16(a.x + row + c) : zero16();
            yv[v] = a.y && in ? load16(a.y + row + c) : zero16();
        }
        float g = a.gate_kind == MOE_LORA_GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.0f;
        if (a.w_post) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float y[8];
                unpack8(yv[v], y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[0] = fmaf(y[i], y[i], sum[0]);
            }
            row_sums<TPR>(sum, scratch[turn]);
            turn = turn == 2 ? 0 : turn + 1;
            g *= rsqrtf(sum[0] / a.H + a.eps);
        }
        sum[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * TPR * 8 + at;
            float x[8], y[8], w[8], gc[8];
            unpack8(xv[v], x);
            if constexpr (NV > 4)   // unpacked again, not kept from the sum of squares
                asm("" : "+v"(yv[v]));
            unpack8(yv[v], y);
            unpack8(a.w_post && c < a.H ? load16(a.w_post + c) : zero16(), w);
            unpack8(a.gate_kind == MOE_LORA_GATE_CHANNEL && c < a.H
                        ? load16(static_cast<const uint16_t *>(a.gate) + c) : zero16(), gc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float b = g * y[i];
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
            const int c = v * TPR * 8 + at;
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

// The six sums of a row (below) from eight of its columns.
__device__ __forceinline__ void add_sums(float (&sums)[6], const float (&r)[8], const float (&z)[8],
                                         const float (&y)[8], const float (&d)[8], const float (&wq)[8],
                                         const float (&wp)[8], const float (&g)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = z[i] * wq[i], v = g[i] * wp[i] * y[i];
        sums[0] = fmaf(r[i], r[i], sums[0]);
        sums[1] = fmaf(q, r[i], sums[1]);
        sums[2] = fmaf(y[i], y[i], sums[2]);
        sums[3] = fmaf(d[i], v, sums[3]);
        sums[4] = fmaf(q, v, sums[4]);
        sums[5] = fmaf(r[i], v, sums[5]);
    }
}

__device__ __forceinline__ void row_values(const NormGradArgs &a, const float (&sums)[6], float &p,
                                           float &mean_q, float &s, float &db)
{
    const float inv_h = 1.0f / a.H;
    p = rsqrtf(sums[0] * inv_h + a.eps);
    mean_q = a.dz ? sums[1] * p * inv_h : 0.0f;
    s = a.w_post ? rsqrtf(sums[2] * inv_h + a.eps) : 1.0f;
    db = s * (sums[3] + p * (sums[4] - p * mean_q * sums[5]));
}

// o + w_pre (0 without dz), o + w_post (or 1) and the channel gate (or 1) of eight columns.
__device__ __forceinline__ void column_weights(const NormGradArgs &a, int c, float (&wq)[8], float (&wp)[8],
                                               float (&g)[8])
{
    const bool in = c < a.H, channel = a.gate_kind == MOE_LORA_GATE_CHANNEL;
    unpack8(a.dz && in ? load16(a.w_pre + c) : zero16(), wq);
    unpack8(a.w_post && in ? load16(a.w_post + c) : zero16(), wp);
    unpack8(channel && in ? load16(static_cast<const uint16_t *>(a.gate) + c) : zero16(), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        wq[i] = a.dz ? a.offset + wq[i] : 0.0f;
        wp[i] = a.w_post ? a.offset + wp[i] : 1.0f;
        g[i] = channel ? g[i] : 1.0f;
    }
}

// {p, m, s, D b} of every row, and the token gate's gradient: a block a row.
__global__ __launch_bounds__(1024) void row_stats_kernel(NormGradArgs a)
{
    __shared__ float scratch[2][16 * 6];
    const bool need_y = a.w_post || a.gate_at >= 0 || a.d_token;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = (size_t)t * a.H;
        float sums[6] = {};
        for (int c = threadIdx.x * 8; c < a.H; c += 1024 * 8) {
            float r[8], z[8], y[8], d[8], wq[8], wp[8], g[8];
            unpack8(a.dz ? load16(a.r + row + c) : zero16(), r);
            unpack8(a.dz ? load16(a.dz + row + c) : zero16(), z);
            unpack8(need_y ? load16(a.y + row + c) : zero16(), y);
            unpack8(a.dr ? load16(a.dr + row + c) : zero16(), d);
            column_weights(a, c, wq, wp, g);
            add_sums(sums, r, z, y, d, wq, wp, g);
        }
        row_sums<1024>(sums, scratch[turn]);
        turn ^= 1;
        if (threadIdx.x == 0) {
            float p, m, s, db;
            row_values(a, sums, p, m, s, db);
            a.stats[t] = float4{p, m, s, db};
            if (a.d_token)
                a.d_token[t] = db;
        }
    }
}

// Blocks walk the rows.  The two means are combined from six sums that need nothing but the row itself, so a row meets
// its block once:
//   S0 = sum r^2, S1 = sum q r, S2 = sum y^2, S3 = sum dr v, S4 = sum q v, S5 = sum r v
// with v = g (o + w_post) y per channel, and then
//   mean(q rh) = p S1 / H =: m,   sum of D g (o + w_post) yh = s (S3 + p S4 - p^2 m S5).
// The column sums of a thread's 8 NV columns stay in its registers over all its rows,
// are joined over the block's rows at a time through LDS at the end, and over the
// blocks by launch_column_sums.  Memory bound: 8192 rows of 2048, everything asked for,
// 201 MB in 41 us (4.9 TB/s, the rate of a large copy) and 4.7 us for the joining.  Two
// blocks a CU, so that one loads while the other reduces: a block of 1024 threads a CU
// 43 us, with the next row loaded ahead 54 (registers spill).
// WIDE: rows of more than 8192 columns.  A block takes 4096 of a row's columns
// (blockIdx.y) and finds the row's sums in `stats`, which row_stats_kernel wrote: it may
// write over its own part of an input, but no other block's.
template <int TPR, int NV, bool WIDE>
__global__ __launch_bounds__(kGradBlock<TPR>, NV == 1 ? 4 : 2)
void block_norm_backward_kernel(NormGradArgs a)
{
    constexpr int kThreads = kGradBlock<TPR>, kRows = kThreads / TPR;
    constexpr int kColumns = TPR * 8;    // of one v
    __shared__ float scratch[2][(kThreads + kWave - 1) / kWave * 6];
    __shared__ float columns[kRows][kColumns];
    const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
    const float inv_h = 1.0f / a.H;
    float s_post[NV][8] = {}, s_pre[NV][8] = {}, s_gate[NV][8] = {};
    const bool need_y = a.w_post || a.gate_at >= 0 || a.d_token;
    const bool channel = a.gate_kind == MOE_LORA_GATE_CHANNEL;
    struct Row {
        u32x4 r[NV], y[NV], d[NV], z[NV];
    };
    const int first = WIDE ? (int)blockIdx.y * kColumns : 0;   // column
    auto load = [&](Row &w, int64_t t) {
        const bool live = t < a.T;
        const size_t row = (size_t)(live ? t : 0) * a.H;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = first + (v * TPR + lane) * 8;
            const bool in = live && c < a.H;
            w.r[v] = a.dz && in ? load16(a.r + row + c) : zero16();
            w.z[v] = a.dz && in ? load16(a.dz + row + c) : zero16();
            w.y[v] = need_y && in ? load16(a.y + row + c) : zero16();
            w.d[v] = a.dr && in ? load16(a.dr + row + c) : zero16();
        }
    };
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)a.blocks * kRows) {
        Row now;
        load(now, t0 + mine);
        const bool live = t0 + mine < a.T;
        const size_t t = live ? t0 + mine : 0, row = t * a.H;
        const float gt = a.gate_kind == MOE_LORA_GATE_TOKEN ? static_cast<const float *>(a.gate)[t] : 1.0f;
        float p, mean_q, s, db;   // db: D b over the gate of tokens
        if constexpr (WIDE) {
            const float4 st = a.stats[t];
            p = st.x, mean_q = st.y, s = st.z, db = st.w;
        } else {
            float sums[6] = {};
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float r[8], z[8], y[8], d[8], wq[8], wp[8], g[8];
                unpack8(now.r[v], r);
                unpack8(now.z[v], z);
                unpack8(now.y[v], y);
                unpack8(now.d[v], d);
                column_weights(a, (v * TPR + lane) * 8, wq, wp, g);
                add_sums(sums, r, z, y, d, wq, wp, g);
            }
            row_sums<TPR>(sums, scratch[turn]);
            turn ^= 1;
            row_values(a, sums, p, mean_q, s, db);
        }
        const float mean_h = a.w_post ? gt * db * inv_h : 0.0f;
        int at = lane * 8;
        if constexpr (TPR == 512)   // the outputs' addresses are found here, not kept for all rows
            asm("" : "+v"(at));
        if (!WIDE && a.d_token && live && lane == 0)
            a.d_token[t] = db;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = first + v * TPR * 8 + at;
            float r[8], z[8], y[8], D[8], wq[8], wp[8], g[8], dx[8], dy[8];
            unpack8(now.r[v], r);
            unpack8(now.z[v], z);
            unpack8(now.y[v], y);
            unpack8(now.d[v], D);
            column_weights(a, c, wq, wp, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (a.dz) {
                    const float rh = r[i] * p;
                    D[i] += p * (z[i] * wq[i] - rh * mean_q);
                    s_pre[v][i] = fmaf(z[i], rh, s_pre[v][i]);
                }
                dx[i] = a.alpha * D[i];
                const float yh = y[i] * s, dB = D[i] * (channel ? g[i] : gt);
                s_post[v][i] = fmaf(dB, yh, s_post[v][i]);
                s_gate[v][i] = fmaf(D[i], yh * wp[i], s_gate[v][i]);
                dy[i] = a.w_post ? s * (dB * wp[i] - yh * mean_h) : dB;
            }
            if (live && c < a.H) {
                if (a.dx)
                    store16(a.dx + row + c, pack8(dx));
                if (a.dy)
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
            for (int c = threadIdx.x; c < kColumns; c += kThreads) {
                float total = 0.0f;
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    total += columns[k][c];
                if (first + v * kColumns + c < a.H)
                    out[(size_t)at * a.H + first + v * kColumns + c] = total;
            }
            __syncthreads();
        }
    }
}

template <int I>
using Int = std::integral_constant<int, I>;

// Calls f with the threads of a row and the vectors of a thread that hold H values.
template <class F>
hipError_t for_width(int H, F f)
{
    const int v = (H + 7) / 8;
    return v <= 8      ? f(Int<8>(), Int<1>())
           : v <= 16   ? f(Int<16>(), Int<1>())
           : v <= 32   ? f(Int<32>(), Int<1>())
           : v <= 64   ? f(Int<64>(), Int<1>())
           : v <= 128  ? f(Int<64>(), Int<2>())
           : v <= 256  ? f(Int<256>(), Int<1>())
           : v <= 512  ? f(Int<256>(), Int<2>())
           : v <= 1024 ? f(Int<1024>(), Int<1>())
           : v <= 2048 ? f(Int<1024>(), Int<2>())
           : v <= 4096 ? f(Int<1024>(), Int<4>())
                       : f(Int<1024>(), Int<8>());
}

// The same for the gradients.  A thread's column sums take 24 registers a vector, so one
// vector a thread as far as a block goes, and whole waves no wider than the row needs
// (2112 columns by 512 threads: 67 us for 16.8 M values, by 320: 60).
template <class F>
hipError_t for_grad_width(int H, F f)
{
    const int v = (H + 7) / 8;
    if (v <= 512)
        return v <= 8     ? f(Int<8>(), Int<1>())
               : v <= 16  ? f(Int<16>(), Int<1>())
               : v <= 32  ? f(Int<32>(), Int<1>())
               : v <= 64  ? f(Int<64>(), Int<1>())
               : v <= 128 ? f(Int<128>(), Int<1>())
               : v <= 192 ? f(Int<192>(), Int<1>())
               : v <= 256 ? f(Int<256>(), Int<1>())
               : v <= 320 ? f(Int<320>(), Int<1>())
               : v <= 384 ? f(Int<384>(), Int<1>())
               : v <= 448 ? f(Int<448>(), Int<1>())
                          : f(Int<512>(), Int<1>());
    return v <= 640   ? f(Int<320>(), Int<2>())
           : v <= 768 ? f(Int<384>(), Int<2>())
           : v <= 896 ? f(Int<448>(), Int<2>())
                      : f(Int<512>(), Int<2>());
}

bool wide(int H) { return H > 8192; }

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

// As many blocks as the CUs hold: each writes one row of column sums.
int norm_grad_blocks(int T, int H)
{
    int rows = 1, most = 128;   // times H / 4096
    if (!wide(H)) {
        most = H <= 4096 ? 512 : 256;
        for_grad_width(H, [&](auto tpr, auto) {
            rows = kGradBlock<tpr()> / tpr();
            return hipSuccess;
        });
    }
    const int need = (T + rows - 1) / rows;
    return need < 1 ? 1 : need < most ? need : most;
}

size_t norm_grad_stats_bytes(int T, int H) { return wide(H) ? (size_t)T * sizeof(float4) : 0; }

hipError_t launch_block_norm_backward(const NormGradArgs &a, hipStream_t s)
{
    if (wide(a.H)) {
        if (a.T > 0) {
            hipLaunchKernelGGL(row_stats_kernel, dim3(a.T < kMostBlocks ? a.T : kMostBlocks), dim3(1024), 0, s, a);
            const hipError_t rc = hipGetLastError();
            if (rc != hipSuccess)
                return rc;
        }
        hipLaunchKernelGGL((block_norm_backward_kernel<512, 1, true>), dim3(a.blocks, (a.H + 4095) / 4096),
                           dim3(512), 0, s, a);
        return hipGetLastError();
    }
    return for_grad_width(a.H, [&](auto tpr, auto nv) {
        hipLaunchKernelGGL((block_norm_backward_kernel<tpr(), nv(), false>), dim3(a.blocks),
                           dim3(kGradBlock<tpr()>), 0, s, a);
        return hipGetLastError();
    });
}

} // namespace moe_lora
