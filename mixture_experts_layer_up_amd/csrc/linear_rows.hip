// linear_rows.hip -- the product with its epilogue for few rows or few outputs, one
// launch:
//   out[m, n] = epilogue(sum_k x[m, k] w[k, n])
// Bound by the stream of w (1 row of 4096 x 16384 weights: 21.5 us, 6.2 TB/s) or, below
// a few MB, by one launch, one chain of loads and the joining (1 row in graph replays:
// 2048 x 1536 3.8 us, 2048 x (2 x 768) for swiglu, half as many blocks of twice the weights, 5.0),
// so w goes from memory straight into MFMA operands: a lane loads CPL neighbouring
// columns of 8 terms, and one byte permutation per two weights makes K-contiguous
// fragments of them, without LDS.  The 16 waves of a block split the
// terms and are joined through LDS in a fixed order.  Any N: CPL divides it.
#include "device_common.h"
#include "kernels_block.h"
#include "linear_epilogue.h"

namespace moe_lora {
namespace {

constexpr int kWaves = 16;

// CPL columns (1, 2 or 4 bf16) of one row of w as dwords
template <int CPL>
struct Columns {
    static constexpr int kWords = CPL < 2 ? 1 : CPL / 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const uint16_t *p)
    {
        if constexpr (CPL == 1) {
            w[0] = *p;
        } else if constexpr (CPL == 2) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x;
            w[1] = v.y;
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = 0;
    }
};

// What a lane loads for 32 terms: 8 rows of w, and 8 terms of each row of x
template <int MT, int SETS, int CPL>
struct Chunk {
    Columns<CPL> w[SETS][8];
    u32x4 x[MT];

    __device__ __forceinline__ void load(const uint16_t *const (&xp)[MT], const uint16_t *wp, int64_t set,
                                         int64_t W, int k, int K)
    {
        if (k < K) {   // K is a multiple of 8
#pragma unroll
            for (int s = 0; s < SETS; ++s)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[s][j].load(wp + s * set + (int64_t)(k + j) * W);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                x[m] = load16(xp[m] + k);
        } else {
#pragma unroll
            for (int s = 0; s < SETS; ++s)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[s][j].zero();
#pragma unroll
            for (int m = 0; m < MT; ++m)
                x[m] = zero16();
        }
    }

    // column c of set s as 8 consecutive terms
    __device__ __forceinline__ u32x4 fragment(int s, int c) const
    {
        u32x4 f;
        const uint32_t halves = (c & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __builtin_amdgcn_perm(w[s][2 * i + 1].w[c / 2], w[s][2 * i].w[c / 2], halves);
        return f;
    }
};

template <int MT, int SETS, int CPL>
__global__ __launch_bounds__(kWaves * 64) void rows_kernel(RowsArgs a)
{
    constexpr int kColumns = SETS * CPL * 16;     // sums of a row, set after set
    constexpr int kStride = kColumns + 4;         // rows of a column meet different banks
    // chunks in flight: as many as leave a wave within its 128 registers
    constexpr int kAhead = SETS * 8 * Columns<CPL>::kWords + 4 * MT <= 20 ? 4 : 2;
    __shared__ float part[kWaves][MT * 16][kStride];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int i = lane & 15, g = lane >> 4;
    const int column_blocks = (a.e.N + 16 * CPL - 1) / (16 * CPL), row_blocks = (a.M + 16 * MT - 1) / (16 * MT);
    const int item = xcd_balanced_item(blockIdx.x, column_blocks * row_blocks);
    if (item < 0)
        return;
    // the row blocks of one column block are neighbours: they share its columns of w
    const int n0 = item / row_blocks * 16 * CPL, m0 = item % row_blocks * 16 * MT;
    const int c = n0 + i * CPL < a.e.N ? n0 + i * CPL : 0;   // N is a multiple of CPL
    const uint16_t *wp = a.w + c;
    const uint16_t *xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xp[m] = a.x + (int64_t)(m0 + m * 16 + i < a.M ? m0 + m * 16 + i : a.M - 1) * a.K;

    f32x4 acc[MT][SETS * CPL];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int f = 0; f < SETS * CPL; ++f)
            acc[m][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Chunk<MT, SETS, CPL> &ch) {
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int f = 0; f < CPL; ++f) {
                const u32x4 fw = ch.fragment(s, f);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[m][s * CPL + f] = mfma_16x16x32(fw, ch.x[m], acc[m][s * CPL + f]);
            }
    };
    // chunks wave, wave + 16, ...; past the last they are zeros
    const int chunks = (a.K + 31) / 32;
    Chunk<MT, SETS, CPL> ring[kAhead];
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
        ring[d].load(xp, wp, a.e.N, a.W, (wave + d * kWaves) * 32 + 8 * g, a.K);
    for (int ch = wave; ch < chunks; ch += kAhead * kWaves) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            multiply(ring[d]);
            ring[d].load(xp, wp, a.e.N, a.W, (ch + (kAhead + d) * kWaves) * 32 + 8 * g, a.K);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int f = 0; f < CPL; ++f)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    part[wave][m * 16 + i][s * CPL * 16 + (4 * g + r) * CPL + f] = acc[m][s * CPL + f][r];
    __syncthreads();
    constexpr int kOut = MT * 16 * 16 * CPL;
    for (int e = threadIdx.x; e < kOut; e += kWaves * 64) {
        const int m = e / (16 * CPL), n = e % (16 * CPL);
        if (m0 + m >= a.M || n0 + n >= a.e.N)
            continue;
        float z = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            z += part[w][m][n];
            if constexpr (SETS == 2)
                up += part[w][m][16 * CPL + n];
        }
        finish_one(a.e, m0 + m, n0 + n, z, up);
    }
}

template <int MT, int SETS, int CPL>
hipError_t launch(const RowsArgs &a, hipStream_t s)
{
    const int blocks = ((a.e.N + 16 * CPL - 1) / (16 * CPL)) * ((a.M + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((rows_kernel<MT, SETS, CPL>), dim3((blocks + 7) / 8 * 8), dim3(kWaves * 64), 0, s, a);
    return hipGetLastError();
}

// Microseconds of a block on a CU that runs others too: its reduction and epilogue,
// and its terms.  Fitted to 64 to 1000 rows, 64 to 2048 terms and 128 to 4096 columns
// within a fifth; a chip with fewer blocks than CUs is up to twice as fast.  The second
// pair: of swiglu, whose blocks have two projections.  It counts where a CU runs several;
// alone on one such a block takes about as long as the others' among their like (240 shapes of
// 17 to 1000 rows, 64 to 2048 terms and 8 to 2048 columns, tiles included: 1493 us in all,
// with the first pair alone 1509, the best of each 1463; 333 rows, 2048 terms, 768 columns
// 15.2 -> 9.7).
struct Body {
    int mt, cpl;
    float fixed, term;
    float fixed_two, term_two;
};
constexpr Body kBodies[] = {{1, 1, 0.8f, 0.0017f, 1.4f, 0.0025f},
                            {1, 2, 1.0f, 0.0014f, 1.7f, 0.0022f},
                            {2, 1, 1.2f, 0.0026f, 1.3f, 0.0033f},
                            {2, 2, 1.3f, 0.0019f, 1.75f, 0.0029f}};

template <int SETS>
hipError_t launch_sets(const RowsPlan &p, const RowsArgs &a, hipStream_t s)
{
    if (p.mt == 2)
        return p.cpl == 2 ? launch<2, SETS, 2>(a, s) : launch<2, SETS, 1>(a, s);
    return p.cpl == 4   ? launch<1, SETS, 4>(a, s)
           : p.cpl == 2 ? launch<1, SETS, 2>(a, s)
                        : launch<1, SETS, 1>(a, s);
}

} // namespace

// Up to 16 rows w is read once whatever the width: 4 columns a lane then stream it best
// (1 row, 4096 x 16384: 21.5 us, two columns 25).  For few blocks one column a lane is
// best, which gives twice as many (32 rows, 2048 x 60: 4.7, two 7.2).
RowsPlan plan_rows(int64_t M, int64_t K, int64_t N, int sets)
{
    RowsPlan best{0, 0, 0.0f};
    for (const Body &b : kBodies) {
        if (N % b.cpl != 0 || (b.mt > 1 && M <= 16))
            continue;
        const int64_t blocks = ((N + 16 * b.cpl - 1) / (16 * b.cpl)) * ((M + 16 * b.mt - 1) / (16 * b.mt));
        const int64_t rounds = (blocks + 255) / 256;
        const bool two = sets == 2 && rounds > 1;
        const float us = 2.0f + (float)rounds * (two ? b.fixed_two + b.term_two * K : b.fixed + b.term * K);
        if (blocks < 1 << 20 && (best.mt == 0 || us < best.us))
            best = {b.mt, b.cpl, us};
        if (b.mt == 1 && b.cpl == 1 && blocks <= 128)
            return best;
    }
    if (M <= 16 && N % 4 == 0 && N > 16 * 2 * 256)
        best = {1, 4, 0.0f};
    return best;
}

hipError_t launch_rows(const RowsPlan &plan, const RowsArgs &a, hipStream_t s)
{
    return a.e.act == MOE_LORA_ACT_SWIGLU ? launch_sets<2>(plan, a, s) : launch_sets<1>(plan, a, s);
}

} // namespace moe_lora
