// linear_rows.hip -- the product with its epilogue for up to 64 rows, one launch:
//   out[m, n] = epilogue(sum_k x[m, k] w[k, n])
// Bound by the stream of w (and, below a few MB, by one launch and one chain of
// loads), so w goes from memory straight into MFMA operands: a lane loads CPL
// neighbouring columns of 8 terms, and one byte permutation per two weights makes
// K-contiguous fragments of them, without LDS.  The 16 waves of a block split the
// terms and are joined through LDS in a fixed order.  Any N: CPL divides it.
#include "device_common.h"
#include "kernels_block.h"
#include "linear_epilogue.h"

namespace moe_lora {
namespace {

constexpr int kWaves = 16;

// CPL columns (1, 2, 4 or 8 bf16) of one row of w as dwords
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
        } else if constexpr (CPL == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
            const u32x4 v = load16(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = v[i];
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
    __shared__ float part[kWaves][MT * 16][kStride];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int i = lane & 15, g = lane >> 4;
    const int blocks = (a.e.N + 16 * CPL - 1) / (16 * CPL);
    const int item = xcd_balanced_item(blockIdx.x, blocks);
    if (item < 0)
        return;
    const int n0 = item * 16 * CPL;
    const int c = n0 + i * CPL < a.e.N ? n0 + i * CPL : 0;   // N is a multiple of CPL
    const uint16_t *wp = a.w + c;
    const uint16_t *xp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xp[m] = a.x + (int64_t)(m * 16 + i < a.M ? m * 16 + i : a.M - 1) * a.K;

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
    // chunks wave, wave + 16, ...; the next one's loads run under this one's products
    const int chunks = (a.K + 31) / 32;
    Chunk<MT, SETS, CPL> one, two;
    one.load(xp, wp, a.e.N, a.W, wave * 32 + 8 * g, a.K);
    for (int ch = wave; ch < chunks; ch += 2 * kWaves) {
        two.load(xp, wp, a.e.N, a.W, (ch + kWaves) * 32 + 8 * g, a.K);
        multiply(one);
        one.load(xp, wp, a.e.N, a.W, (ch + 2 * kWaves) * 32 + 8 * g, a.K);
        multiply(two);
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
        if (m >= a.M || n0 + n >= a.e.N)
            continue;
        float z = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            z += part[w][m][n];
            if constexpr (SETS == 2)
                up += part[w][m][16 * CPL + n];
        }
        finish_one(a.e, m, n0 + n, z, up);
    }
}

template <int MT, int SETS, int CPL>
hipError_t launch(const RowsArgs &a, hipStream_t s)
{
    const int blocks = (a.e.N + 16 * CPL - 1) / (16 * CPL);
    hipLaunchKernelGGL((rows_kernel<MT, SETS, CPL>), dim3((blocks + 7) / 8 * 8), dim3(kWaves * 64), 0, s, a);
    return hipGetLastError();
}

// Columns a lane loads: the partial sums of 16 waves fit the LDS up to 8 / (MT SETS),
// and N is a multiple; the fewest that leave at most 256 blocks.
int columns_per_lane(int M, int N, int sets)
{
    const int mt = M <= 16 ? 1 : M <= 32 ? 2 : 4, most = 8 / (mt * sets);
    int cpl = 1;
    while (cpl < most && N % (2 * cpl) == 0 && (N + 16 * cpl - 1) / (16 * cpl) > 256)
        cpl *= 2;
    return cpl;
}

template <int MT, int SETS>
hipError_t launch_columns(const RowsArgs &a, hipStream_t s)
{
    const int cpl = columns_per_lane(a.M, a.e.N, SETS);
    if constexpr (8 / (MT * SETS) >= 8)
        if (cpl == 8)
            return launch<MT, SETS, 8>(a, s);
    if constexpr (8 / (MT * SETS) >= 4)
        if (cpl == 4)
            return launch<MT, SETS, 4>(a, s);
    if constexpr (8 / (MT * SETS) >= 2)
        if (cpl == 2)
            return launch<MT, SETS, 2>(a, s);
    return launch<MT, SETS, 1>(a, s);
}

} // namespace

bool rows_kernel_takes(int64_t M, int64_t K, int64_t N, bool gated)
{
    (void)K, (void)N, (void)gated;
    return M <= 64;
}

hipError_t launch_rows(const RowsArgs &a, hipStream_t s)
{
    const bool gated = a.e.act == MOE_LORA_ACT_SWIGLU;
    if (a.M <= 16)
        return gated ? launch_columns<1, 2>(a, s) : launch_columns<1, 1>(a, s);
    if (a.M <= 32)
        return gated ? launch_columns<2, 2>(a, s) : launch_columns<2, 1>(a, s);
    return gated ? launch_columns<4, 2>(a, s) : launch_columns<4, 1>(a, s);
}

} // namespace moe_lora
