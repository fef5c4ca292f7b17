// linear_tile.hip -- products of many rows on the matrix units:
//   out[m, n] = epilogue(sum_k Q[m, k] P[k, n])
// for the three products of a linear layer: x w, dz w^T and x^T dz.  Weights and
// activations are read as they are; where the contraction index is strided in
// memory (w in x w, both operands of x^T dz) the fragments are read from LDS with
// the transposing read, so no operand is laid out anew.
//
// A block owns a tile of BM rows and BN columns.  Steps of 64 terms of both
// operands go through two LDS buffers, written by direct global->LDS loads that
// run under the MFMAs of the step before.  D = P^T Q^T tiles: a lane then holds
// four neighbouring columns of one row, which the epilogue stores at once.
#include "block_dma.h"
#include "device_common.h"
#include "kernels_block.h"
#include "linear_epilogue.h"

namespace moe_lora {
namespace {

constexpr int kStep = 64;   // terms of a step

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// One operand's share of an LDS buffer: R outer indices (rows of the output or
// columns) by 64 terms, R * 128 bytes.
//  Contiguous: outer index r at r * 128, its eight 16-byte pieces of 8 terms
//    XOR-swizzled by bits 1..3 of r, so that the 16 rows x 16 bytes of a fragment
//    read meet every bank once.
//  Strided: term k at k * 2R, its 32-byte units of 16 outer indices XOR-swizzled by
//    bits 0, 1 and 3 of k: a transposing read takes 32 bytes of 16 terms, 8 of them
//    a half wave, which then meet every bank once.
template <int R>
__device__ __forceinline__ int unit_swizzle(int k)
{
    if constexpr (R == 64)   // two terms a bank line
        return ((k >> 1) & 1) | ((k >> 2) & 2);
    else
        return (k & 3) | ((k >> 1) & 4);
}

// Addresses of the direct loads of one operand: NT threads, R / 8 * 64 / NT pieces each.
template <int R, int NT, bool STRIDED>
struct Loader {
    static constexpr int kLoads = R * 8 / NT;
    uint32_t offset[kLoads];   // bytes from the step's base; kNone: reads as zeros
    int term[kLoads];          // first term of the piece, within the step

    // outer index `first + r`, below `count`; for STRIDED the source column of unit u
    // is given by column(u) (swiglu tiles alternate gate and up units)
    template <class Column>
    __device__ __forceinline__ void init(int tid, int first, int count, int ld, Column column)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int piece = i * NT + tid;
            if constexpr (STRIDED) {
                constexpr int kUnits = R / 16;
                const int k = piece / (R / 8), slot = piece % (R / 8);
                const int unit = (slot >> 1) ^ (unit_swizzle<R>(k) & (kUnits - 1));
                const int c = column(unit, (slot & 1) * 8);
                term[i] = k;
                offset[i] = c < 0 ? kNone : (uint32_t)(k * ld + c) * 2u;
            } else {
                const int r = piece >> 3, q = (piece & 7) ^ ((r >> 1) & 7);
                term[i] = q * 8;
                offset[i] = first + r < count ? (uint32_t)(r * ld + q * 8) * 2u : kNone;
            }
        }
    }

    // `left`: terms that remain from the step's first on
    __device__ __forceinline__ void issue(u32x4 resource, uint32_t lds, int left)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            buffer_load_lds16(resource, term[i] < left ? offset[i] : kNone, lds + i * NT * 16);
    }
};

// MFMA operand fragment of 16 outer indices and 32 terms (half h of the step).
template <int R, bool STRIDED>
__device__ __forceinline__ u32x4 fragment(const char *tile, int sixteen, int h, int lane)
{
    const int g = lane >> 4, i = lane & 15;
    if constexpr (STRIDED) {
        const int k = 32 * h + 8 * g + (i >> 2);
        const int unit = sixteen ^ (unit_swizzle<R>(k) & (R / 16 - 1));
        const char *p = tile + k * 2 * R + unit * 32 + (i & 3) * 8;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 2 * R));
        const uint2 lo = __builtin_bit_cast(uint2, a), hi = __builtin_bit_cast(uint2, b);
        return u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
        const int r = sixteen * 16 + i;
        return *reinterpret_cast<const u32x4 *>(tile + r * 128 + (((4 * h + g) ^ ((r >> 1) & 7)) * 16));
    }
}

// WM x WN waves share the tile; GATED: columns are swiglu pairs, the tile's units
// of 16 alternate gate and up columns, BN / 2 outputs wide.
template <int BM, int BN, int WM, int WN, bool QS, bool PS, bool GATED, bool SPLIT>
__global__ __launch_bounds__(WM *WN * 64, BM * BN * WM * WN >= 256 * 256 * 8 ? 2 : 2)
void product_kernel(ProductArgs a)
{
    constexpr int NT = WM * WN * 64;
    constexpr int kQ = BM * 128, kP = BN * 128, kBuffer = kQ + kP;
    constexpr int MT = BM / WM / 16, NTL = BN / WN / 16;
    __shared__ __attribute__((aligned(1024))) char lds[2 * kBuffer];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();

    // consecutive tiles of one XCD are neighbours in both directions
    const int tiles = a.tiles_m * a.tiles_n;
    const int item = xcd_balanced_item(blockIdx.x, tiles * a.splits);
    if (item < 0)
        return;
    const int split = item / tiles, tile = item - split * tiles;
    constexpr int kBand = 8;
    const int band = tile / (kBand * a.tiles_n);
    const int band_rows = a.tiles_m - band * kBand < kBand ? a.tiles_m - band * kBand : kBand;
    const int inside = tile - band * kBand * a.tiles_n;
    const int tm = band * kBand + inside % band_rows, tn = inside / band_rows;
    const int m0 = tm * BM, n0 = tn * (GATED ? BN / 2 : BN);
    const int k0 = split * a.k_per;
    const int K = a.K - k0 < a.k_per ? a.K - k0 : a.k_per;
    const int steps = (K + kStep - 1) / kStep;

    // rows a tile does not have read as zeros
    Loader<BM, NT, QS> lq;
    Loader<BN, NT, PS> lp;
    lq.init(tid, m0, a.M, a.ldq, [&](int unit, int c) {
        const int m = m0 + unit * 16 + c;
        return m < a.M ? unit * 16 + c : -1;   // M is a multiple of 8 where it is contiguous
    });
    lp.init(tid, n0, a.C, a.ldp, [&](int unit, int c) {
        if constexpr (GATED) {
            const int n = n0 + (unit >> 1) * 16 + c;
            return n < a.e.half ? (unit & 1) * a.e.half + (unit >> 1) * 16 + c : -1;
        } else {
            const int n = n0 + unit * 16 + c;
            return n < a.C ? unit * 16 + c : -1;
        }
    });
    const char *q = reinterpret_cast<const char *>(a.Q + (QS ? (size_t)k0 * a.ldq + m0 : (size_t)m0 * a.ldq + k0));
    const char *p = reinterpret_cast<const char *>(a.P + (PS ? (size_t)k0 * a.ldp + n0 : (size_t)n0 * a.ldp + k0));
    const size_t q_step = QS ? (size_t)kStep * a.ldq * 2 : kStep * 2;
    const size_t p_step = PS ? (size_t)kStep * a.ldp * 2 : kStep * 2;
    const uint32_t base = lds_base(lds) + wave * 1024;

    auto issue = [&](int s) {
        const uint32_t at = base + (s & 1) * kBuffer;
        lq.issue(buffer_resource(q + s * q_step), at, K - s * kStep);
        lp.issue(buffer_resource(p + s * p_step), at + kQ, K - s * kStep);
    };

    f32x4 acc[MT][NTL];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NTL; ++n)
            acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int wm = wave / WN * MT, wn = wave % WN * NTL;   // in sixteens

    issue(0);
    landed_barrier();
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps)
            issue(s + 1);
        const char *tq = lds + (s & 1) * kBuffer, *tp = tq + kQ;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 fp[NTL];
#pragma unroll
            for (int n = 0; n < NTL; ++n)
                fp[n] = fragment<BN, PS>(tp, wn + n, h, lane);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const u32x4 fq = fragment<BM, QS>(tq, wm + m, h, lane);
#pragma unroll
                for (int n = 0; n < NTL; ++n)
                    acc[m][n] = mfma_16x16x32(fp[n], fq, acc[m][n]);
            }
        }
        landed_barrier();
    }

    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t row = m0 + (wm + m) * 16 + i;
        if (row >= a.M)
            continue;
        if constexpr (SPLIT) {
            float *out = a.partial + ((size_t)split * a.M + row) * a.C;
#pragma unroll
            for (int n = 0; n < NTL; ++n) {
                const int c = n0 + (wn + n) * 16 + 4 * g;
                if (c < a.C)   // C is a multiple of 8
                    *reinterpret_cast<f32x4 *>(out + c) = acc[m][n];
            }
        } else {
#pragma unroll
            for (int n = 0; n < NTL; n += GATED ? 2 : 1) {
                float z[4], up[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z[j] = acc[m][n][j];
                    up[j] = GATED ? acc[m][n + (GATED ? 1 : 0)][j] : 0.0f;
                }
                finish_four(a.e, row, n0 + (GATED ? (wn + n) / 2 : wn + n) * 16 + 4 * g, z, up);
            }
        }
    }
}

// Sums the splits and finishes: a thread per four columns of a row.
__global__ __launch_bounds__(256) void join_kernel(ProductArgs a)
{
    const bool gated = a.e.act == MOE_LORA_ACT_SWIGLU;
    const int width = gated ? a.e.half : a.C;
    const int per_row = width / 4;
    const int64_t items = (int64_t)a.M * per_row;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < items; x += (int64_t)gridDim.x * 256) {
        const int64_t m = x / per_row;
        const int n = (int)(x - m * per_row) * 4;
        const float *in = a.partial + m * a.C + n;
        f32x4 z = {}, up = {};
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            z += *reinterpret_cast<const f32x4 *>(in + (size_t)s * a.M * a.C);
            if (gated)
                up += *reinterpret_cast<const f32x4 *>(in + (size_t)s * a.M * a.C + a.e.half);
        }
        float zs[4] = {z[0], z[1], z[2], z[3]}, us[4] = {up[0], up[1], up[2], up[3]};
        finish_four(a.e, m, n, zs, us);
    }
}

struct Tile {
    int rows, columns;
};
constexpr Tile kTiles[] = {{256, 256}, {128, 128}, {64, 64}};

template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(Product kind, const ProductArgs &a, hipStream_t s)
{
    const bool gated = kind == Product::forward && a.e.act == MOE_LORA_ACT_SWIGLU;
    const int64_t items = (int64_t)a.tiles_m * a.tiles_n * a.splits;
    const dim3 grid((items + 7) / 8 * 8), block(WM * WN * 64);
#define MOE_LAUNCH(QS, PS, GATED, SPLIT) \
    hipLaunchKernelGGL((product_kernel<BM, BN, WM, WN, QS, PS, GATED, SPLIT>), grid, block, 0, s, a)
    if (kind == Product::forward) {
        if (a.splits > 1)
            MOE_LAUNCH(false, true, false, true);
        else if (gated)
            MOE_LAUNCH(false, true, true, false);
        else
            MOE_LAUNCH(false, true, false, false);
    } else if (kind == Product::input_grad) {
        if (a.splits > 1)
            MOE_LAUNCH(false, false, false, true);
        else
            MOE_LAUNCH(false, false, false, false);
    } else {
        if (a.splits > 1)
            MOE_LAUNCH(true, true, false, true);
        else
            MOE_LAUNCH(true, true, false, false);
    }
#undef MOE_LAUNCH
    return hipGetLastError();
}

} // namespace

ProductPlan plan_product(Product kind, int64_t M, int64_t C, int64_t K, bool gated)
{
    auto tiles_of = [&](const Tile &t) { return ((M + t.rows - 1) / t.rows) * ((C + t.columns - 1) / t.columns); };
    int tile = 2;
    if (tiles_of(kTiles[0]) >= 192)
        tile = 0;
    else if (tiles_of(kTiles[1]) >= 128)
        tile = 1;
    ProductPlan p{};
    p.tile = tile;
    const int64_t tiles = tiles_of(kTiles[tile]);
    int64_t splits = 1;
    if (tiles < 192) {
        splits = 512 / tiles;
        const int64_t most = K / 256;   // four steps a split at least
        splits = splits < most ? splits : most;
        splits = splits < 1 ? 1 : splits;
    }
    const int64_t steps = (K + kStep - 1) / kStep;
    const int64_t per = (steps + splits - 1) / splits;
    p.splits = (int)((steps + per - 1) / per);
    p.k_per = (int)(per * kStep);
    const bool pairs = gated && p.splits == 1;
    p.tiles_m = (int)((M + kTiles[tile].rows - 1) / kTiles[tile].rows);
    const int64_t width = pairs ? C / 2 : C, columns = pairs ? kTiles[tile].columns / 2 : kTiles[tile].columns;
    p.tiles_n = (int)((width + columns - 1) / columns);
    return p;
}

hipError_t launch_product(Product kind, const ProductPlan &plan, const ProductArgs &given, hipStream_t s)
{
    ProductArgs a = given;
    a.tiles_m = plan.tiles_m;
    a.tiles_n = plan.tiles_n;
    a.splits = plan.splits;
    a.k_per = plan.k_per;
    hipError_t rc = plan.tile == 0   ? launch_tile<256, 256, 2, 4>(kind, a, s)
                    : plan.tile == 1 ? launch_tile<128, 128, 2, 2>(kind, a, s)
                                     : launch_tile<64, 64, 2, 2>(kind, a, s);
    if (rc != hipSuccess || a.splits == 1)
        return rc;
    const bool gated = kind == Product::forward && a.e.act == MOE_LORA_ACT_SWIGLU;
    const int64_t items = (int64_t)a.M * ((gated ? a.e.half : a.C) / 4);
    const int64_t blocks = (items + 255) / 256;
    hipLaunchKernelGGL(join_kernel, dim3(blocks < 1 << 20 ? blocks : 1 << 20), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe_lora
