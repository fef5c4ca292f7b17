// linear_tile.hip -- products of many rows on the matrix units:
//   out[m, n] = epilogue(sum_k Q[m, k] P[k, n])
// for the three products of a linear layer: x w, dz w^T and x^T dz.  Weights and
// activations are read as they are; where the contraction index is strided in
// memory (w in x w, both operands of x^T dz) the fragments are read from LDS with
// the transposing read, so no operand is laid out anew.
//
// A block owns a tile of BM rows and BN columns.  Steps of 64 terms of both
// operands go through a ring of STAGES LDS buffers, written by direct global->LDS
// loads; the fragments of 32 terms are read from LDS under the MFMAs of the 32
// before, so a buffer is free for the loads after next half way through its step.  The fragments give
// D^T: a lane holds four neighbouring columns of one row.
#include "block_dma.h"
#include "device_common.h"
#include "kernels_block.h"
#include "linear_epilogue.h"

namespace moe_lora {
namespace {

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// One operand's share of an LDS buffer: R outer indices (rows of the output or
// columns) by 64 terms, R * 128 bytes.
//  Contiguous: outer index r at r * 128, its eight 16-byte pieces of 8 terms
//    XOR-swizzled by bits 1..3 of r, so that the 16 rows x 16 bytes of a fragment
//    read meet every bank once.  A row's share of a step is a whole 128-byte line:
//    with steps of 32 terms the loads alone took 81 us instead of 71 for 8192 x 2048
//    outputs of 4096 terms.
//  Strided: term k at k * 2R, its 32-byte units of 16 outer indices XOR-swizzled by
//    bits 0, 1 and 3 of k: a transposing read takes 32 bytes of 16 terms, 8 of them
//    a half wave, which then meet every bank once.
constexpr int BK = 64;   // terms of a step

__device__ __forceinline__ int piece_swizzle(int r) { return (r >> 1) & 7; }

template <int R>
__device__ __forceinline__ int unit_swizzle(int k)
{
    if constexpr (R == 64)   // two terms a bank line
        return ((k >> 1) & 1) | ((k >> 2) & 2);
    else
        return (k & 3) | ((k >> 1) & 4);
}

// Addresses of the direct loads of one operand: NT threads, R * BK / 8 / NT pieces each.
template <int R, int NT, bool STRIDED>
struct Loader {
    static constexpr int kLoads = R * BK / 8 / NT;
    static_assert(kLoads * NT * 8 == R * BK, "whole pieces for every thread");
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
                constexpr int kPieces = BK / 8;
                const int r = piece / kPieces, q = (piece % kPieces) ^ piece_swizzle(r);
                term[i] = q * 8;
                offset[i] = first + r < count ? (uint32_t)(r * ld + q * 8) * 2u : kNone;
            }
        }
    }

    // `left`: terms that remain from the step's first on
    __device__ __forceinline__ void issue(int i, u32x4 resource, uint32_t lds, int left) const
    {
        buffer_load_lds16(resource, term[i] < left ? offset[i] : kNone, lds + i * NT * 16);
    }
};

// MFMA operand fragment of 16 outer indices and 32 terms (half h of a step).
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
        return *reinterpret_cast<const u32x4 *>(tile + r * BK * 2 + ((4 * h + g) ^ piece_swizzle(r)) * 16);
    }
}

enum Store {
    kPartial,  // fp32 sums of a split
    kPlain,    // bf16, nothing else, C a multiple of 8
    kFull,     // the epilogue
    kGated     // the epilogue of swiglu pairs: the tile's units of 16 columns alternate gate
               // and up, it is BN / 2 outputs wide
};

// LDS of a block: its ring of buffers, and after the loop the waves' slabs.
template <int BM, int BN, int STAGES, int WM, int WN>
struct Shared {
    static constexpr int kBuffer = (BM + BN) * BK * 2;
    static constexpr int kRing = STAGES * kBuffer;
    static constexpr int kSlab = BM / WM < 64 ? BM / WM : 64;   // rows a wave turns around at once
    static constexpr int kTurn = BN / WN + 4;                   // floats of such a row: banks shift by 4 a row
    static constexpr int kTurns = WM * WN * kSlab * kTurn * 4;
    static constexpr int kBytes = kRing > kTurns ? kRing : kTurns;
};

// Work item `item` of a product by WM x WN waves.
template <int BM, int BN, int STAGES, int WM, int WN, bool QS, bool PS, Store STORE>
__device__ __forceinline__ void product(const ProductArgs &a, char *lds, int item)
{
    using S = Shared<BM, BN, STAGES, WM, WN>;
    constexpr bool GATED = STORE == kGated;
    constexpr int NT = WM * WN * 64;
    constexpr int kQ = BM * BK * 2, kBuffer = S::kBuffer, kRing = S::kRing;
    constexpr int MT = BM / WM / 16, NTL = BN / WN / 16;
    constexpr int kSlab = S::kSlab, kTurn = S::kTurn;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();

    // consecutive tiles of one XCD are neighbours in both directions
    const int tiles = a.tiles_m * a.tiles_n;
    const int split = item / tiles, tile = item - split * tiles;
    constexpr int kBand = 8;
    const int band = tile / (kBand * a.tiles_n);
    const int band_rows = a.tiles_m - band * kBand < kBand ? a.tiles_m - band * kBand : kBand;
    const int inside = tile - band * kBand * a.tiles_n;
    const int tm = band * kBand + inside % band_rows, tn = inside / band_rows;
    const int m0 = tm * BM, n0 = tn * (GATED ? BN / 2 : BN);
    const int k0 = split * a.k_per;
    const int K = a.K - k0 < a.k_per ? a.K - k0 : a.k_per;
    // A gradient in two parts (dz is Q of dz w^T, P of x^T dz): every 64 terms are two steps,
    // one for each part, and the other operand's are loaded twice, the second time from the
    // caches.
    constexpr bool GRADIENT = QS == PS;
    const int doubled = GRADIENT && a.part != 0;
    const int steps = ((K + BK - 1) / BK) << doubled;

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
    const size_t q_step = QS ? (size_t)BK * a.ldq * 2 : BK * 2;
    const size_t p_step = PS ? (size_t)BK * a.ldp * 2 : BK * 2;
    const size_t part = doubled ? (size_t)a.part * 2 : 0;
    const size_t q_back = QS ? 0 : part, p_back = QS ? part : 0;   // what the first part's step went on
    const uint32_t base = lds_base(lds) + wave * 1024;

    // loads of a step past the last read nothing and write zeros: the waits stay the same
    constexpr int kLoads = lq.kLoads + lp.kLoads;
    int next = 0, next_at = 0;
    auto issue = [&](int i) {
        const int left = K - (next >> doubled) * BK;
        if (i < lq.kLoads)
            lq.issue(i, buffer_resource(q), base + next_at, left);
        else
            lp.issue(i - lq.kLoads, buffer_resource(p), base + next_at + kQ, left);
        if (i == kLoads - 1) {
            const bool first_part = doubled & ~next;
            q += first_part ? q_back : q_step - q_back;
            p += first_part ? p_back : p_step - p_back;
            ++next;
            next_at = next_at + kBuffer == kRing ? 0 : next_at + kBuffer;
        }
    };

    f32x4 acc[MT][NTL];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NTL; ++n)
            acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int wm = wave / WN * MT, wn = wave % WN * NTL;   // in sixteens

    struct Fragments {
        u32x4 p[NTL], q[MT];
    };
    Fragments one, two;
    int at = 0;
    auto read_p = [&](Fragments &f, int n, int h) { f.p[n] = fragment<BN, PS>(lds + at + kQ, wn + n, h, lane); };
    auto read_q = [&](Fragments &f, int m, int h) { f.q[m] = fragment<BM, QS>(lds + at, wm + m, h, lane); };
    // The products of one half step, between them the reads of the next and, after the
    // barrier, the loads.  The scheduling barriers keep them there: left alone, the reads
    // sink to their uses.
    auto half = [&](const Fragments &now, Fragments &after, int h, bool load) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int n = m * NTL / MT; n < (m + 1) * NTL / MT; ++n)
                read_p(after, n, h);
            read_q(after, m, h);
            if (load)
#pragma unroll
                for (int i = m * kLoads / MT; i < (m + 1) * kLoads / MT; ++i)
                    issue(i);
#pragma unroll
            for (int n = 0; n < NTL; ++n)
                acc[m][n] = mfma_16x16x32(now.p[n], now.q[m], acc[m][n]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int st = 0; st < STAGES; ++st)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            issue(i);
    landed_barrier<(STAGES - 1) * kLoads>();
#pragma unroll
    for (int n = 0; n < NTL; ++n)
        read_p(one, n, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
        read_q(one, m, 0);
    for (int s = 0; s < steps; ++s) {
        half(one, two, 1, false);
        at = at + kBuffer == kRing ? 0 : at + kBuffer;
        // the next step has landed, and every wave holds the rest of this one in registers
        landed_barrier<(STAGES - 2) * kLoads>();
        half(two, one, 0, true);
    }
    landed_barrier<0>();

    // Each wave turns its part around in LDS of its own (the last barrier has freed it),
    // kSlab rows at a time, so that a lane finishes eight neighbouring columns and the
    // finishing code is there once: unrolled over the fragments it missed the instruction
    // cache for 40 us a block.
    float *turn = reinterpret_cast<float *>(lds) + wave * kSlab * kTurn;
    const int i = lane & 15, g = lane >> 4;
    constexpr int kOut = GATED ? NTL * 8 : NTL * 16;   // outputs of a row of the wave's part
    constexpr int kLanes = kOut / 8, kAtOnce = 64 / kLanes;
    const int mine = lane / kLanes, c = lane % kLanes * 8;
    // swiglu: output columns c .. c + 7 lie in the gate unit c / 16 * 2, the up unit follows
    const int z_at = GATED ? (c >> 4) * 32 + (c & 15) : c;
    const int column = n0 + wn * (GATED ? 8 : 16) + c;
#pragma unroll
    for (int slab = 0; slab < MT * 16 / kSlab; ++slab) {
#pragma unroll
        for (int m = 0; m < kSlab / 16; ++m)
#pragma unroll
            for (int n = 0; n < NTL; ++n)
                *reinterpret_cast<f32x4 *>(turn + (m * 16 + i) * kTurn + n * 16 + 4 * g) =
                    acc[slab * (kSlab / 16) + m][n];
        lds_order();
        const int first = m0 + wm * 16 + slab * kSlab;
        if (STORE >= kFull && !a.e.wide) {   // element by element, neighbours side by side
#pragma unroll 4
            for (int x = lane; x < kSlab * kOut; x += 64) {
                const int r = x / kOut, o = x % kOut;
                const float *from = turn + r * kTurn + (GATED ? (o >> 4) * 32 + (o & 15) : o);
                finish_element(a.e, a.M, first + r, n0 + wn * (GATED ? 8 : 16) + o, from[0], GATED ? from[16] : 0.0f);
            }
        } else {
#pragma unroll 4
            for (int r = mine; r < kSlab; r += kAtOnce) {
                const int64_t row = first + r;
                if (row >= a.M || column >= (GATED ? a.e.half : a.C))
                    continue;
                const float *from = turn + r * kTurn + z_at;
                float z[8], up[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    z[j] = from[j];
                    up[j] = GATED ? from[16 + j] : 0.0f;
                }
                if constexpr (STORE == kPartial) {
                    float *out = a.partial + ((size_t)split * a.M + row) * a.C + column;
                    *reinterpret_cast<f32x4 *>(out) = f32x4{z[0], z[1], z[2], z[3]};
                    *reinterpret_cast<f32x4 *>(out + 4) = f32x4{z[4], z[5], z[6], z[7]};
                } else if constexpr (STORE == kPlain) {
                    store16(static_cast<uint16_t *>(a.e.out) + row * a.C + column, pack_eight(z));
                } else {
                    finish_eight(a.e, row, column, z, up);
                }
            }
        }
        lds_order();
    }
}

template <int BM, int BN, int STAGES, int WM, int WN, bool QS, bool PS, Store STORE>
__global__ __launch_bounds__(WM *WN * 64, 2) void product_kernel(ProductArgs a)
{
    __shared__ __attribute__((aligned(1024))) char lds[Shared<BM, BN, STAGES, WM, WN>::kBytes];
    const int item = xcd_balanced_item(blockIdx.x, a.tiles_m * a.tiles_n * a.splits);
    if (item >= 0)
        product<BM, BN, STAGES, WM, WN, QS, PS, STORE>(a, lds, item);
}

// Both gradients in one launch: the blocks of the one with the longer ones first
// (`first_blocks` of the grid), either spread over the XCDs by itself.
template <int BM, int BN, int STAGES, int WM, int WN, Store STORE>
__global__ __launch_bounds__(WM *WN * 64, 2)
void both_gradients_kernel(ProductArgs w, ProductArgs x, int x_first, int first_blocks)
{
    __shared__ __attribute__((aligned(1024))) char lds[Shared<BM, BN, STAGES, WM, WN>::kBytes];
    const int block = blockIdx.x;
    const bool first = block < first_blocks;
    const int mine = first ? block : block - first_blocks;
    if (first == (x_first != 0)) {
        const int item = xcd_balanced_item(mine, x.tiles_m * x.tiles_n);
        if (item >= 0)
            product<BM, BN, STAGES, WM, WN, false, false, kPlain>(x, lds, item);
    } else {
        const int item = xcd_balanced_item(mine, w.tiles_m * w.tiles_n * w.splits);
        if (item >= 0)
            product<BM, BN, STAGES, WM, WN, true, true, STORE>(w, lds, item);
    }
}

// Sums the splits, ascending, and finishes: a thread per eight columns of a row (one
// where N or the pointers do not allow eight).
__global__ __launch_bounds__(256) void join_kernel(ProductArgs a)
{
    const bool gated = a.e.act == MOE_LORA_ACT_SWIGLU;
    const int width = gated ? a.e.half : a.C;
    const size_t apart = (size_t)a.M * a.C;
    if (!a.e.wide) {
        const int64_t items = (int64_t)a.M * width;
        for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < items; x += (int64_t)gridDim.x * 256) {
            const int64_t m = x / width;
            const int c = (int)(x - m * width);
            const float *in = a.partial + m * a.C + c;
            float z = 0.0f, up = 0.0f;
#pragma unroll 4
            for (int s = 0; s < a.splits; ++s) {
                z += in[s * apart];
                if (gated)
                    up += in[s * apart + a.e.half];
            }
            finish_element(a.e, a.M, m, c, z, up);
        }
        return;
    }
    const int per_row = width / 8;
    const int64_t items = (int64_t)a.M * per_row;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < items; x += (int64_t)gridDim.x * 256) {
        const int64_t m = x / per_row;
        const int n = (int)(x - m * per_row) * 8;
        const float *in = a.partial + m * a.C + n;
        float z[8] = {}, up[8] = {};
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[i] += in[s * apart + i];
        if (gated) {
            in += a.e.half;
#pragma unroll 4
            for (int s = 0; s < a.splits; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    up[i] += in[s * apart + i];
        }
        finish_eight(a.e, m, n, z, up);
    }
}

// Tile shapes, and the microseconds that a step of 64 terms takes a block alone on its
// CU (few CUs busy) and among others, measured with 2048 to 8192 rows, 1536 to
// 4096 columns and as many terms.  Larger tiles read LDS and the second-level cache
// less per product; smaller ones fill the chip with fewer rows.
// `rest`: what a block takes beside its steps, on a CU with others.
struct Tile {
    int rows, columns;
    float alone, shared, rest;
};
constexpr int kTileShapes = 4;
constexpr Tile kTiles[kTileShapes] = {{256, 256, 1.05f, 1.45f, 4.0f},
                                      {256, 128, 0.60f, 0.92f, 3.0f},
                                      {128, 128, 0.55f, 0.48f, 1.5f},
                                      {64, 64, 0.20f, 0.20f, 0.5f}};
constexpr int kCus = 256;

template <int BM, int BN, int STAGES, int WM, int WN>
hipError_t launch_tile(Product kind, const ProductArgs &a, hipStream_t s)
{
    const bool gated = kind == Product::forward && a.e.act == MOE_LORA_ACT_SWIGLU;
    const bool plain = kind != Product::forward && a.e.wide && !a.e.padded;
    const int64_t items = (int64_t)a.tiles_m * a.tiles_n * a.splits;
    const dim3 grid((items + 7) / 8 * 8), block(WM * WN * 64);
#define MOE_LAUNCH(QS, PS, STORE) \
    hipLaunchKernelGGL((product_kernel<BM, BN, STAGES, WM, WN, QS, PS, STORE>), grid, block, 0, s, a)
    if (kind == Product::forward) {
        if (a.splits > 1)
            MOE_LAUNCH(false, true, kPartial);
        else if (gated)
            MOE_LAUNCH(false, true, kGated);
        else
            MOE_LAUNCH(false, true, kFull);
    } else if (kind == Product::input_grad) {   // always plain: K is a multiple of 8
        if (a.splits > 1)
            MOE_LAUNCH(false, false, kPartial);
        else
            MOE_LAUNCH(false, false, kPlain);
    } else {
        if (a.splits > 1)
            MOE_LAUNCH(true, true, kPartial);
        else if (plain)
            MOE_LAUNCH(true, true, kPlain);
        else
            MOE_LAUNCH(true, true, kFull);
    }
#undef MOE_LAUNCH
    return hipGetLastError();
}

} // namespace

namespace {

ProductPlan cut(int t, int64_t M, int64_t C, int64_t K, int64_t splits, bool gated)
{
    const Tile &tile = kTiles[t];
    const int64_t steps = (K + BK - 1) / BK, per = steps > 0 ? (steps + splits - 1) / splits : 1;
    ProductPlan p{};
    p.tile = t;
    p.k_per = (int)(per * BK);
    p.splits = steps > 0 ? (int)((steps + per - 1) / per) : 1;
    const bool pairs = gated && p.splits == 1;
    const int64_t width = pairs ? C / 2 : C, columns = pairs ? tile.columns / 2 : tile.columns;
    p.tiles_m = (int)((M + tile.rows - 1) / tile.rows);
    p.tiles_n = (int)((width + columns - 1) / columns);
    return p;
}

int64_t blocks_of(const ProductPlan &p) { return (int64_t)p.tiles_m * p.tiles_n * p.splits; }

// A step of a block alone on its CU, which takes longer as more CUs are busy.
float alone(const Tile &tile, int64_t blocks)
{
    const float share = blocks < kCus ? (float)blocks / kCus : 1.0f;
    return tile.alone + (tile.shared > tile.alone ? (tile.shared - tile.alone) * share : 0.0f);
}

// A split's fp32 sums are written and read again, at about 5 TB/s, and a second kernel
// starts after the first (3 us): 2048 x 1536 sums of 8192 terms take 87 us whole (128 x
// 128 tiles), 61 us as two splits of 256 x 128 tiles, 83 us as six.
float joining(const ProductPlan &p, int64_t M, int64_t C)
{
    return p.splits > 1 ? 3.0f + (float)p.splits * M * C * 8.0f / 5e6f : 0.0f;
}

// f(splits) for every cutting of the terms that is worth a look, the whole first
template <class F>
void for_splits(int64_t tiles, int64_t K, F f)
{
    const int64_t steps = (K + BK - 1) / BK;
    int64_t last = 0;
    for (int64_t splits = 1; splits <= 64; ++splits) {
        const int64_t per = (steps + splits - 1) / splits;
        if (splits > 1 && (per < 4 || tiles * splits > 4 * kCus))
            return;
        if (per != last)   // else the same cutting with empty splits
            f(splits);
        last = per;
    }
}

} // namespace

// The tile and split that take the least time by the figures above.
ProductPlan plan_product(int64_t M, int64_t C, int64_t K, bool gated, int parts)
{
    ProductPlan best{};
    for (int t = 0; t < kTileShapes; ++t) {
        const ProductPlan whole = cut(t, M, C, K, 1, false);
        for_splits(blocks_of(whole), K, [&](int64_t splits) {
            ProductPlan p = cut(t, M, C, K, splits, gated);
            const int64_t each = (blocks_of(cut(t, M, C, K, splits, false)) + kCus - 1) / kCus;   // of the busiest CU
            const float steps = (float)(p.k_per / BK * parts);
            p.us = steps * (each == 1 ? alone(kTiles[t], blocks_of(p)) : each * kTiles[t].shared) + joining(p, M, C);
            if (best.tiles_m == 0 || p.us < best.us)
                best = p;
        });
    }
    return best;
}

// The same for the two gradients in one launch: the CUs' work in all, the longest block,
// and what a block takes beside its steps.
float plan_both(int64_t M, int64_t in, int64_t columns, int parts, ProductPlan *dw, ProductPlan *dx)
{
    float least = 0.0f;
    for (int t = 0; t < kTileShapes; ++t) {
        const Tile &tile = kTiles[t];
        const ProductPlan x = cut(t, M, in, columns, 1, false), whole = cut(t, in, columns, M, 1, false);
        for_splits(blocks_of(whole), M, [&](int64_t splits) {
            const ProductPlan w = cut(t, in, columns, M, splits, false);
            const float x_steps = (float)(x.k_per / BK * parts), w_steps = (float)(w.k_per / BK * parts);
            const float all = (blocks_of(x) * (x_steps * tile.shared + tile.rest) +
                               blocks_of(w) * (w_steps * tile.shared + tile.rest)) / kCus;
            const float longest = (x_steps > w_steps ? x_steps : w_steps) * alone(tile, blocks_of(x) + blocks_of(w)) +
                                  tile.rest;
            const float us = (all > longest ? all : longest) + joining(w, in, columns);
            if (least == 0.0f || us < least) {
                least = us;
                *dw = w;
                *dx = x;
            }
        });
    }
    return least;
}

namespace {

ProductArgs with_plan(const ProductArgs &given, const ProductPlan &plan)
{
    ProductArgs a = given;
    a.tiles_m = plan.tiles_m;
    a.tiles_n = plan.tiles_n;
    a.splits = plan.splits;
    a.k_per = plan.k_per;
    return a;
}

hipError_t launch_join(const ProductArgs &a, hipStream_t s)
{
    const bool gated = a.e.act == MOE_LORA_ACT_SWIGLU;
    const int64_t items = (int64_t)a.M * (gated ? a.e.half : a.C) / (a.e.wide ? 8 : 1);
    const int64_t blocks = (items + 255) / 256;
    hipLaunchKernelGGL(join_kernel, dim3(blocks < 1 << 20 ? blocks : 1 << 20), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_product(Product kind, const ProductPlan &plan, const ProductArgs &given, hipStream_t s)
{
    const ProductArgs a = with_plan(given, plan);
    const hipError_t rc = plan.tile == 0   ? launch_tile<256, 256, 2, 2, 4>(kind, a, s)
                          : plan.tile == 1 ? launch_tile<256, 128, 3, 4, 2>(kind, a, s)
                          : plan.tile == 2 ? launch_tile<128, 128, 2, 2, 2>(kind, a, s)
                                           : launch_tile<64, 64, 4, 2, 2>(kind, a, s);
    return rc != hipSuccess || a.splits == 1 ? rc : launch_join(a, s);
}

namespace {

template <int BM, int BN, int STAGES, int WM, int WN>
hipError_t launch_both(const ProductArgs &w, const ProductArgs &x, hipStream_t s)
{
    auto padded = [](int64_t n) { return (int)((n + 7) / 8 * 8); };
    const int w_blocks = padded((int64_t)w.tiles_m * w.tiles_n * w.splits), x_blocks = padded((int64_t)x.tiles_m * x.tiles_n);
    const int x_first = x.K > w.k_per, first = x_first ? x_blocks : w_blocks;
    const dim3 grid(w_blocks + x_blocks), block(WM * WN * 64);
    if (w.splits > 1)
        hipLaunchKernelGGL((both_gradients_kernel<BM, BN, STAGES, WM, WN, kPartial>), grid, block, 0, s, w, x, x_first,
                           first);
    else if (w.e.wide && !w.e.padded)
        hipLaunchKernelGGL((both_gradients_kernel<BM, BN, STAGES, WM, WN, kPlain>), grid, block, 0, s, w, x, x_first,
                           first);
    else
        hipLaunchKernelGGL((both_gradients_kernel<BM, BN, STAGES, WM, WN, kFull>), grid, block, 0, s, w, x, x_first,
                           first);
    return hipGetLastError();
}

} // namespace

hipError_t launch_both_gradients(const ProductPlan &dw, const ProductArgs &w_given, const ProductPlan &dx,
                                 const ProductArgs &x_given, hipStream_t s)
{
    const ProductArgs w = with_plan(w_given, dw), x = with_plan(x_given, dx);
    const hipError_t rc = dw.tile == 0   ? launch_both<256, 256, 2, 2, 4>(w, x, s)
                          : dw.tile == 1 ? launch_both<256, 128, 3, 4, 2>(w, x, s)
                          : dw.tile == 2 ? launch_both<128, 128, 2, 2, 2>(w, x, s)
                                         : launch_both<64, 64, 4, 2, 2>(w, x, s);
    return rc != hipSuccess || w.splits == 1 ? rc : launch_join(w, s);
}

} // namespace moe_lora
