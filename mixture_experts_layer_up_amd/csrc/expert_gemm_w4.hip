// expert_gemm_w4.hip -- grouped products with 4-bit weights, few rows per
// expert (w4_gemm.h has the mathematics).
//
// The stream of codes bounds these shapes.  A block is NW waves on one row
// tile of 16 rows: WN 64-column slabs times KS shares of K (WN * KS = NW).
// Each wave streams its own codes through a ring of registers, so no wave
// waits for another in the main loop; the tile's activations (and its LoRA
// shrink rows) are staged in LDS in MFMA fragment order for all slabs of the
// block, a panel of K at a time.  KS is 1 when there are enough slabs to fill
// the GPU; a few tokens touch only a few experts, and then several waves
// share one slab's K and add up through LDS at the end.
//
// Measured with hidden 2048, inter 768, 128 experts top-8, rank-16 adapters:
// 64 tokens (group 64, zero points) gate_up 40 us for 231 MB from HBM, 5.7
// TB/s (a large copy on the same card: 4.9), down 29 us for 127 MB.  A ring of
// three steps, or four waves per SIMD, spill registers and are slower.  Groups of
// 32 with zero points spill 2 and 4 registers as it is, stored once and loaded
// once a panel: 64 tokens 108 us a layer, 101 without zero points, 96 in groups
// of 128.  One token 8.4 and 6.8 us: latency, the work list, its rows, the
// activations and the first codes being loaded in turn.
#include <algorithm>

#include "w4_gemm.h"
#include "w4_launch.h"

namespace moe_lora {
namespace {

constexpr int kRing = 2;         // steps in flight per wave
constexpr int kExpandSteps = 2;  // LoRA expand steps in flight

// Steps whose activations are staged at a time.  Half of a 2048-row K leaves
// LDS for three blocks per CU (64 tokens, 128 experts: 40 us for gate_up, 49 us
// with all of it); blocks of 8 waves, few by definition, take it whole.
constexpr int panel_steps(int NW) { return NW == 8 ? 16 : 8; }

template <int NW, int G, bool kGated, bool kZeros>
__global__ __launch_bounds__(NW * kWave, 3) void expert_gemm_w4_kernel(GemmW4Args a, int ks_log)
{
    constexpr int D = kRing, kPanelSteps = panel_steps(NW);
    constexpr int kXs = 128 / G * 16;  // group sums of a step
    extern __shared__ u32x4 lds[];     // [S chunk][lane], [K chunk][lane], group sums; at the end the K shares
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = wave_id();
    const int KS = 1 << ks_log, WN = NW >> ks_log;
    const int n_sg = (a.n_slabs + WN - 1) / WN;  // slab groups

    const int logical = xcd_balanced_item(blockIdx.x, n_tiles_used(a) * n_sg);
    if (logical < 0)
        return;
    const TileW4 te = find_tile(a, logical / n_sg);
    const int le = te.le;
    if (le < 0)
        return;
    // the row tiles of one slab group are neighbours and share its codes in L2
    const int nt = (te.rows + a.tile_rows - 1) / a.tile_rows;
    const int in_expert = logical - te.first * n_sg;
    const int sg = in_expert / nt;
    const int sub = in_expert - sg * nt;
    const int row0 = te.row + sub * a.tile_rows;
    const int n_rows = min(a.tile_rows, te.rows - sub * a.tile_rows);
    const int I = kGated ? a.I : 0;

    const int ks = wave & (KS - 1);
    const int slab_raw = sg * WN + (wave >> ks_log);
    const bool active = slab_raw < a.n_slabs;  // uniform; an idle wave only helps staging
    const SlabW4 w = find_slab(a, le, min(slab_raw, a.n_slabs - 1));
    const int n_steps = a.k_units / 2;
    const int s_chunks = a.S ? (a.r + 31) >> 5 : 0;
    u32x4 *frag = lds + s_chunks * kWave;
    float *xs = reinterpret_cast<float *>(frag + min(kPanelSteps, n_steps) * kStepChunks * kWave);
    const DecodeW4 decode;

    f32x4 acc[1][kNS];
    zero_acc(acc);
    const uint16_t *arow = nullptr;
    uint32_t adapters = 0xffffffffu;

    for (int p0 = 0; p0 < n_steps; p0 += kPanelSteps) {
        const int ps = min(kPanelSteps, n_steps - p0);
        const int sb = p0 + ((ks * ps) >> ks_log);  // this wave's steps
        const int ns = p0 + (((ks + 1) * ps) >> ks_log) - sb;
        const bool expand = a.S && p0 == 0 && ks == 0 && active;
        Expand<1, 1, kExpandSteps> ex;
        // the first codes are on their way before the rows are known
        StepW4<G> st[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
            load_step<G, kZeros>(st[d], a, w, min(sb + d, n_steps - 1), lane);
        if (p0 == 0) {
            int slot = 0;
            adapters = find_row<kGated>(a, row0 + min(lane & 15, n_rows - 1), true, &arow, &slot);
            arow += (lane >> 4) * 8;
            for (int c = wave; c < s_chunks; c += NW)
                lds[c * kWave + lane] = load_s(a, slot, c, lane);
            if (expand)  // its first operands travel while the activations are staged
                ex.start(adapters_used(adapters, 1), a, w, I, lane);
        } else {
            lds_barrier();  // the panel before is done with
        }
        for (int t = wave; t < ps; t += NW) {
            u32x4 v[kStepChunks];
            load_unit(v, arow, p0 + t, a.K);
            store_unit<1, G, kZeros>(v, p0 + t, a.K, frag + t * kStepChunks * kWave, xs + t * kXs, lane);
        }
        lds_barrier();
        if (!active)
            continue;
        if (expand)
            ex.run(acc, a, w, I, adapters, lds, lane);

        auto step = [&](const StepW4<G> &s, int i) {
            const int t = sb - p0 + i;
            main_step<1, 1, G, kZeros>(acc, s, decode, frag + t * kStepChunks * kWave, xs + t * kXs, lane);
        };
        int i0 = 0;
        for (; i0 + D < ns; i0 += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                step(st[d], i0 + d);
                load_step<G, kZeros>(st[d], a, w, sb + min(i0 + d + D, ns - 1), lane);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (i0 + d < ns)
                step(st[d], i0 + d);
    }

    if (ks_log > 0) {  // waves with a later share of K hand their sums to the first
        lds_barrier();
        f32x4 *part = reinterpret_cast<f32x4 *>(lds);
        const int wn = wave >> ks_log;
        if (ks > 0) {
#pragma unroll
            for (int n = 0; n < kNS; ++n)
                part[(((ks - 1) * WN + wn) * kNS + n) * kWave + lane] = acc[0][n];
        }
        lds_barrier();
        if (ks > 0)
            return;
        for (int i = 1; i < KS; ++i)
#pragma unroll
            for (int n = 0; n < kNS; ++n)
                acc[0][n] += part[(((i - 1) * WN + wn) * kNS + n) * kWave + lane];
    }
    if (active)
        store_slab<1, kGated>(acc, a, row0, n_rows, w.slab, lane);
}

template <int NW, int G, bool kGated, bool kZeros>
hipError_t launch_few(const GemmW4Args &a, int log, hipStream_t s)
{
    const int WN = NW >> log;
    const int blocks = (a.n_tiles * ((a.n_slabs + WN - 1) / WN) + 7) / 8 * 8;
    const int staged = std::min(panel_steps(NW), a.k_units / 2) * step_lds_bytes(1, G) +
                       (a.S ? (a.r + 31) / 32 * 1024 : 0);
    const int parts = log ? (NW - WN) * kNS * kWave * 16 : 0;
    hipLaunchKernelGGL((expert_gemm_w4_kernel<NW, G, kGated, kZeros>), dim3(blocks), dim3(NW * kWave),
                       std::max(staged, parts), s, a, log);
    return hipGetLastError();
}

} // namespace

hipError_t launch_gemm_w4(const GemmW4Args &a, bool gated, hipStream_t s)
{
    if (a.n_tiles <= 0)
        return hipSuccess;
    if (a.tile_rows > 16)
        return launch_gemm_w4_many(a, gated, s);
    return with_format(a.group, gated, a.zeros != nullptr, [&](auto G, auto gt, auto zr) {
        const int log = w4_k_shares_log(std::min(a.n_tiles, a.n_busy), a.n_slabs, a.k_units / 2);
        return log == 3 ? launch_few<8, G(), gt(), zr()>(a, log, s) : launch_few<4, G(), gt(), zr()>(a, log, s);
    });
}

} // namespace moe_lora
