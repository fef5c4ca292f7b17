// expert_gemm_w4_many.hip -- grouped products with 4-bit weights, tens to
// hundreds of rows per expert (w4_gemm.h has the mathematics).
//
// Decoding a weight costs about one instruction, whatever the rows it meets, so
// a wave keeps 64 columns and up to 64 rows: each decoded fragment meets up
// to four row tiles.  A block is 4 waves on one row tile set of 16 * MT rows
// and 256 columns (one slab a wave); the activations go through two LDS
// buffers, one step ahead, each staged once for the four slabs with its group
// sums; the codes go straight to the registers of the one wave that needs
// them, two steps ahead.  Two blocks share a CU (MT = 4), so that one's
// decoding and scaling (VALU) runs under the other's matrix instructions.  A
// block runs several slab groups of its rows in turn, and the pipeline runs on
// across them.
//
// Measured with hidden 2048, inter 768, 128 experts top-8: 384 tokens, rank 16,
// gate_up 60 us and down 48 us for 233 and 137 MB of weights and adapters: 3.9
// and 2.9 TB/s, between the stream's rate and the loop's issue.  2048 tokens,
// rank 64: gate_up 171..204 us (machines differ in clock), down 144..163 us, with
// the matrix units busy 30% and 21% of the time.  What bounds that is a wave's
// own issue: per step and wave the MFMAs, the LDS reads and the decoding and
// scaling take about 1000, 1000 and 700 cycles, and two waves per SIMD overlap
// them only in part.  The LoRA expand is 17 and 52 us of it (181 and 153 us against 164 and 101 without
// adapters): every 64-row tile loads its slab's B rows (half a cache line a row
// and step) again.
//
// Groups of 32 rows hold four groups' scales and zero points per step: with zero
// points or 64-row tiles they spill 2 to 18 registers, stored before the loops
// and loaded again behind them, once a block.  384 and 2048 tokens, rank 16, groups of 32 / 64 /
// 128: 167 / 155 / 151 and 390 / 352 / 328 us a layer, with zero points 189 / 163
// / 156 and 454 / 376 / 344.
#include "w4_gemm.h"
#include "w4_launch.h"

namespace moe_lora {
namespace {

// A block's share: what the whole block agrees on.
struct Job {
    int le, row0, n_rows, sg0, sg1;
};

// The block's work with NM of its MT row tiles (rows behind n_rows repeat the
// last one and are not stored).
template <int NM, int MT, int G, bool kGated, bool kZeros>
__device__ __forceinline__ void run_job(const GemmW4Args &a, const Job &job, u32x4 *lds, int wave, int lane)
{
    constexpr int kUnit = kStepChunks * MT * kWave;  // fragments of a step (16-byte pieces)
    constexpr int kXs = 128 / G * MT * 16;           // its group sums
    constexpr int SB = 4 / MT;                       // steps staged together: a unit per wave
    constexpr int kExpandSteps = MT == 4 ? 2 : 4;    // in flight: what the registers hold
    const int I = kGated ? a.I : 0;
    const int n_steps = a.k_units / 2;
    const int n_pairs = (n_steps + 1) / 2;

    u32x4 *frag = lds;
    float *xs = reinterpret_cast<float *>(lds + 2 * SB * kUnit);
    u32x4 *sfrag = reinterpret_cast<u32x4 *>(xs + 2 * SB * kXs);
    const DecodeW4 decode;

    auto slab_of = [&](int sg) { return find_slab(a, job.le, min(sg * 4 + wave, a.n_slabs - 1)); };
    SlabW4 w = slab_of(job.sg0);
    StepW4<G> st[2];
    load_step<G, kZeros>(st[0], a, w, 0, lane);
    load_step<G, kZeros>(st[1], a, w, min(1, n_steps - 1), lane);

    // this wave stages row tile um of step (its half of SB)
    const int um = wave % MT, uh = wave / MT;
    const uint16_t *arow = nullptr;
    int slot = 0;
    uint32_t adapters = 0xffffffffu;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int p = job.row0 + min(m * 16 + (lane & 15), job.n_rows - 1);
        const uint32_t l = find_row<kGated>(a, p, um == m, &arow, &slot);
        adapters = (adapters & ~(0xffu << (8 * m))) | (l << (8 * m));
    }
    arow += (lane >> 4) * 8;
    u32x4 v[kStepChunks];
    load_unit(v, arow, uh, a.K);
    const int s_chunks = a.S ? (a.r + 31) >> 5 : 0;
    for (int c = uh; c < s_chunks; c += SB)
        sfrag[(c * MT + um) * kWave + lane] = load_s(a, slot, c, lane);
    auto stage = [&](int buf, int step) {
        store_unit<MT, G, kZeros>(v, step, a.K, frag + (buf * SB + uh) * kUnit + um * kWave, xs + (buf * SB + uh) * kXs + um * 16,
                          lane);
    };
    stage(0, uh);
    lds_barrier();
    const unsigned long long used = a.S ? adapters_used(adapters, NM) : 0;

    f32x4 acc[NM][kNS];
    zero_acc(acc);
    auto compute = [&](const StepW4<G> &s, int b) {  // b: step buffer 0 .. 2 SB - 1
        main_step<NM, MT, G, kZeros>(acc, s, decode, frag + b * kUnit, xs + b * kXs, lane);
    };
    int buf = 0;  // SB == 2: buffer of the current pair
    for (int sg = job.sg0; sg < job.sg1; ++sg) {
        const SlabW4 wn = slab_of(min(sg + 1, job.sg1 - 1));
        for (int p = 0; p < n_pairs; ++p) {
            // behind its last pair the ring goes on with the next slab
            const bool last = p + 1 == n_pairs;
            const SlabW4 wl = last ? wn : w;
            const int next = last ? 0 : 2 * p + 2;
            if (SB == 2) {
                load_unit(v, arow, next + uh, a.K);
                compute(st[0], buf * 2);
                load_step<G, kZeros>(st[0], a, wl, next, lane);
                if (2 * p + 1 < n_steps)
                    compute(st[1], buf * 2 + 1);
                load_step<G, kZeros>(st[1], a, wl, min(next + 1, n_steps - 1), lane);
                stage(buf ^ 1, next + uh);
                lds_barrier();
                buf ^= 1;
            } else {
                load_unit(v, arow, 2 * p + 1, a.K);
                compute(st[0], 0);
                load_step<G, kZeros>(st[0], a, wl, next, lane);
                stage(1, 2 * p + 1);
                lds_barrier();
                load_unit(v, arow, next, a.K);
                if (2 * p + 1 < n_steps)
                    compute(st[1], 1);
                load_step<G, kZeros>(st[1], a, wl, min(next + 1, n_steps - 1), lane);
                stage(0, next);
                lds_barrier();
            }
        }
        if (used) {
            Expand<NM, MT, kExpandSteps> ex;
            ex.start(used, a, w, I, lane);
            ex.run(acc, a, w, I, adapters, sfrag, lane);
        }
        if (sg * 4 + wave < a.n_slabs)
            store_slab<NM, kGated>(acc, a, job.row0, job.n_rows, w.slab, lane);
        zero_acc(acc);
        w = wn;
        // No store may be outstanding in the loop above: the compiler would have
        // to wait for all loads wherever it waits for one.
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    }
}

template <int MT, int G, bool kGated, bool kZeros>
__global__ __launch_bounds__(256, 2) void expert_gemm_w4_many_kernel(GemmW4Args a, int per)
{
    extern __shared__ u32x4 lds[];  // two buffers of SB steps, their group sums, S fragments
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = wave_id();
    const int n_sg = (a.n_slabs + 3) / 4;
    const int n_jobs = (n_sg + per - 1) / per;

    const int logical = xcd_balanced_item(blockIdx.x, n_tiles_used(a) * n_jobs);
    if (logical < 0)
        return;
    const TileW4 te = find_tile(a, logical / n_jobs);
    if (te.le < 0)
        return;
    // the row tiles of one job are neighbours and share its codes in L2; an
    // expert's rows are cut evenly
    const int nt = (te.rows + a.tile_rows - 1) / a.tile_rows;
    const int in_expert = logical - te.first * n_jobs;
    const int at = in_expert / nt;
    const int sub = in_expert - at * nt;
    const int rows_per = ((te.rows + nt - 1) / nt + 15) & ~15;
    const Job job{te.le, te.row + sub * rows_per, min(rows_per, te.rows - sub * rows_per), at * per,
                  min(n_sg, at * per + per)};
    const int n_mt = (job.n_rows + 15) >> 4;
    if (MT == 4 && n_mt <= 2)
        run_job<2, MT, G, kGated, kZeros>(a, job, lds, wave, lane);
    else if (MT == 4 && n_mt == 3)
        run_job<MT == 4 ? 3 : 1, MT, G, kGated, kZeros>(a, job, lds, wave, lane);
    else if (MT == 2 && n_mt == 1)
        run_job<1, MT, G, kGated, kZeros>(a, job, lds, wave, lane);
    else
        run_job<MT, MT, G, kGated, kZeros>(a, job, lds, wave, lane);
}

template <int MT, int G, bool kGated, bool kZeros>
hipError_t launch_many(const GemmW4Args &a, hipStream_t s)
{
    const int n_sg = (a.n_slabs + 3) / 4;
    const int per = w4_groups_per_block(w4_row_tiles(a.n_tiles, a.n_busy, a.n_local, a.tile_rows), n_sg);
    const int blocks = (a.n_tiles * ((n_sg + per - 1) / per) + 7) / 8 * 8;
    const int lds = 2 * (4 / MT) * step_lds_bytes(MT, G) + (a.S ? (a.r + 31) / 32 * MT * 1024 : 0);
    hipLaunchKernelGGL((expert_gemm_w4_many_kernel<MT, G, kGated, kZeros>), dim3(blocks), dim3(256), lds, s, a,
                       per);
    return hipGetLastError();
}

} // namespace

hipError_t launch_gemm_w4_many(const GemmW4Args &a, bool gated, hipStream_t s)
{
    return with_format(a.group, gated, a.zeros != nullptr, [&](auto G, auto gt, auto zr) {
        return a.tile_rows == 32 ? launch_many<2, G(), gt(), zr()>(a, s) : launch_many<4, G(), gt(), zr()>(a, s);
    });
}

} // namespace moe_lora
