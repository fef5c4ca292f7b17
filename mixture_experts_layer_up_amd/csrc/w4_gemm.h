// w4_gemm.h -- what the grouped products with 4-bit weights share.
//
// Computed is what expert_gemm.hip computes, with expert weights
// w[k][n] = s[g][n] (q[k][n] - z[g][n]), g = k / group (w4_layout.h):
//   gate_up:  h = x_t W13[e] + B_gu[l,e] s_gu[p];  act[p] = SiLU(h[:I]) h[I:]
//   down:     y[p] = act[p] W2[e] + B_dn[l,e] s_dn[p]
//
// The codes never become rounded weights.  A code enters the MFMA as the
// exact bf16 number 16 + q (one rotate and one and-or per pair of weights),
// and per group, with x's group sum xs taken by MFMAs against ones when the
// activations are staged (once for all columns),
//   sum_k x_k w_k = s ( sum_k x_k (16 + q_k)  -  (16 + z) sum_k x_k )
// in fp32.  bf16 products are exact in fp32, so the only roundings are the fp32
// sums', of terms of size (16 + q) |x| and (16 + z) |x|.  The error of a column
// is thus at most about (K + group) 2^-24 sum_k s (32 + q_k + z) |x_k|, absolute:
// where the sum itself cancels (a weight of 0, activations of one sign), it does
// not shrink with it.  For the same reason a group sum overflows when 31 times
// the sum of its |x| does, that is for activations above about 8e34.
//
// A wave's work is one 64-column slab: K in steps of 128 rows, and the LoRA
// expand as more K: per adapter that the tile's rows use, steps of 32 rank
// positions in which the rows of other adapters are 0.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "kernels_w4.h"
#include "mfma_pipeline.h"
#include "w4_layout.h"

namespace moe_lora {
namespace {

// 16 bytes at the alignment of bf16 values (rows of ranks that are no multiple of 8)
typedef u32x4 __attribute__((aligned(2))) u32x4_unaligned;

constexpr int kStepChunks = 4;  // 32-row chunks of a step
constexpr int kStepBytes = 2 * kW4UnitBytes;

// Decoding.  Its constants are opaque to the compiler and in the two kinds of
// register one v_and_or_b32 can take (as literals it would split each into an
// and and an or).
struct DecodeW4 {
    uint32_t mask, k16;
    __device__ __forceinline__ DecodeW4() : mask(0x00780078u), k16(0x41804180u)
    {
        asm("" : "+s"(mask));
        asm("" : "+v"(k16));
    }
    // Four exact bf16 pairs 16 + q of one word of codes.
    __device__ __forceinline__ u32x4 operator()(uint32_t w) const
    {
        return u32x4{(w & mask) | k16, (__builtin_amdgcn_alignbit(w, w, 4) & mask) | k16,
                     (__builtin_amdgcn_alignbit(w, w, 8) & mask) | k16,
                     (__builtin_amdgcn_alignbit(w, w, 12) & mask) | k16};
    }
};

// One step's B operand of one wave: b[2 u + h] holds tiles 2h and 2h + 1 of
// unit u, word (tile & 1) * 2 + chunk.
template <int G>
struct StepW4 {
    static constexpr int kGroups = 128 / G;
    u32x4 b[4];
    uint2 sc[kGroups];     // four tiles' bf16 scales
    uint32_t zr[kGroups];  // four tiles' 16 + zero point
};

// The block's entry of the work list, as wave-uniform values: everything that
// follows from it (the slab's addresses above all) then lives in scalar registers.
struct TileW4 {
    int le, row, rows, first;
};

__device__ __forceinline__ int n_tiles_used(const GemmW4Args &a)
{
    return __builtin_amdgcn_readfirstlane(*a.tile_count);
}

__device__ __forceinline__ TileW4 find_tile(const GemmW4Args &a, int i)
{
    const int4 t = a.tiles[i];
    return TileW4{__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y),
                  __builtin_amdgcn_readfirstlane(t.z), __builtin_amdgcn_readfirstlane(t.w)};
}

// A wave's slab (uniform).
struct SlabW4 {
    const uint8_t *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
    int le, slab;
};

__device__ __forceinline__ SlabW4 find_slab(const GemmW4Args &a, int le, int slab)
{
    const size_t at = (size_t)le * a.n_slabs + slab;
    return SlabW4{a.codes + at * a.k_units * kW4UnitBytes, a.scales + at * a.n_groups * 64,
                  a.zeros ? a.zeros + at * a.n_groups * 64 : nullptr, le, slab};
}

template <int G, bool kZeros>
__device__ __forceinline__ void load_step(StepW4<G> &st, const GemmW4Args &a, const SlabW4 &w, int step, int lane)
{
    const uint8_t *pc = w.codes + (size_t)step * kStepBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        st.b[i] = load16_stream(pc + (unsigned)(lane * 16 + i * 1024));
#pragma unroll
    for (int g = 0; g < StepW4<G>::kGroups; ++g) {
        // groups behind K read the last real one's scale
        const size_t at = (size_t)min(step * StepW4<G>::kGroups + g, a.n_groups - 1) * 64;
        st.sc[g] = *reinterpret_cast<const uint2 *>(w.scales + at + (unsigned)((lane & 15) * 4));
        if (kZeros)
            st.zr[g] = *reinterpret_cast<const uint32_t *>(w.zeros + at + (unsigned)((lane & 15) * 4));
    }
}

// An expand step: 32 rank positions from q0 of one adapter.
struct ExpandStep {
    int l, q0;
};

// Where the lane reads tile n's 8 rank positions of an expand step: elements
// behind the (uniform) row of the tile's first column.  A row of the LoRA B
// stack that is not a whole number of 16 bytes is read at its own alignment; a
// lane whose 16 bytes would end behind the stack reads the stack's last 16
// (`back` elements further back than asked).
struct ExpandRow {
    const uint16_t *base;
    unsigned off;
    int back;
};

__device__ __forceinline__ ExpandRow expand_row(const GemmW4Args &a, const SlabW4 &w, ExpandStep e, int n, int I,
                                                int lane)
{
    const size_t stack = a.lb_shared ? (size_t)e.l : (size_t)e.l * a.E_l + w.le;
    const size_t first = (stack * a.n_canon + w4_column(w.slab, n, 0, I)) * a.r;
    const size_t room = (size_t)a.lb_stacks * a.n_canon * a.r - 8 - first;  // >= 16 r - 8
    const int q = e.q0 + (lane >> 4) * 8;
    const int off = (lane & 15) * a.r + (q < a.r ? q : 0);  // <= 16 r
    const int at = min(off, (int)(room < 65536 ? room : 65536));
    return ExpandRow{a.LB + first, (unsigned)at, off - at};
}

__device__ __forceinline__ void load_expand(u32x4 (&b)[kNS], const GemmW4Args &a, const SlabW4 &w, ExpandStep e,
                                            int I, int lane)
{
#pragma unroll
    for (int n = 0; n < kNS; ++n) {
        const ExpandRow r = expand_row(a, w, e, n, I, lane);
        b[n] = *reinterpret_cast<const u32x4_unaligned *>(r.base + r.off);
    }
}

// Ranks that are not a multiple of 8: moves what load_expand read further back
// than asked to its place and clears the positions past the rank.
__device__ __forceinline__ void fix_expand(u32x4 (&b)[kNS], const GemmW4Args &a, const SlabW4 &w, ExpandStep e,
                                           int I, int lane)
{
    const int left = a.r - (e.q0 + (lane >> 4) * 8);  // valid positions
    u32x4 mask;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        mask[i] = (left > 2 * i ? 0x0000ffffu : 0u) | (left > 2 * i + 1 ? 0xffff0000u : 0u);
#pragma unroll
    for (int n = 0; n < kNS; ++n) {
        const int back = expand_row(a, w, e, n, I, lane).back;
        u32x4 v = b[n];
        v = back & 4 ? u32x4{v.z, v.w, 0u, 0u} : v;
        v = back & 2 ? u32x4{v.y, v.z, v.w, 0u} : v;
        if (back & 1)
            v = u32x4{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
        b[n] = v & mask;
    }
}

// The activations of one step and row tile: four A fragments, loaded from the
// lane's row (at its K quarter; behind K the row's end again).
__device__ __forceinline__ void load_unit(u32x4 (&v)[kStepChunks], const uint16_t *row, int step, int K)
{
#pragma unroll
    for (int c = 0; c < kStepChunks; ++c)
        v[c] = load16(row + min(step * 128 + c * 32, K - 32));
}

// Stores them to LDS, 0 behind K, with their group sums: frag[chunk * MT][lane],
// and per group the 16 rows' -sum (times 24 = 16 + z in formats without zero
// points) at xs[group * MT * 16].  The sums come from MFMAs against ones, whose
// every column is the row's sum.  (The clearing is here and not at the load,
// which it would make wait.)
template <int MT, int G, bool kZeros>
__device__ __forceinline__ void store_unit(u32x4 (&v)[kStepChunks], int step, int K, u32x4 *frag, float *xs,
                                           int lane)
{
    const u32x4 ones{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    if (step * 128 + 128 > K) {
#pragma unroll
        for (int c = 0; c < kStepChunks; ++c)
            v[c] = keep_if(v[c], step * 128 + c * 32 < K);
    }
#pragma unroll
    for (int c = 0; c < kStepChunks; ++c)
        frag[c * MT * kWave + lane] = v[c];
#pragma unroll
    for (int g = 0; g < 128 / G; ++g) {
        f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < G / 32; ++i)
            sum = mfma_16x16x32(v[g * (G / 32) + i], ones, sum);
        if ((lane & 15) == 0)
            *reinterpret_cast<f32x4 *>(xs + g * MT * 16 + (lane >> 4) * 4) = sum * (kZeros ? -1.0f : -24.0f);
    }
}

// A main step over NM of the MT staged row tiles: per group, MFMAs over its
// chunks into accumulators that start from -(16 + z) xs, then acc += s grp.
// frag and xs as store_unit left them.  NM is a constant: a branch around a
// row tile would keep the LDS reads from running ahead of the MFMAs.  With
// more than two row tiles the columns go in two halves, each reading the
// fragments again: the group's accumulators then need half the registers.
template <int NM, int MT, int G, bool kZeros>
__device__ __forceinline__ void main_step(f32x4 (&acc)[NM][kNS], const StepW4<G> &st, const DecodeW4 &decode,
                                          const u32x4 *frag, const float *xs, int lane)
{
    constexpr int kGroupChunks = G / 32;
    constexpr int NN = NM > 2 ? 2 : 4;  // column tiles at a time
#pragma unroll
    for (int g = 0; g < StepW4<G>::kGroups; ++g) {
        const uint2 sc = st.sc[g];
        const float s[kNS] = {__uint_as_float(sc.x << 16), __uint_as_float(sc.x & 0xffff0000u),
                              __uint_as_float(sc.y << 16), __uint_as_float(sc.y & 0xffff0000u)};
#pragma unroll
        for (int n0 = 0; n0 < kNS; n0 += NN) {
            f32x4 grp[NM][NN], sum[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m)
                sum[m] = *reinterpret_cast<const f32x4 *>(xs + (g * MT + m) * 16 + (lane >> 4) * 4);
#pragma unroll
            for (int i = 0; i < kGroupChunks; ++i) {
                const int c = g * kGroupChunks + i;
                u32x4 x[NM];
#pragma unroll
                for (int m = 0; m < NM; ++m)
                    x[m] = frag[(c * MT + m) * kWave + lane];
#pragma unroll
                for (int n = 0; n < NN; ++n) {
                    const u32x4 b = decode(st.b[(c >> 1) * 2 + ((n0 + n) >> 1)][(n & 1) * 2 + (c & 1)]);
                    const float z = kZeros ? (float)((st.zr[g] >> (8 * (n0 + n))) & 0xffu) : 1.0f;
#pragma unroll
                    for (int m = 0; m < NM; ++m)
                        grp[m][n] = mfma_16x16x32(x[m], b, i > 0 ? grp[m][n] : kZeros ? sum[m] * z : sum[m]);
                }
            }
#pragma unroll
            for (int n = 0; n < NN; ++n) {
#pragma unroll
                for (int m = 0; m < NM; ++m) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[m][n0 + n][i] = fmaf(s[n0 + n], grp[m][n][i], acc[m][n0 + n][i]);
                    // the sums are made here: sunk to their use in a later step,
                    // they would keep the group's accumulators alive
                    asm volatile("" : "+v"(acc[m][n0 + n]));
                }
            }
        }
    }
}

// The steps' activations in LDS: fragments and group sums of `steps` steps.
constexpr int step_lds_bytes(int MT, int G) { return MT * (kStepChunks * 1024 + 128 / G * 64); }

// The adapters of a tile's rows, one byte per row tile m: that of row m * 16 +
// lane % 16, 0xff for none.
__device__ __forceinline__ unsigned long long adapters_used(uint32_t adapters, int n_mt)
{
    unsigned long long used = 0;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const uint32_t l = (adapters >> (8 * m)) & 0xffu;
        if (m < n_mt && l != 0xffu)
            used |= 1ull << l;
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1)  // lanes 0..15 hold all rows
        used |= __shfl_xor(used, off);
    return uniform_u64(used);
}

// The expand step after e, or l < 0: rank positions of one adapter first, then
// the next of `used`.
__device__ __forceinline__ ExpandStep next_expand(ExpandStep e, unsigned long long *used, int r)
{
    if (e.l >= 0 && e.q0 + 32 < r)
        return ExpandStep{e.l, e.q0 + 32};
    if (!*used)
        return ExpandStep{-1, 0};
    const int l = (int)__builtin_ctzll(*used);
    *used &= *used - 1;
    return ExpandStep{l, 0};
}

// Whether an expand step's operand may hold an infinity or NaN.  Read as fp16,
// those bf16 bit patterns are all NaN, and so are the finite ones above 2^121,
// which only cost time; a NaN survives a maximum.
__device__ __forceinline__ bool maybe_nonfinite(const u32x4 (&b)[kNS])
{
    typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
    f16x2 top = {0, 0};
#pragma unroll
    for (int n = 0; n < kNS; ++n) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t u = b[n][i], v = b[n][i + 1];
            top = __builtin_elementwise_maximum(
                __builtin_elementwise_maximum(top, __builtin_bit_cast(f16x2, u)), __builtin_bit_cast(f16x2, v));
        }
    }
    return top.x != top.x || top.y != top.y;
}

// The whole expand of a wave, over NM of MT row tiles, with NE steps' operands
// in flight: the steps of `used` adapters in order, each its rank positions.
// Rows of other adapters, or of none, meet an adapter's B rows as zeros.  Where
// a B row holds an infinity or NaN, 0 times it is NaN, so steps that may
// hold one are left for a second pass, which adds to the adapter's own rows only.
template <int NM, int MT, int NE>
struct Expand {
    unsigned long long used;
    ExpandStep at;      // the next one to load, l < 0: none
    ExpandStep e[NE];
    u32x4 b[NE][kNS];

    __device__ __forceinline__ void load(int i, const GemmW4Args &a, const SlabW4 &w, int I, int lane)
    {
        e[i] = at;
        if (at.l >= 0) {  // uniform
            load_expand(b[i], a, w, at, I, lane);
            at = next_expand(at, &used, a.r);
        }
    }
    __device__ __forceinline__ void start(unsigned long long adapters, const GemmW4Args &a, const SlabW4 &w,
                                          int I, int lane)
    {
        used = adapters;
        at = next_expand(ExpandStep{-1, 0}, &used, a.r);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            load(i, a, w, I, lane);
    }
    // sfrag: S fragments [rank chunk][m][lane]
    __device__ __forceinline__ void run(f32x4 (&acc)[NM][kNS], const GemmW4Args &a, const SlabW4 &w, int I,
                                        uint32_t adapters, const u32x4 *sfrag, int lane)
    {
        unsigned long long wild = 0;  // adapters with steps left for run_wild
        while (e[0].l >= 0) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                if (e[i].l < 0)
                    continue;
                if (a.r & 7)
                    fix_expand(b[i], a, w, e[i], I, lane);
                if (__ballot(maybe_nonfinite(b[i]))) {  // uniform
                    wild |= 1ull << e[i].l;
                } else {
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const u32x4 v = keep_if(sfrag[(e[i].q0 / 32 * MT + m) * kWave + lane],
                                                ((adapters >> (8 * m)) & 0xffu) == (uint32_t)e[i].l);
#pragma unroll
                        for (int n = 0; n < kNS; ++n)
                            acc[m][n] = mfma_16x16x32(v, b[i][n], acc[m][n]);
                    }
                }
                load(i, a, w, I, lane);
            }
        }
        if (wild)
            run_wild(acc, wild, a, w, I, adapters, sfrag, lane);
    }
    // The steps that may hold infinities or NaN of the adapters in `wild`: products apart
    // from the sums, added to the rows of the step's adapter only.
    __device__ __forceinline__ void run_wild(f32x4 (&acc)[NM][kNS], unsigned long long wild, const GemmW4Args &a,
                                             const SlabW4 &w, int I, uint32_t adapters, const u32x4 *sfrag,
                                             int lane)
    {
        for (ExpandStep s = next_expand(ExpandStep{-1, 0}, &wild, a.r); s.l >= 0; s = next_expand(s, &wild, a.r)) {
            u32x4 v[kNS];
            load_expand(v, a, w, s, I, lane);
            if (a.r & 7)
                fix_expand(v, a, w, s, I, lane);
            if (!__ballot(maybe_nonfinite(v)))
                continue;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const u32x4 x = sfrag[(s.q0 / 32 * MT + m) * kWave + lane];
                unsigned own = 0;  // bit j: row 4 (lane / 16) + j is the adapter's
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    own |= (((__shfl(adapters, (lane >> 4) * 4 + j) >> (8 * m)) & 0xffu) == (uint32_t)s.l) << j;
#pragma unroll
                for (int n = 0; n < kNS; ++n) {
                    const f32x4 part = mfma_16x16x32(x, v[n], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[m][n][j] += (own >> j) & 1 ? part[j] : 0.0f;
                }
            }
        }
    }
};

// The lane's row of row tile m of a tile: the adapter (0xff: none), and the
// activation row and slot where `mine`.
template <bool kGated>
__device__ __forceinline__ uint32_t find_row(const GemmW4Args &a, int p, bool mine, const uint16_t **row, int *slot)
{
    uint32_t adapter = 0xffu;
    if (kGated || a.S) {
        const int x = a.perm2exp[p];
        const int tok = x / a.k;
        const int l = a.S && a.mapping ? a.mapping[tok] : -1;
        adapter = l >= 0 && l < a.L ? (uint32_t)l : 0xffu;
        if (mine) {
            *row = a.X + (size_t)(kGated ? tok : p) * a.K;
            *slot = x;
        }
    } else if (mine) {
        *row = a.X + (size_t)p * a.K;
    }
    return adapter;
}

// One S fragment (32 rank positions of a row tile) from the lane's slot; bf16, as
// the shrinks, which the bf16 layer uses too, leave it.
__device__ __forceinline__ u32x4 load_s(const GemmW4Args &a, int slot, int chunk, int lane)
{
    const int q = chunk * 32 + (lane >> 4) * 8;
    return keep_if(load16(a.S + (size_t)slot * a.rp + min(q, a.rp - 8)), q < a.rp);
}

// Writes a wave's 64 columns of a tile from its accumulators: lane l holds
// rows 4 (l / 16) + i of column l % 16, and gate and up of a column sit in
// neighbouring tiles of the same lane.  The activations are rounded to bf16, as
// in the bf16 layer: they are the down product's MFMA operand, and two operands
// for their upper and lower halves would double its matrix work.  With the bf16
// shrink outputs (the expand's operand, for the same reason) the layer errs by
// 2.4e-3 against 64 bits, in 2-norms, where rounding the exact output to bf16
// errs by 1.7e-3.
template <int NM, bool kGated>
__device__ __forceinline__ void store_slab(const f32x4 (&acc)[NM][kNS], const GemmW4Args &a, int row0,
                                           int n_rows, int slab, int lane)
{
    asm("" : "+v"(lane));  // addresses are made here, not kept through the main loop
    const int width = kGated ? a.I : a.n_canon;
    const size_t base = (size_t)row0 * width + slab * (kGated ? 32 : 64);  // uniform
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = m * 16 + (lane >> 4) * 4 + i;
            const size_t at = base + (size_t)(unsigned)row * width + (lane & 15);
            if (row < n_rows) {
                if (kGated) {
                    uint16_t *y = static_cast<uint16_t *>(a.Y) + at;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        y[j * 16] = (uint16_t)float_to_bf16_bits(silu_f32(acc[m][2 * j][i]) * acc[m][2 * j + 1][i]);
                } else if (a.y_f32) {
#pragma unroll
                    for (int n = 0; n < kNS; ++n)
                        static_cast<float *>(a.Y)[at + n * 16] = acc[m][n][i];
                } else {
#pragma unroll
                    for (int n = 0; n < kNS; ++n)
                        static_cast<uint16_t *>(a.Y)[at + n * 16] = (uint16_t)float_to_bf16_bits(acc[m][n][i]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// f with the group size and the flags as constants.
template <typename F>
hipError_t with_format(int group, bool gated, bool zeros, F f)
{
    auto flags = [&](auto G) {
        using T = std::true_type;
        using N = std::false_type;
        return gated ? (zeros ? f(G, T{}, T{}) : f(G, T{}, N{})) : (zeros ? f(G, N{}, T{}) : f(G, N{}, N{}));
    };
    return group == 32   ? flags(std::integral_constant<int, 32>{})
           : group == 64 ? flags(std::integral_constant<int, 64>{})
                         : flags(std::integral_constant<int, 128>{});
}

} // namespace
} // namespace moe_lora
