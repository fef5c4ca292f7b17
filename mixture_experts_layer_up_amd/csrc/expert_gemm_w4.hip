// expert_gemm_w4.hip -- grouped expert products with 4-bit weights.
//
// What is computed is what expert_gemm.hip computes, with expert weights
// w[k][n] = s[g][n] (q[k][n] - z[g][n]), g = k / group (w4_layout.h):
//   gate_up:  h = x_t W13[e] + B_gu[l,e] s_gu[p];  act[p] = SiLU(h[:I]) h[I:]
//   down:     y[p] = act[p] W2[e] + B_dn[l,e] s_dn[p]
//
// The codes never become rounded weights.  A code enters the MFMA as the
// exact bf16 number v = (16 + q) / 16 (one rotate and one and-or per pair of
// weights), and per group, with x's group sum taken by one more MFMA against
// ones (its accumulator has the layout of the others),
//   sum_k x_k w_k = 16 s ( sum_k x_k v_k  -  (16 + z) / 16 sum_k x_k )
// in fp32.  bf16 products are exact in fp32, so the only roundings are the
// fp32 sums'; the subtraction cancels at most a factor of about (16 + z) / 8
// of their 24 bits.
//
// Design for gfx950, few rows per expert: as in expert_gemm.hip a block is 4
// waves on one (row tile, 64-column slab), the waves split K and reduce
// through LDS, the codes go from memory straight into registers.
#include <algorithm>

#include "device_common.h"
#include "gemm_index.h"
#include "kernels_w4.h"
#include "mfma_pipeline.h"
#include "w4_layout.h"

namespace moe_lora {
namespace {

// One unit's operands of one wave: 64 K rows x 64 columns of codes, the rows'
// activations, the scales (and zero points) of the unit's groups.
template <int MT, bool kZeros>
struct UnitW4 {
    u32x4 b[2];       // [h]: tiles 2h, 2h + 1; word (tile & 1) * 2 + chunk
    u32x4 a[2][MT];   // [chunk][row tile]
    uint2 sc[2];      // [chunk]: four tiles' bf16 scales
    uint32_t zr[2];   // [chunk]: four tiles' zero points
};

// Four exact bf16 pairs (16 + q) / 16 of one word of codes.
__device__ __forceinline__ u32x4 decode_w4(uint32_t w)
{
    constexpr uint32_t kMask = 0x00780078u, kOne = 0x3f803f80u;
    return u32x4{(w & kMask) | kOne, (__builtin_amdgcn_alignbit(w, w, 4) & kMask) | kOne,
                 (__builtin_amdgcn_alignbit(w, w, 8) & kMask) | kOne,
                 (__builtin_amdgcn_alignbit(w, w, 12) & kMask) | kOne};
}

template <int MT, int D, bool kGated, bool kRank8, bool kZeros>
__global__ __launch_bounds__(256, MT == 1 ? 3 : MT == 2 ? 2 : 1) void expert_gemm_w4_kernel(GemmW4Args a)
{
    constexpr int NS = kNS;
    __shared__ float part[Part<MT>::kFloats];
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = wave_id();

    const int logical = xcd_balanced_item(blockIdx.x, *a.tile_count * a.n_slabs);
    if (logical < 0)
        return;
    const int4 te = a.tiles[logical / a.n_slabs];
    const int le = te.x;
    if (le < 0)
        return;
    const int nt = (te.z + a.tile_rows - 1) / a.tile_rows;
    const int in_expert = logical - te.w * a.n_slabs;
    const int slab = in_expert / nt;
    const int sub = in_expert - slab * nt;
    const int row0 = te.y + sub * a.tile_rows;
    const int n_rows = min(a.tile_rows, te.z - sub * a.tile_rows);
    const int n_mt = (n_rows + 15) >> 4;

    // contiguous run of units of this wave
    const int ub = wave * a.k_units / 4, ue = (wave + 1) * a.k_units / 4;
    const int nu = ue - ub;
    const size_t slab_index = (size_t)le * a.n_slabs + slab;
    const uint8_t *codes = a.codes + slab_index * a.k_units * kW4UnitBytes + lane * 16;
    const uint16_t *scales = a.scales + slab_index * a.n_groups * 64 + (lane & 15) * 4;
    const uint8_t *zeros = kZeros ? a.zeros + slab_index * a.n_groups * 64 + (lane & 15) * 4 : nullptr;

    const bool lora = a.S != nullptr && a.L > 0 && a.r > 0;
    const uint16_t *aptr[MT];
    int xslot[MT];
    int adapter[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int p = row0 + min(m * 16 + (lane & 15), n_rows - 1);
        const int x = a.perm2exp[p];
        xslot[m] = x;
        const int tok = x / a.k;
        aptr[m] = a.X + (size_t)(a.gather_by_token ? tok : p) * a.K + (lane >> 4) * 8;
        const int l = (lora && a.mapping) ? a.mapping[tok] : -1;
        adapter[m] = (l >= 0 && l < a.L) ? l : -1;
    }

    auto load_unit = [&](UnitW4<MT, kZeros> &st, int i) {
        const int u = min(ub + i, a.k_units - 1);
        const uint8_t *pc = codes + (size_t)u * kW4UnitBytes;
        st.b[0] = load16_stream(pc);
        st.b[1] = load16_stream(pc + 1024);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int k0 = min(u * 64 + c * 32, a.K - 32);
            const int g = k0 / a.group;
            st.sc[c] = *reinterpret_cast<const uint2 *>(scales + (size_t)g * 64);
            if (kZeros)
                st.zr[c] = *reinterpret_cast<const uint32_t *>(zeros + (size_t)g * 64);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (m < n_mt)
                    st.a[c][m] = load16(aptr[m] + k0);
        }
    };

    f32x4 acc[MT][NS], grp[MT][NS], xs[MT];
    zero_acc(acc);
    zero_acc(grp);
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xs[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const u32x4 ones{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};

    auto close_group = [&](uint2 sc, uint32_t zr) {
        const float s[NS] = {bf16_bits_to_float(sc.x & 0xffffu), bf16_bits_to_float(sc.x >> 16),
                             bf16_bits_to_float(sc.y & 0xffffu), bf16_bits_to_float(sc.y >> 16)};
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const float z = kZeros ? (float)((zr >> (8 * n)) & 0xffu) : 8.0f;
            const float c = (16.0f + z) * 0.0625f;
            const float s16 = s[n] * 16.0f;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[m][n][i] = fmaf(s16, fmaf(-c, xs[m][i], grp[m][n][i]), acc[m][n][i]);
                grp[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
            xs[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };

    auto compute_unit = [&](const UnitW4<MT, kZeros> &st, int i) {
        const int u = ub + i;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int k0 = u * 64 + c * 32;
            if (k0 < a.K) {
                u32x4 b[NS];
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    b[n] = decode_w4(st.b[n >> 1][(n & 1) * 2 + c]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m < n_mt) {
                        xs[m] = mfma_16x16x32(st.a[c][m], ones, xs[m]);
#pragma unroll
                        for (int n = 0; n < NS; ++n)
                            grp[m][n] = mfma_16x16x32(st.a[c][m], b[n], grp[m][n]);
                    }
                }
                const int k1 = k0 + 32;
                if (k1 % a.group == 0 || k1 >= a.K || (c == 1 && i == nu - 1))
                    close_group(st.sc[c], st.zr[c]);
            }
        }
    };

    if (nu > 0) {
        UnitW4<MT, kZeros> st[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
            load_unit(st[d], d);
        for (int i0 = 0; i0 < nu; i0 += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i0 + d < nu)
                    compute_unit(st[d], i0 + d);
                load_unit(st[d], i0 + d + D);
            }
        }
    }

    // LoRA expand: 32 rank positions of the concatenated adapters per chunk,
    // waves take chunks round-robin; rows keep only their own adapter's block
    if (lora) {
        const DecodeBShape bs{0, NS, a.n_slabs, kGated ? 1 : 0, a.I, a.L, a.r, a.rp,
                              a.E_l, a.n_canon, a.lb_shared};
        const int n_ext = (a.L * a.rp + 31) >> 5;
        for (int vc = 0; vc * 4 + wave < n_ext; ++vc) {
            u32x4 b[NS];
            const int g = (vc * 4 + wave) * 32 + (lane >> 4) * 8;
            const int aid = g / a.rp, q0 = g - aid * a.rp;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const DecodeBLoad d = decode_b_load(bs, wave, lane, vc, 0, le, slab, n);
                if (kRank8) {
                    b[n] = load16_stream(a.LB + d.off16);
                } else {
                    const uint16_t *pe = a.LB + d.lora_row;
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const uint32_t lo = pe[min(d.q0 + i, a.r - 1)];
                        const uint32_t hi = pe[min(d.q0 + i + 1, a.r - 1)];
                        w[i >> 1] = (d.q0 + i < a.r ? lo : 0u) | ((d.q0 + i + 1 < a.r ? hi : 0u) << 16);
                    }
                    b[n] = keep_if(u32x4{w[0], w[1], w[2], w[3]}, d.aid < a.L);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m < n_mt) {
                    // the load stays in S's row for every lane; other adapters' lanes keep 0
                    const u32x4 sv = keep_if(load16(a.S + (size_t)xslot[m] * a.rp + q0), adapter[m] == aid);
#pragma unroll
                    for (int n = 0; n < NS; ++n)
                        acc[m][n] = mfma_16x16x32(sv, b[n], acc[m][n]);
                }
            }
        }
    }

    store_partials<MT, NS>(part, acc, n_mt, wave, lane);
    __syncthreads();

    if (kGated) {
        uint16_t *Y = static_cast<uint16_t *>(a.Y);
        for (int item = tid; item < n_rows * 4; item += 256) {
            const int row = item >> 2;
            const int jj = (item >> 1) & 1;
            const int c0 = (item & 1) * 8;
            uint32_t packed[4];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float gate = sum_partials<MT>(part, row, (2 * jj) * 16 + c0 + i + h);
                    const float up = sum_partials<MT>(part, row, (2 * jj + 1) * 16 + c0 + i + h);
                    v[h] = silu_f32(gate) * up;
                }
                packed[i >> 1] = float_to_bf16_bits(v[0]) | (float_to_bf16_bits(v[1]) << 16);
            }
            store16(Y + (size_t)(row0 + row) * a.I + (slab * 2 + jj) * 16 + c0,
                    u32x4{packed[0], packed[1], packed[2], packed[3]});
        }
    } else {
        for (int item = tid; item < n_rows * 8; item += 256) {
            const int row = item >> 3;
            const int c0 = (item & 7) * 8;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = sum_partials<MT>(part, row, c0 + i);
            const size_t at = (size_t)(row0 + row) * a.n_canon + slab * 64 + c0;
            if (a.y_f32) {
                float *Y = static_cast<float *>(a.Y) + at;
                store16(Y, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
                store16(Y + 4, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
            } else {
                uint32_t packed[4];
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    packed[i >> 1] = float_to_bf16_bits(v[i]) | (float_to_bf16_bits(v[i + 1]) << 16);
                store16(static_cast<uint16_t *>(a.Y) + at,
                        u32x4{packed[0], packed[1], packed[2], packed[3]});
            }
        }
    }
}

template <int MT, int D, bool kGated, bool kRank8>
hipError_t launch_rank(const GemmW4Args &a, int blocks, hipStream_t s)
{
    if (a.zeros)
        hipLaunchKernelGGL((expert_gemm_w4_kernel<MT, D, kGated, kRank8, true>), dim3(blocks), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((expert_gemm_w4_kernel<MT, D, kGated, kRank8, false>), dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <bool kGated, bool kRank8>
hipError_t launch_rows(const GemmW4Args &a, int blocks, hipStream_t s)
{
    switch (a.tile_rows) {
    case 16:
        return launch_rank<1, 4, kGated, kRank8>(a, blocks, s);
    case 32:
        return launch_rank<2, 2, kGated, kRank8>(a, blocks, s);
    default:
        return launch_rank<4, 2, kGated, kRank8>(a, blocks, s);
    }
}

} // namespace

int gemm_w4_tile_rows(int n_slots, int E_l)
{
    const int mean = n_slots / std::max(1, E_l);
    return mean <= 10 ? 16 : mean <= 24 ? 32 : 64;
}

hipError_t launch_gemm_w4(const GemmW4Args &a, bool gated, hipStream_t s)
{
    const int blocks = (a.n_tiles * a.n_slabs + 7) / 8 * 8;
    if (blocks <= 0)
        return hipSuccess;
    const bool rank8 = (a.r & 7) == 0;
    if (gated)
        return rank8 ? launch_rows<true, true>(a, blocks, s) : launch_rows<true, false>(a, blocks, s);
    return rank8 ? launch_rows<false, true>(a, blocks, s) : launch_rows<false, false>(a, blocks, s);
}

} // namespace moe_lora
