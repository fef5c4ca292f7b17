// w4_layout.h -- where the packed 4-bit expert weights lie.
//
// A 4-bit expert weight of one projection is w[k][n] = (q[k][n] - z[g][n]) s[g][n]
// with codes q and zero points z in 0..15 (z = 8 everywhere when the format has
// none), bf16 scales s, and groups g = k / group of consecutive K rows.
//
// Packed, per expert e and 64-column slab s (the slabs and their column order
// are those of the bf16 pack, pack.hip), three regions follow each other:
//   codes   unit u of 64 K rows x 64 columns = 2048 bytes at
//           ((e * NS + s) * KU + u) * 2048; inside, half h (column tiles 2h,
//           2h + 1), lane l, word i: the 32-bit word holds the 8 codes of rows
//           64 u + 32 (i & 1) + 8 (l / 16) + 0..7, column l % 16 of tile
//           2h + i / 2: what one lane feeds one 16x16x32 MFMA as B operand.
//           One 16-byte load per lane and half is 1 KiB contiguous.
//   scales  bf16 at ((e * NS + s) * NG + g) * 64 + (column % 16) * 4 + tile:
//           a lane's four tiles are one 8-byte load
//   zeros   bytes 16 + z in the same order (formats with zero points only):
//           what the products subtract, one conversion from float
// Row counts that are not whole steps of 128 rows (two units) are padded with
// units of code 0, which meet zero activations.
//
// Nibble order inside a word.  The MFMA operand wants bf16 pairs (rows 2j,
// 2j + 1) in one register.  With 16 + q = bits 0x4180 | q << 3, the
// code of row 2j sits at bit 3 + 4j and that of row 2j + 1 at bit 19 + 4j,
// both modulo 32 (the last nibble wraps): rotating the word right by 4j and
// one and-or then make the pair, 7 instructions for 8 weights.
#pragma once

#include <stddef.h>
#include <stdint.h>

#if defined(__HIP__)
#define MOE_LORA_W4_HD __host__ __device__
#else
#define MOE_LORA_W4_HD
#endif

namespace moe_lora {

constexpr int kW4UnitK = 64;         // K rows of one unit
constexpr int kW4UnitBytes = 2048;   // 64 x 64 codes

struct W4Layout {
    int n_slabs;     // 64-column slabs: N / 64
    int k_units;     // units that cover K, in whole steps
    int n_groups;    // ceil(K / group)
    size_t scales;   // byte offset of the scales region
    size_t zeros;    // byte offset of the zero points (= bytes when there are none)
    size_t bytes;
};

MOE_LORA_W4_HD inline W4Layout w4_layout(int E_l, int K, int N, int group, bool has_zeros)
{
    W4Layout l;
    l.n_slabs = N / 64;
    l.k_units = (K + 2 * kW4UnitK - 1) / (2 * kW4UnitK) * 2;
    l.n_groups = (K + group - 1) / group;
    const size_t slabs = (size_t)E_l * l.n_slabs;
    l.scales = slabs * l.k_units * kW4UnitBytes;          // a multiple of 2048
    l.zeros = l.scales + slabs * l.n_groups * 64 * 2;     // a multiple of 128
    l.bytes = l.zeros + (has_zeros ? slabs * l.n_groups * 64 : 0);
    return l;
}

// Bit position of the code of row i (0..7) in its word.
MOE_LORA_W4_HD inline int w4_nibble_bit(int i)
{
    return (3 + 4 * (i >> 1) + 16 * (i & 1)) & 31;
}

// Column of the unpacked weight that column c (0..15) of tile t (0..3) of
// slab s holds: gate and up tiles alternate in gate_up (I > 0), as in pack.hip.
MOE_LORA_W4_HD inline int w4_column(int slab, int t, int c, int I)
{
    const int nt = slab * 4 + t;
    return I > 0 ? (nt & 1) * I + (nt >> 1) * 16 + c : nt * 16 + c;
}

} // namespace moe_lora
