"""How the 4-bit products are cut into blocks, on a machine without a GPU: the
rules of w4_launch.h, compiled as plain C++."""
import subprocess

import pytest

from mixture_experts_layer_up_amd import build

PROGRAM = r"""
#include <cstdio>
#include "w4_launch.h"
using namespace moe_lora;

// lines "groups tiles n_sg" -> groups per block; "layer T k E E_l n_slabs steps"
// -> rows per tile, row tiles, groups per block, log2 of the K shares
int main()
{
    char what[16];
    int T, k, E, E_l, slabs, steps;
    while (std::scanf("%15s", what) == 1) {
        if (what[0] == 'g') {
            if (std::scanf("%d %d", &T, &k) != 2)
                return 1;
            std::printf("%d\n", w4_groups_per_block(T, k));
            continue;
        }
        if (std::scanf("%d %d %d %d %d %d", &T, &k, &E, &E_l, &slabs, &steps) != 6)
            return 1;
        const int n = T * k, rows = w4_tile_rows(n, E, E_l), local = w4_local_slots(n, E, E_l);
        const int busy = local < E_l ? local : E_l, tiles = w4_row_tiles(n / rows + E_l, busy, local, rows);
        std::printf("%d %d %d %d\n", rows, tiles, w4_groups_per_block(tiles, (slabs + 3) / 4),
                    w4_k_shares_log(busy, slabs, steps));
    }
    return 0;
}
"""

# Layers (arguments of a case in _w4.py) whose products run several slab groups
# a block; what each product's column count gives is asserted below and their
# results in test_gpu_w4_blocks.py.  32- and 64-row tiles; K of one, an even and an
# odd number of steps; a shorter last job; column counts that end inside a group;
# adapters.
BLOCKS = [
    dict(name="rows32_down", T=4000, H=8384, I=96, E=4, k=1, L=2, rg=8, rd=16, group=32, zeros=1),
    dict(name="rows32_down_whole_jobs", T=4000, H=8704, I=128, E=4, k=1, L=2, rg=0, rd=40, group=128),
    dict(name="rows32_gate_up", T=4000, H=320, I=4192, E=4, k=1, L=2, rg=13, rd=8, group=64, zeros=1),
    dict(name="rows32_gate_up_even", T=4000, H=192, I=4320, E=4, k=1, L=3, rg=40, rd=0, group=128),
    dict(name="rows64_down", T=8200, H=8384, I=64, E=3, k=1, L=2, rg=8, rd=72, group=64, zeros=1),
    dict(name="rows64_both", T=16400, H=1792, I=864, E=4, k=2, L=2, rg=16, rd=8, group=128),
    dict(name="rows64_gate_up", T=8200, H=320, I=4192, E=3, k=1, L=2, rg=64, rd=8, group=32, zeros=1),
]


@pytest.fixture(scope="session")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("w4_launch")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{build.CSRC}", str(d / "rule.cpp"), "-o", str(d / "rule")],
                   check=True, capture_output=True)

    def call(what, cases):
        text = "".join(f"{what} {' '.join(map(str, c))}\n" for c in cases)
        r = subprocess.run([str(d / "rule")], input=text, capture_output=True, text=True, check=True)
        rows = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
        return [v[0] if what == "groups" else v for v in rows]
    return call


def test_groups_per_block_are_even_and_make_enough_blocks(rule):
    """Jobs of one tile differ by less than the number of jobs allows: the longest
    is no longer than the mean, rounded up, and one job fewer would leave too few
    blocks."""
    pairs = [(t, n) for t in (1, 3, 16, 60, 128, 200, 511, 512, 600, 1023, 1024, 2048, 5000) for n in range(1, 40)]
    for (tiles, n_sg), per in zip(pairs, rule("groups", pairs)):
        jobs = -(-n_sg // per)
        assert 1 <= per <= n_sg
        assert per == -(-n_sg // jobs), f"{tiles} tiles, {n_sg} groups: {jobs} jobs of up to {per}"
        assert jobs == n_sg or tiles * jobs >= 2048
        # one job fewer, where the groups can be cut so
        fewer = [j for j in range(1, jobs) if -(-n_sg // -(-n_sg // j)) == j]
        assert not fewer or tiles * fewer[-1] < 2048


def _layer(c):
    """Rule arguments of gate_up and down."""
    E_l = c.get("E_l") or c["E"]
    return {p: (c["T"], c["k"], c["E"], E_l, N // 64, -(-K // 128))
            for p, N, K in (("gate_up", 2 * c["I"], c["H"]), ("down", c["H"], c["I"]))}


@pytest.mark.parametrize("c", BLOCKS, ids=lambda c: c["name"])
def test_blocks_cases_run_several_groups(rule, c):
    args = {p: a for p, a in _layer(c).items() if p in c["name"] or c["name"] == "rows64_both"}
    short = False
    for a, (rows, tiles, per, _) in zip(args.values(), rule("layer", args.values())):
        n_sg = -(-a[4] // 4)
        assert rows == int(c["name"][4:6]) and 2 <= per <= n_sg
        short |= n_sg % per > 0
    assert short == (c["name"] not in ("rows32_down_whole_jobs", "rows32_gate_up_even"))


@pytest.mark.parametrize("T,k,E,E_l", [(2048, 8, 128, 16), (8192, 8, 256, 32), (1024, 4, 64, 8), (16384, 8, 256, 32)])
def test_shards_are_cut_by_their_own_slots(rule, T, k, E, E_l):
    """A shard's many-row launches make blocks for the slots it gets, as a layer of
    its experts alone with that many slots would."""
    hidden, inter = 2048, 768
    shard = _layer(dict(T=T, k=k, E=E, E_l=E_l, H=hidden, I=inter))
    alone = _layer(dict(T=T * E_l // E, k=k, E=E_l, H=hidden, I=inter))
    for s, a in zip(rule("layer", shard.values()), rule("layer", alone.values())):
        assert s == a
    for (rows, tiles, per, _), a in zip(rule("layer", shard.values()), shard.values()):
        n_sg = -(-a[4] // 4)
        assert rows > 16 and tiles * rows <= max(T * k * E_l // E, E_l * rows)
        assert per == 1 or tiles * -(-n_sg // per) >= 2048


@pytest.mark.parametrize("T", [1, 2, 4, 8])
def test_few_tokens_of_a_shard_share_k(rule, T):
    """K is cut until the slabs of the experts that the shard's slots touch make a
    wave per SIMD (1024) or there are 8 shares."""
    for a in _layer(dict(T=T, k=8, E=128, E_l=16, H=2048, I=768)).values():
        (rows, _, _, log), = rule("layer", [a])
        busy = min(16, T)  # T * 8 * 16 / 128 slots
        assert rows == 16
        assert log == 3 or busy * a[4] << log >= 1024 or a[5] >> (log + 1) < 1
