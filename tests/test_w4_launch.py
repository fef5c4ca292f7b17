"""How the 4-bit products are cut into blocks, on a machine without a GPU: the
rules of w4_launch.h, compiled as plain C++."""
import subprocess

import pytest

from mixture_experts_layer_up_amd import build

PROGRAM = r"""
#include <cstdio>
#include "w4_launch.h"
using namespace moe_lora;

int main()
{
    int a, b;
    while (std::scanf("%d %d", &a, &b) == 2)
        std::printf("%d\n", w4_groups_per_block(a, b));
    return 0;
}
"""

# Layers (arguments of a case in _w4.py) whose products run several slab groups
# a block; what each product's column count gives is asserted below and their
# results in test_gpu_w4_blocks.py.  32- and 64-row tiles; K of one, an even and an
# odd number of steps; a shorter last job; column counts that end inside a group;
# adapters.
BLOCKS = [
    dict(name="rows32_down", T=4000, H=4288, I=96, E=4, k=1, L=2, rg=8, rd=16, group=32, zeros=1),
    dict(name="rows32_down_whole_jobs", T=4000, H=4608, I=128, E=4, k=1, L=2, rg=0, rd=40, group=128),
    dict(name="rows32_gate_up", T=4000, H=320, I=2144, E=4, k=1, L=2, rg=13, rd=8, group=64, zeros=1),
    dict(name="rows32_gate_up_even", T=4000, H=192, I=2208, E=4, k=1, L=3, rg=40, rd=0, group=128),
    dict(name="rows64_down", T=8200, H=4288, I=64, E=3, k=1, L=2, rg=8, rd=72, group=64, zeros=1),
    dict(name="rows64_both", T=16400, H=1280, I=608, E=4, k=2, L=2, rg=16, rd=8, group=128),
    dict(name="rows64_gate_up", T=8200, H=320, I=2144, E=3, k=1, L=2, rg=64, rd=8, group=32, zeros=1),
]


@pytest.fixture(scope="session")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("w4_launch")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{build.CSRC}", str(d / "rule.cpp"), "-o", str(d / "rule")],
                   check=True, capture_output=True)

    def call(pairs):
        text = "".join(f"{a} {b}\n" for a, b in pairs)
        r = subprocess.run([str(d / "rule")], input=text, capture_output=True, text=True, check=True)
        return [int(v) for v in r.stdout.split()]
    return call


def test_groups_per_block_are_even_and_make_enough_blocks(rule):
    """Jobs of one tile differ by less than the number of jobs allows: the longest
    is no longer than the mean, rounded up, and one job fewer would leave too few
    blocks."""
    pairs = [(t, n) for t in (1, 3, 16, 60, 128, 200, 511, 512, 600, 1023, 1024, 5000) for n in range(1, 40)]
    for (tiles, n_sg), per in zip(pairs, rule(pairs)):
        jobs = -(-n_sg // per)
        assert 1 <= per <= n_sg
        assert per == -(-n_sg // jobs), f"{tiles} tiles, {n_sg} groups: {jobs} jobs of up to {per}"
        assert jobs == n_sg or tiles * jobs >= 1024
        # one job fewer, where the groups can be cut so
        fewer = [j for j in range(1, jobs) if -(-n_sg // -(-n_sg // j)) == j]
        assert not fewer or tiles * fewer[-1] < 1024


@pytest.mark.parametrize("c", BLOCKS, ids=lambda c: c["name"])
def test_blocks_cases_run_several_groups(rule, c):
    rows = int(c["name"][4:6])
    tiles = c["T"] * c["k"] // rows
    n_sg = {"gate_up": -(-2 * c["I"] // 256), "down": -(-c["H"] // 256)}
    named = [p for p in n_sg if p in c["name"]] or list(n_sg)
    per = dict(zip(named, rule([(tiles, n_sg[p]) for p in named])))
    assert all(2 <= v <= n_sg[p] for p, v in per.items()), per
    short = {p for p, v in per.items() if n_sg[p] % v}
    assert bool(short) == (c["name"] not in ("rows32_down_whole_jobs", "rows32_gate_up_even"))
