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
