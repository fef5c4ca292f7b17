"""No kernel of the block keeps registers in scratch memory (no GPU needed)."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_up_amd import build

SOURCES = ["block_norm.hip", "clip.hip", "column_sums.hip", "linear_grad.hip"]


@pytest.mark.parametrize("name", SOURCES)
def test_no_scratch(name, tmp_path):
    out = tmp_path / "out.s"
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, name), "-o",
                    str(out)], check=True, capture_output=True)
    kernels = re.findall(r"\.name:\s+(_Z\S+).*?\.private_segment_fixed_size:\s+(\d+).*?\.vgpr_spill_count:\s+(\d+)",
                         out.read_text(), re.S)
    assert kernels
    bad = [(k, int(scratch), int(spills)) for k, scratch, spills in kernels if int(scratch) or int(spills)]
    assert not bad, bad
