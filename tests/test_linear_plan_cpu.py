"""Which kernel a product takes, seen in its workspace (no GPU needed): the one for few
rows needs none, tiles need a padded copy of a weight whose width is no multiple of 8."""
import pytest

from mixture_experts_layer_up_amd import binding

SWIGLU = binding.ACTIVATIONS.index("swiglu")


# rows, terms, columns; microseconds of the few-row kernel and of tiles
@pytest.mark.parametrize("M,K,N", [(512, 64, 1085),      # 10.4, 7.7
                                   (512, 2048, 333),     # 23.5, 17.9
                                   (200, 4096, 1085)])   # 42.4, 38.1
def test_two_projections_cost_more(M, K, N):
    """swiglu's blocks have twice the columns: where a CU runs several, tiles win earlier."""
    assert binding.linear_workspace_size(binding.LinearShape(M, K, N, SWIGLU, 0)) > 0
    assert binding.linear_workspace_size(binding.LinearShape(M // 4, K, N, SWIGLU, 0)) == 0
    assert binding.linear_workspace_size(binding.LinearShape(M // 4, K, N, 0, 0)) == 0
