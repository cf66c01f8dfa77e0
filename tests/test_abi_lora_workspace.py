"""How the adapters' weight gradients split their rows, seen in the workspace they ask
for, without a GPU."""
import pytest

import mixture_experts_layer_06_amd as moe


@pytest.mark.parametrize("dt,cols", [(moe.BF16, 128), (moe.F32, 64)])
@pytest.mark.parametrize("e,M", [(1, 4096), (1, 512), (3, 9000), (4, 16384), (1, 100000)])
@pytest.mark.parametrize("R", [1, 2, 3, 4, 7, 8, 16, 64])
def test_stretches_of_256_rows_at_least(dt, cols, e, M, R):
    """A column more of A within a block's columns, where only the stretches' partial sums
    grow: stretches x adapters x ranks x 4 bytes."""
    lo, hi = (moe.lora_bwd_workspace_size(dt, e, M, h, 64, R) for h in (cols - 32, cols))
    stretches = (hi - lo) / (32 * e * R * 4)
    assert stretches <= max(1, M // e // 256) + 256 / (32 * e * R * 4)  # sizes are multiples of 256
