"""Tree attention on the GPU with a node_start that does not divide the nodes."""
import pytest
import torch

from distillation_ce_tvd_gb300 import binding
from test_gpu_tree_attention import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 8), (72, 16), (128, 5)])
@pytest.mark.parametrize("starts", [[0, 3, 2, 9], [0, 3, 5, 8], [0, 3, 5, 10], [1, 3, 5, 9],
                                    [-1, 3, 5, 9], [0, 3, 12, 9]])
def test_it_is_reported(dim, page, starts):
    c = case([20, 30, 40], [3, 2, 4], 4, 2, dim, page, tree=False, seed=dim)
    ref, _ = check(c)
    c["starts"] = starts
    out, _, st = run(c)
    assert st == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    if starts[:2] == [0, 3] and min(starts[1:]) == 3:      # request 0 is as before, and alone in its rows
        assert torch.equal(out[:3], ref[:3])
