"""Block norms at the ends of what their documentation allows: no rows, values and eps far from one."""
import pytest
import torch

from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def norm_ws(cfg):
    return torch.empty(moe.moe_norm_workspace_size(cfg), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("captured", [False, True])
def test_sums_over_no_rows_are_zero_whatever_they_are_multiplied_by(captured):
    d = 264
    cfg = moe.make_norm_config(0, d, gate="channel")
    ws = norm_ws(cfg)
    e = torch.empty(0, d, device=DEV, dtype=BF)
    w = torch.ones(d, device=DEV, dtype=BF)
    w[3], w[200] = float("inf"), float("nan")
    sums = [torch.full((d,), 5.0, device=DEV) for _ in range(3)]

    def call():
        moe.moe_block_norm_backward(cfg, e, e, w, w, w, e, e, e, e, *sums, ws)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graph.replay()
    else:
        call()
    for s in sums:
        assert (s == 0).all()
