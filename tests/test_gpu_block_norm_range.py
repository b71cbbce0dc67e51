"""Block norms at the ends of what their documentation allows: no rows, values and eps far from one."""
import pytest
import torch

from sparse_expert_moe_b200 import moe

from test_gpu_block_norm import U32, backward, check, f64, gate64, make, pullback64, tiny

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


@pytest.mark.parametrize("T,d", [(8, 264), (8, 16384), (1500, 1024), (4800, 136)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_backward_of_rows_far_from_one(T, d, gate):
    """Rows of zeros, of values near one, 1e15 and 1e-13, with an eps of 1e-30 (1 / sqrt(mean square +
    eps) up to 1e15): its cube leaves the range of fp32, the gradients do not.  Tolerances as in the
    test of the formula, the magnitudes being those of each row."""
    eps = 1e-30
    x = make(T, d, gate, "f32", "f32", "f32", seed=19)
    scale = torch.tensor([0.0, 1.0, 1e15, 1e-13], device=DEV)[torch.arange(T, device=DEV) % 4][:, None]
    x["r"] *= scale
    x["y"] *= scale.roll(1, 0)
    x["dh"] *= 1e-2
    x["dr_out"] *= 1e-2
    got = backward(x, x["r"], T, d, gate, "f32", "f32", "f32", eps=eps)
    e = torch.tensor(eps, dtype=torch.float32).double().item()
    none = torch.zeros(T, d, device=DEV, dtype=torch.float64)
    dx, tol, dwp, tdwp, _ = pullback64(f64(x["r"]), f64(x["w_pre"]), 0.0, f64(x["dh"]), none, e)
    G = f64(x["dr_out"]) + dx
    tG = tol + 4 * U32 * (G.abs() + dx.abs())
    check(got["dr"], G, U32 * G.abs() + tG + 2 * U32 * G.abs() + tiny("f32"), "dr")
    check(got["dw_pre"], dwp.sum(0), tdwp.sum(0) + (T + 64) * U32 * dwp.abs().sum(0), "dw_pre")
    g = gate64(x, gate)
    dy, tdy, dwq, tdwq, _ = pullback64(f64(x["y"]), f64(x["w_post"]), 0.0, g * G,
                                       g.abs() * (tG + 4 * U32 * G.abs()), e)
    check(got["dy"], dy, U32 * dy.abs() + tdy + tiny("f32"), "dy")
    check(got["dw_post"], dwq.sum(0), tdwq.sum(0) + (T + 64) * U32 * dwq.abs().sum(0), "dw_post")
