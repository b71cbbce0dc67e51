"""The block norms and the grouped products where they are in full swing: rows staged ahead and a ring
that wraps, CTAs that take several tiles, pieces that end one tile and begin the next.  The shapes
are taken from the conditions that choose the kernels; formulas and tolerances are those of
test_gpu_block_norm.py and test_gpu_grouped_product.py."""
import random

import numpy as np
import pytest
import torch

import oracle
import test_gpu_block_norm as norms
import test_gpu_grouped_product as products
from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


# ------------------------------------------------------------------------------------ norms
def staged_forward(T, d, res, act, gate, branch):
    """The host's rule: two vectors of 8 per thread up to d = 8192, four above; four and three stages."""
    nvec = d // 8
    vpt, stages = (2, 4) if nvec <= 1024 else (4, 3)
    tpr = -(-(-(-nvec // vpt)) // 32) * 32
    size = {"bf16": 1, "f32": 2}
    units = size[res] + (branch + (gate == "full")) * size[act]
    return nvec > 64 and stages * vpt * 512 * 16 * units <= 216 * 1024 and T >= stages * 148 * (512 // tpr)


@pytest.mark.parametrize("T,d,gate,res,act,out,post,pre,branch", [
    (1501, 7168, "none", "bf16", "bf16", "bf16", True, True, True),
    (1501, 7168, "channel", "bf16", "bf16", "bf16", True, True, True),
    (1501, 7168, "token", "bf16", "bf16", "f32", True, True, True),
    (1501, 7168, "full", "bf16", "bf16", "bf16", True, True, True),
    (1501, 7168, "token", "f32", "bf16", "bf16", True, True, True),
    (1501, 7168, "channel", "bf16", "f32", "f32", True, True, True),
    (1501, 7168, "channel", "bf16", "bf16", "bf16", False, True, True),
    (1501, 7168, "token", "bf16", "bf16", "bf16", True, False, True),
    (1501, 7168, "none", "f32", "f32", "f32", False, True, False),
    (4801, 1024, "token", "bf16", "bf16", "bf16", True, True, True),      # eight rows per CTA
    (4801, 1024, "full", "bf16", "bf16", "bf16", True, True, True),
    (3001, 1032, "token", "bf16", "bf16", "bf16", True, True, True),      # threads without a second vector
    (3001, 1032, "none", "f32", "bf16", "f32", True, True, True),
    (1501, 4096, "token", "f32", "bf16", "bf16", True, True, True),       # two rows per CTA
    (1501, 8192, "full", "bf16", "bf16", "bf16", True, True, True),
    (700, 9000, "token", "bf16", "bf16", "bf16", True, True, True),       # four vectors, some without
    (700, 16384, "channel", "bf16", "bf16", "bf16", True, True, True),
    (700, 16384, "none", "f32", "f32", "bf16", False, True, False),
])
def test_staged_forward(T, d, gate, res, act, out, post, pre, branch):
    assert staged_forward(T, d, res, act, gate, branch)
    a, b, off = np.float32(0.9).item(), np.float32(0.7).item(), 1.0
    x = norms.make(T, d, gate, res, act, "bf16", post, pre, branch, seed=23)
    r_out, h, _ = norms.forward(x, T, d, gate, res, act, "bf16", out, a=a, b=b, off=off)
    r, mag, hr, hm = norms.reference(x, gate, 1e-6, a, b, off)
    U32 = norms.U32
    norms.check(r_out, r, norms.half_step(res) * r.abs() + 64 * U32 * mag + norms.tiny(res), "r_out")
    if pre:
        norms.check(h, hr, norms.half_step(out) * hr.abs() + 128 * U32 * hm + norms.tiny(out), "h")


@pytest.mark.parametrize("T,d,gate", [(1501, 7168, "token"), (3001, 1152, "channel"), (700, 16384, "none")])
def test_staged_rows_quantised(T, d, gate):
    assert staged_forward(T, d, "bf16", "bf16", gate, True)
    x = norms.make(T, d, gate, seed=29)
    x["r"][0, :128] = x["y"][0, :128] = 0
    _, h32, _ = norms.forward(x, T, d, gate, "bf16", "bf16", "bf16", "f32")
    _, codes, scale = norms.forward(x, T, d, gate, "bf16", "bf16", "bf16", "e4m3")
    r, mag, hr, hm = norms.reference(x, gate, 1e-6, 1.0, 1.0, 0.0)
    norms.check(h32, hr, norms.U32 * hr.abs() + 128 * norms.U32 * hm + norms.tiny("f32"), "h")
    want, ws = oracle.quantize_e4m3_blocks(h32.double().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), ws.astype(np.float32))
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want)


def staged_backward(T, d, res, act, gate):
    nvec = d // 8
    vpt = 1 if nvec <= 32 else 2
    rows = 512 // (-(-(-(-nvec // vpt)) // 32) * 32)
    size = {"bf16": 1, "f32": 2}
    units = 2 * size[res] + (2 + (gate == "full")) * size[act]
    # more than three rows per slot: the ring of three wraps
    return nvec <= 1024 and 3 * vpt * 512 * 16 * units <= 216 * 1024 and T > 3 * 148 * rows


@pytest.mark.parametrize("T,d,gate,res,act,post,pre,branch", [
    (1500, 7168, "token", "bf16", "bf16", True, True, True),
    (1500, 7168, "channel", "bf16", "bf16", True, True, True),
    (1500, 7168, "none", "bf16", "bf16", False, True, True),
    (1500, 7168, "token", "bf16", "bf16", True, False, True),
    (1500, 7168, "none", "bf16", "bf16", False, True, False),
    (5003, 520, "token", "bf16", "bf16", True, True, True),               # threads without a second vector
    (3001, 1032, "channel", "bf16", "bf16", True, True, True),
    (900, 8192, "token", "bf16", "bf16", True, True, True),
    (9001, 256, "full", "bf16", "bf16", True, True, True),                # sixteen rows per CTA
    (9001, 256, "token", "f32", "f32", True, True, True),
    (9001, 128, "full", "f32", "bf16", True, True, True),                 # half of the threads idle
])
def test_staged_backward(T, d, gate, res, act, post, pre, branch):
    assert staged_backward(T, d, res, act, gate)
    norms.test_backward_against_the_formula(T, d, gate, res, act, "bf16", post, pre, branch)


# ------------------------------------------------------------------------------------ products
def ragged(groups, most, seed):
    r = random.Random(seed)
    return [r.choice([0, r.randint(0, most), r.randint(0, most)]) for _ in range(groups)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["gemm", "dgrad"])
def test_several_tiles_per_pair(op, out):
    """99 tiles of 256 x 256 and more for 74 pairs: whole tiles, then a last round, cut or not."""
    for sizes, inner in (([700], 200), ([300, 0, 33, 500], 328), ([700], 1544)):
        n, k = (8200, inner) if op == "gemm" else (inner, 8200)
        products.run_rows(op, sizes, n, k, out, start=1, spare=3)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["gemm", "dgrad"])
def test_small_groups_shared_evenly(op, out):
    """75 tiles of 256 x 32 and more for 148 CTAs: every CTA's share ends one tile and begins the next."""
    for sizes, outer, inner in (([3], 38400, 328), (ragged(64, 14, 1), 1032, 584)):
        n, k = (outer, inner) if op == "gemm" else (inner, outer)
        assert sum(sizes) + 4 <= 8 * len(sizes) or sum(sizes) + 4 <= 32
        products.run_rows(op, sizes, n, k, out, start=1, spare=3)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", [([500, 0, 33, 1000], 2056, 2568), ([333], 2568, 2056)])
def test_several_weight_gradient_tiles_per_pair(sizes, n, k, out):
    products.test_weight_gradient(sizes, n, k, out)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", [
    ([1100], 5128, 1040),                        # 189 fold tiles of 128 x 256 for 148 CTAs, nine K blocks
    ([300, 0, 17, 800], 5128, 2064),
    ([3], 38400, 656),                           # stream kernel: 150 tiles
    (ragged(64, 14, 2), 1032, 1168)])            # ... and groups of a few rows
def test_block_scaled_product_in_steady_state(sizes, n, k, out):
    products.fp8_case(sizes, n, k, out, start=1, spare=4)


# ------------------------------------------------------------------------------------ order
def test_gates_and_scales_written_by_the_kernel_just_before():
    """Launches overlap the kernel before them.  A token gate (a gradient that the backward pass has
    just written) and the scales of e4m3 rows (of the norm just before, into both 8-bit kernels) are
    read behind the wait like everything else: the same results as with an idle GPU in between."""
    def case(T, d, n):
        g = torch.Generator(DEV).manual_seed(T)

        def rand(*s, dt=BF):
            return torch.randn(*s, device=DEV, generator=g).to(dt)
        w = torch.randn(1, n, d, device=DEV, generator=g).mul_(50).to(torch.float8_e4m3fn)
        return dict(T=T, d=d, n=n, w=w, sw=torch.rand(1, -(-n // 128), d // 128, device=DEV, generator=g),
                    wn=1 + rand(d, dt=torch.float32) * 0.1, gate=rand(T, dt=torch.float32),
                    ins=[[rand(T, d) for _ in range(4)] for _ in range(2)])

    def run(c, i, apart):
        T, d, n = c["T"], c["d"], c["n"]
        r, y, dh, dr = c["ins"][i]
        back = moe.make_norm_config(T, d, gate="token", weight="f32")
        quant = moe.make_norm_config(T, d, gate="token", weight="f32", out="e4m3")
        prod = moe.make_product_config(1, T, n, d, dtype="e4m3_fs", out="f32")
        steps = [
            lambda: moe.moe_block_norm_backward(back, r, y, c["wn"], c["gate"], c["wn"], dh, dr, c["dr"], c["dy"],
                                                c["dgate"], None, None, c["nws"]),
            lambda: moe.moe_block_norm(quant, c["dr"], c["dy"], c["wn"], c["dgate"], c["wn"], c["r1"], c["h"], c["hs"]),
            lambda: moe.moe_grouped_gemm(prod, None, c["h"], c["hs"], c["w"], c["sw"], c["out"], c["ws"]),
        ]
        for s in steps:
            s()
            if apart:
                torch.cuda.synchronize()
        return c["out"].clone(), c["r1"].clone(), c["hs"].clone()

    for T, d, n in ((20, 512, 384), (300, 2048, 640), (2000, 1024, 640)):
        c = case(T, d, n)
        back = moe.make_norm_config(T, d, gate="token", weight="f32")
        prod = moe.make_product_config(1, T, n, d, dtype="e4m3_fs", out="f32")
        c.update(dr=torch.empty(T, d, device=DEV, dtype=BF), dy=torch.empty(T, d, device=DEV, dtype=BF),
                 dgate=torch.empty(T, device=DEV), r1=torch.empty(T, d, device=DEV, dtype=BF),
                 h=torch.empty(T, d, device=DEV, dtype=torch.float8_e4m3fn), hs=torch.empty(T, d // 128, device=DEV),
                 out=torch.empty(T, n, device=DEV),
                 nws=torch.empty(moe.moe_norm_workspace_size(back), dtype=torch.uint8, device=DEV),
                 ws=torch.zeros(moe.moe_product_workspace_size(prod), dtype=torch.uint8, device=DEV))
        want = [run(c, i, True) for i in range(2)]
        for _ in range(20):
            for i in range(2):
                for have, ref in zip(run(c, i, False), want[i]):
                    assert torch.equal(have, ref)
        assert moe.moe_read_device_status(c["ws"]) == 0
