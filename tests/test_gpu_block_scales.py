"""Block scales of the 8-bit product whose product is at the ends of the range of fp32, in both kernels,
beside rows and columns with ordinary scales."""
import pytest
import torch

from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [[5], [20, 0, 30], [150], [300, 7, 90]]


def spread(s, rows, cols):
    """A block scale [.., ceil(k / 128)] over the values it stands for, `rows` of them per row."""
    return s.double().repeat_interleave(128, -1)[..., :cols].repeat_interleave(rows, -2)


def make(sizes, out, huge):
    """Rows by turns with scales near one, 2^70, 2^-75 and zero; blocks of 128 columns with scales near
    `huge`, 2^-65 and one.  Where large scales meet the codes are zero or the smallest."""
    n, k = 384, 400
    G, R, kb = len(sizes), sum(sizes), 4
    g = torch.Generator(DEV).manual_seed(R)

    def rand(*s):
        return torch.rand(*s, device=DEV, generator=g)

    a = (torch.randn(R, k, device=DEV, generator=g) * 100).clamp(-448, 448)
    w = (torch.randn(G, n, k, device=DEV, generator=g) * 100).clamp(-448, 448)
    a[1::4] = (rand(len(range(1, R, 4)), k) < 0.1) * 2.0 ** -9     # (the smallest code)
    w[:, :128] = (rand(G, 128, k) < 0.1) * 2.0 ** -9
    a[:, 256:384] = 0                                              # a block without values
    a, w = a.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
    sa, sw = 1 + rand(R, kb), 1 + rand(G, 3, kb)
    sa[1::4] *= 2.0 ** 69
    sa[2::4] *= 2.0 ** -75
    sa[3::4] = 0
    sw[:, 0] *= -huge / 2
    sw[:, 1] *= 2.0 ** -65
    cfg = moe.make_product_config(G, R, n, k, dtype="e4m3_fs", out=out)
    ws = torch.zeros(moe.moe_product_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    y = torch.full((R, n), float("nan"), device=DEV, dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    off = torch.tensor([0] + sizes, device=DEV).cumsum(0).to(torch.int32)
    moe.moe_grouped_gemm(cfg, off, a, sa, w, sw, y, ws)
    return a, sa, w, sw, y, ws


def check(sizes, a, sa, w, sw, y, part):
    """The outputs that `part` picks.  Tolerance: 128 products of a block cut at 2^-23 of the largest, in
    8 steps at most, one rounding for each block and its factor, and the output's; and for each of the 4
    blocks half a step of the subnormals, 2^-150, times 128 * 448^2 < 2^25 where its factor is one."""
    k, kb, lo = a.shape[1], 4, 0
    f = torch.finfo(y.dtype)
    for i, m in enumerate(sizes):
        x = a[lo:lo + m].double() * spread(sa[lo:lo + m], 1, k)
        v = w[i].double() * spread(sw[i], 128, k)
        ref, mag = x @ v.T, x.abs() @ v.abs().T
        tol = f.eps / 2 * ref.abs() + ((128 + 8 + 16) * 2.0 ** -23 + (kb + 2) * 2.0 ** -24) * mag
        tol = tol + kb * 2.0 ** -125 + f.smallest_normal * f.eps   # (the output's own subnormals)
        bad = ~((y[lo:lo + m].double() - ref).abs() <= tol) & part(torch.arange(lo, lo + m, device=DEV))
        assert not bad.any(), (i, int(bad.sum()), bad.nonzero()[:4].tolist())
        lo += m


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES)
def test_products_of_scales_from_the_smallest_to_the_largest(sizes, out):
    """Products of scales from 2^-140 to just below 2^127: every output."""
    *x, y, ws = make(sizes, out, 2.0 ** 57)
    assert moe.moe_read_device_status(ws) == 0
    check(sizes, *x, y, lambda rows: torch.ones(len(rows), 384, device=DEV, dtype=torch.bool))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES)
def test_products_of_scales_past_the_largest_number_are_reported(sizes, out):
    """Scales of 2^70 that meet in 128 columns of every fourth row: the status says so, those outputs are
    infinite or NaN, and all others are right."""
    *x, y, ws = make(sizes, out, 2.0 ** 70)
    assert moe.moe_read_device_status(ws) == 7
    columns = torch.arange(384, device=DEV) < 128
    assert not torch.isfinite(y[1::4, :128]).any()
    check(sizes, *x, y, lambda rows: ~((rows % 4 == 1)[:, None] & columns))
    moe.moe_reset_device_status(ws)
    assert moe.moe_read_device_status(ws) == 0
