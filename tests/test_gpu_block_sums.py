"""How far the sums of the grouped products may be off, by the length of the inner index."""
import pytest
import torch

from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def product_ws(cfg):
    return torch.zeros(moe.moe_product_workspace_size(cfg), dtype=torch.uint8, device=DEV)


def product(op, x, y, out):
    """One group: x [rows, inner] with y [n, k] (rows for wgrad); y's layout is the op's."""
    rows = x.shape[0]
    n, k = {"gemm": y.shape, "dgrad": y.shape, "wgrad": (y.shape[1], x.shape[1])}[op]
    cfg = moe.make_product_config(1, rows, n, k, out="bf16" if out == BF else "f32")
    ws = product_ws(cfg)
    if op == "wgrad":
        got = torch.empty(n, k, device=DEV, dtype=out)
        moe.moe_grouped_gemm_wgrad(cfg, None, y, x, got, ws)
    elif op == "gemm":
        got = torch.empty(rows, n, device=DEV, dtype=out)
        moe.moe_grouped_gemm(cfg, None, x, None, y, None, got, ws)
    else:
        got = torch.empty(rows, k, device=DEV, dtype=out)
        moe.moe_grouped_gemm_dgrad(cfg, None, x, y, got, ws)
    assert moe.moe_read_device_status(ws) == 0
    return got


@pytest.mark.parametrize("op,rows,n,k", [("gemm", 3, 38400, 7168), ("gemm", 300, 10240, 7168), ("dgrad", 5, 7168, 38400),
                                         ("dgrad", 260, 7168, 10240), ("wgrad", 7168, 2048, 2560)])
def test_bf16_outputs_are_roundings_of_32_bit_sums(op, rows, n, k):
    """A bf16 output is the rounding of a sum whose root mean square error is below 50 * 2^-24 of the
    results' (the bound of the fp32 outputs: 512 products at a time on the tensor cores).  Such a sum
    rounds to another value than the exact one where a border between two values lies between them: with
    probability |error| / spacing, and then by one spacing, at most 2^-7 of the value.  So the squares of
    the differences add up to |error| * spacing <= |error| * 2^-7 * |value| per element, and by Cauchy
    and Schwarz to 50 * 2^-24 * 2^-7 of the results' squares: a relative 2-norm below 1.53e-4."""
    g = torch.Generator(DEV).manual_seed(5)
    x = torch.randn(rows, n if op == "dgrad" else k, device=DEV, generator=g).to(BF)
    y = torch.randn(*((rows, n) if op == "wgrad" else (n, k)), device=DEV, generator=g).to(BF)
    got = product(op, x, y, BF)
    ref = {"wgrad": lambda: y.double().T @ x.double(), "gemm": lambda: x.double() @ y.double().T,
           "dgrad": lambda: x.double() @ y.double()}[op]()
    rounded = ref.to(BF).double()
    off = float((got.double() - rounded).norm() / rounded.norm())
    assert off <= (50 * 2.0 ** -24 * 2.0 ** -7) ** 0.5, off


@pytest.mark.parametrize("groups,rows", [(2, 1 << 20), (2, 1 << 23), (1, 1 << 24)])
def test_sums_over_millions_of_rows(groups, rows):
    """A weight gradient over so many rows that adding sums of 512 one after another would round the
    same way thousands of times.  dy is 1, and each 512 rows of a add up to 512 + j / 128 exactly (j
    per column), which every binade of a running sum cuts off elsewhere.  Of m sums of 512, 64 are
    added to one, and those m / 64 to the next, with one rounding of half a step each; up to 4 parts
    of a cut tile and the output round once more: 64 + m / 64 + 5 times 2^-24 of the value."""
    total = groups * rows
    a = torch.ones(total, 8, device=DEV, dtype=BF)
    extra = (4 * torch.arange(8, device=DEV) + 3).to(BF) / 128
    a.view(-1, 512, 8)[:, 5] += extra
    dy = torch.ones(total, 8, device=DEV, dtype=BF)
    cfg = moe.make_product_config(groups, total, 8, 8, out="f32")
    off = (rows * torch.arange(groups + 1, device=DEV)).to(torch.int32)
    ws, dw = product_ws(cfg), torch.empty(groups, 8, 8, device=DEV)
    moe.moe_grouped_gemm_wgrad(cfg, off, dy, a, dw, ws)
    assert moe.moe_read_device_status(ws) == 0 and (ws[:256] == 0).all()
    m = rows // 512
    want = m * (512 + extra.double())
    off = float(((dw.double() - want).abs() / want).max())
    assert off <= (64 + m / 64 + 5) * 2.0 ** -24, off


@pytest.mark.parametrize("out", [BF, torch.float32])
def test_long_ragged_weight_gradients(out):
    """Groups of odd sizes on both sides of the second level of sums, columns behind a tile's last.  In
    32 bits the root mean square of the errors is below that of one sum of 512 (32 steps of the tensor
    cores, 2^-24 each) and of the roundings of 64 + 3 additions and 5 of parts and output, 104 * 2^-24
    of the results' (running sums are smaller than their results)."""
    sizes, n, k = [70001, 0, 5, 32768, 32769, 40003], 264, 200
    g = torch.Generator(DEV).manual_seed(9)
    R = sum(sizes) + 7
    dy, a = (torch.randn(R, c, device=DEV, generator=g).to(BF) for c in (n, k))
    dy[sum(sizes):] = float("nan")
    off = torch.tensor([0] + sizes, device=DEV).cumsum(0).to(torch.int32)
    cfg = moe.make_product_config(len(sizes), R, n, k, out="bf16" if out == BF else "f32")
    ws, dw = product_ws(cfg), torch.full((len(sizes), n, k), float("nan"), device=DEV, dtype=out)
    moe.moe_grouped_gemm_wgrad(cfg, off, dy, a, dw, ws)
    assert moe.moe_read_device_status(ws) == 0 and (ws[:256] == 0).all()
    bar = 104 * 2.0 ** -24
    for i, m in enumerate(sizes):
        lo = sum(sizes[:i])
        ref = dy[lo:lo + m].double().T @ a[lo:lo + m].double()
        if out == BF:                            # see test_bf16_outputs_are_roundings_of_32_bit_sums
            ref = ref.to(BF).double()
        error = (dw[i].double() - ref).square().mean().sqrt()
        assert error <= (bar if out != BF else (bar * 2.0 ** -7) ** 0.5) * ref.square().mean().sqrt(), (m, float(error))
