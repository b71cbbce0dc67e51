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
