"""moe_grouped_gemm and its gradients against sums in 64 bits.

Tolerance per element.  The tensor cores add 16 (e4m3: 32) exact products to the accumulator in
one step, cutting each addend at 2^-23 of the largest; with S the sum of the products'
magnitudes that is at most 2^-23 S per addend, K + K / 16 addends in all.  e4m3 adds one
rounding per product of two scales and per block of 128.  The result rounds once to its type:
eps / 2 of its value."""
import numpy as np
import pytest
import torch

from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CUT = 2.0 ** -23


def offsets_of(sizes, start=0):
    return torch.from_numpy(np.concatenate([[start], start + np.cumsum(sizes)]).astype(np.int32)).to(DEV)


def workspace(cfg):
    return torch.zeros(moe.moe_product_workspace_size(cfg), dtype=torch.uint8, device=DEV)


def randn(seed, *shape):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(torch.bfloat16)


def within(got, ref, mag, K, out, extra=0.0):
    tol = torch.finfo(TYPES[out]).eps / 2 * ref.abs() + ((K + K / 16 + 16) * CUT + extra) * mag
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((got.double() - ref).abs().max()), bad.nonzero()[:4].tolist())


def run_rows(op, sizes, n, k, out="bf16", start=0, spare=0, seed=0, poison=True):
    """Forward or dgrad on ragged groups; rows outside the groups hold NaN and must neither
    be used nor written."""
    G, used = len(sizes), sum(sizes)
    R = start + used + spare
    inner, outer = (k, n) if op == "gemm" else (n, k)
    cfg = moe.make_product_config(G, R, n, k, out=out)
    x, w = randn(seed + 1, R, inner), randn(seed + 2, G, n, k)
    if poison:
        x[:start] = float("nan")
        x[start + used:] = float("nan")
    y = torch.full((R, outer), -7.0, device=DEV, dtype=TYPES[out])
    ws = workspace(cfg)
    off = offsets_of(sizes, start)
    if op == "gemm":
        moe.moe_grouped_gemm(cfg, off, x, None, w, None, y, ws)
    else:
        moe.moe_grouped_gemm_dgrad(cfg, off, x, w, y, ws)
    assert moe.moe_read_device_status(ws) == 0
    assert (ws[:256] == 0).all()                       # join counters left as they were found
    lo = start
    for g, m in enumerate(sizes):
        wm = w[g].double()
        wm = wm.T if op == "gemm" else wm
        xs = x[lo:lo + m].double()
        within(y[lo:lo + m], xs @ wm, xs.abs() @ wm.abs(), inner, out)
        lo += m
    assert (y[:start] == -7).all() and (y[lo:] == -7).all()
    return y


# small groups (stream kernel): one row, empties, 16 / 17 / 32 / 33 rows, odd sizes of n and k
FEW = [([1], 128, 64), ([1], 8, 8), ([5, 0, 1, 16, 17, 0, 32, 33], 256, 256), ([3, 0, 0, 2], 264, 200),
       ([1] * 40, 136, 72), ([8, 8, 8], 520, 1032), ([0, 0, 7], 1000, 328), ([200] + [0] * 30, 384, 640)]
# larger groups (pair kernel): 256-row tiles and their edges, several tiles per group
MANY = [([300], 256, 128), ([256], 256, 64), ([257, 0, 255, 31, 500], 264, 200), ([33], 8, 8),
        ([1000, 1, 700], 512, 1032), ([64, 65, 96, 97], 136, 520), ([2100], 1000, 328)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", FEW + MANY)
def test_rows_forward(sizes, n, k, out):
    run_rows("gemm", sizes, n, k, out, start=3, spare=5)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", FEW + MANY)
def test_rows_gradient(sizes, n, k, out):
    run_rows("dgrad", sizes, n, k, out, start=3, spare=5)


@pytest.mark.parametrize("op", ["gemm", "dgrad"])
@pytest.mark.parametrize("sizes", [[1], [24], [129], [700]])
def test_long_inner_sums_are_shared_out(op, sizes):
    """Few tiles, many K blocks: every CTA takes a share of the same tiles."""
    one = run_rows(op, sizes, 512, 4096, "f32") if op == "gemm" else run_rows(op, sizes, 4096, 512, "f32")
    two = run_rows(op, sizes, 512, 4096, "f32") if op == "gemm" else run_rows(op, sizes, 4096, 512, "f32")
    assert torch.equal(one, two)                        # joined in a fixed order


def test_no_offsets_is_one_group():
    for R in (1, 40, 300):
        cfg = moe.make_product_config(1, R, 256, 192)
        x, w, ws = randn(1, R, 192), randn(2, 1, 256, 192), workspace(cfg)
        y = torch.empty(R, 256, device=DEV, dtype=torch.bfloat16)
        z = torch.empty_like(y)
        moe.moe_grouped_gemm(cfg, None, x, None, w, None, y, ws)
        moe.moe_grouped_gemm(cfg, offsets_of([R]), x, None, w, None, z, ws)
        assert torch.equal(y, z)
        within(y, x.double() @ w[0].double().T, x.double().abs() @ w[0].double().abs().T, 192, "bf16")


# ------------------------------------------------------------------------------------ weights
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", [([1], 8, 8), ([17], 128, 128), ([64], 256, 256), ([5, 0, 63, 65, 16], 264, 200),
                                       ([0, 0], 64, 72), ([300, 1, 129], 136, 520), ([1000, 40], 512, 136),
                                       ([3000], 128, 264), ([2049], 40, 1032)])
def test_weight_gradient(sizes, n, k, out, start=2, spare=9):
    G, used = len(sizes), sum(sizes)
    R = start + used + spare
    cfg = moe.make_product_config(G, R, n, k, out=out)
    dy, a = randn(3, R, n), randn(4, R, k)
    dy[:start] = float("nan")
    a[start + used:] = float("inf")                     # rows of nobody, right behind the last group
    dy[start + used:] = float("nan")
    dw = torch.full((G, n, k), float("nan"), device=DEV, dtype=TYPES[out])
    ws = workspace(cfg)
    moe.moe_grouped_gemm_wgrad(cfg, offsets_of(sizes, start), dy, a, dw, ws)
    assert moe.moe_read_device_status(ws) == 0 and (ws[:256] == 0).all()
    lo = start
    for g, m in enumerate(sizes):
        d, x = dy[lo:lo + m].double(), a[lo:lo + m].double()
        within(dw[g], d.T @ x, d.abs().T @ x.abs(), m, out)
        if m == 0:
            assert (dw[g] == 0).all()
        lo += m


def test_weight_gradient_keeps_the_next_group_out():
    """A group of NaN rows between two others: only its own gradient has them."""
    sizes, n, k = [37, 20, 50], 136, 72
    R = sum(sizes)
    cfg = moe.make_product_config(3, R, n, k, out="f32")
    dy, a = randn(5, R, n), randn(6, R, k)
    dy[37:57] = float("nan")
    a[37:57] = float("nan")
    dw = torch.empty(3, n, k, device=DEV)
    ws = workspace(cfg)
    moe.moe_grouped_gemm_wgrad(cfg, offsets_of(sizes), dy, a, dw, ws)
    assert torch.isnan(dw[1]).all() and torch.isfinite(dw[0]).all() and torch.isfinite(dw[2]).all()


def test_weight_gradient_without_rows():
    cfg = moe.make_product_config(2, 0, 16, 24, out="f32")
    dw = torch.full((2, 16, 24), float("nan"), device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm_wgrad(cfg, off, 256, 256, dw, workspace(cfg))
    assert (dw == 0).all()


# ------------------------------------------------------------------------------------ e4m3
def codes(seed, *shape):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)


def fp8_case(sizes, n, k, out="bf16", start=0, spare=0, seed=0):
    G, used = len(sizes), sum(sizes)
    R = start + used + spare
    kb, nb = -(-k // 128), -(-n // 128)
    cfg = moe.make_product_config(G, R, n, k, dtype="e4m3_fs", out=out)
    a, w = codes(seed + 1, R, k), codes(seed + 2, G, n, k)
    g = torch.Generator(DEV).manual_seed(seed + 3)
    sa = torch.rand(R, kb, device=DEV, generator=g) + 0.3
    sw = torch.rand(G, nb, kb, device=DEV, generator=g) - 0.4     # any finite value: negative too
    if spare:
        a.view(torch.uint8)[start + used:] = 0x7F                 # NaN codes outside the groups
        sa[start + used:] = float("inf")
    y = torch.full((R, n), -7.0, device=DEV, dtype=TYPES[out])
    ws = workspace(cfg)
    moe.moe_grouped_gemm(cfg, offsets_of(sizes, start), a, sa, w, sw, y, ws)
    assert moe.moe_read_device_status(ws) == 0 and (ws[:256] == 0).all()
    lo = start
    for i, m in enumerate(sizes):
        if m:
            x = a[lo:lo + m].double() * sa[lo:lo + m].double().repeat_interleave(128, 1)[:, :k]
            v = w[i].double() * sw[i].double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
            # 32 products per step: fewer cuts than `within` counts; scales and blocks: kb + 2 roundings
            within(y[lo:lo + m], x @ v.T, x.abs() @ v.abs().T, 128, out, extra=(kb + 2) * 2.0 ** -24)
        lo += m
    assert (y[:start] == -7).all() and (y[lo:] == -7).all()
    return y


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", [
    ([1], 128, 128), ([1], 8, 16), ([1], 264, 144), ([5, 0, 1, 16, 17, 0, 32, 33], 256, 256), ([3, 0, 0, 2], 392, 2064),
    ([1] * 20, 136, 1200), ([300], 256, 128), ([257, 0, 255, 31, 500], 264, 400), ([33], 8, 16),
    ([128, 129, 160, 1], 640, 1040), ([1100], 200, 2064)])
def test_block_scaled_product(sizes, n, k, out):
    fp8_case(sizes, n, k, out, start=1, spare=4)


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_block_scaled_long_sums_are_shared_out(rows):
    assert torch.equal(fp8_case([rows], 384, 7168, "f32"), fp8_case([rows], 384, 7168, "f32"))


# ------------------------------------------------------------------------------------ faults
@pytest.mark.parametrize("off", [[0, 5, 3], [0, 3, 11], [-1, 3, 5]])
def test_bad_offsets_set_the_status_and_write_nothing(off):
    cfg = moe.make_product_config(2, 10, 64, 64)
    off = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, w = randn(1, 10, 64), randn(2, 2, 64, 64)
    for op in ("gemm", "dgrad", "wgrad"):
        ws = workspace(cfg)
        out = torch.full((2, 64, 64) if op == "wgrad" else (10, 64), -7.0, device=DEV, dtype=torch.bfloat16)
        if op == "gemm":
            moe.moe_grouped_gemm(cfg, off, x, None, w, None, out, ws)
        elif op == "dgrad":
            moe.moe_grouped_gemm_dgrad(cfg, off, x, w, out, ws)
        else:
            moe.moe_grouped_gemm_wgrad(cfg, off, x, x, out, ws)
        assert moe.moe_read_device_status(ws) == 5
        assert (out == -7).all()


def test_captured_and_replayed_on_another_stream():
    """The three products captured into one graph, replayed on new inputs."""
    sizes, n, k = [40, 0, 300, 5], 264, 328
    R = sum(sizes)
    cfg = moe.make_product_config(4, R, n, k, out="f32")
    off, ws = offsets_of(sizes), workspace(cfg)
    a, dy, w = randn(1, R, k), randn(2, R, n), randn(3, 4, n, k)
    y, da, dw = (torch.empty(s, device=DEV) for s in ((R, n), (R, k), (4, n, k)))

    def calls():
        moe.moe_grouped_gemm(cfg, off, a, None, w, None, y, ws)
        moe.moe_grouped_gemm_dgrad(cfg, off, dy, w, da, ws)
        moe.moe_grouped_gemm_wgrad(cfg, off, dy, a, dw, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    a.copy_(randn(11, R, k))
    dy.copy_(randn(12, R, n))
    w.copy_(randn(13, 4, n, k))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, da, dw)]
    calls()
    torch.cuda.synchronize()
    for g, e in zip(got, (y, da, dw)):
        assert torch.equal(g, e)
    assert moe.moe_read_device_status(ws) == 0
