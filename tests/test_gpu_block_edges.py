"""Calls of the block norms and the grouped products that their documentation allows and that the
tests of their formulas do not make: outputs in place of inputs at sizes where rows are staged
ahead, tensors aligned to their elements or to 16 bytes only, the largest number of groups, a row
of NaN beside others."""
import numpy as np
import pytest
import torch

from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def randn(seed, *shape, dtype=BF):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def shifted(t, elements):
    """The same values in memory that starts `elements` behind an allocation's start."""
    flat = torch.empty(t.numel() + elements, device=t.device, dtype=t.dtype)
    out = flat[elements:].view(t.shape)
    out.copy_(t)
    return out


def same(a, b):
    """Equal, NaN with NaN (an e4m3 conversion of values past 448 leaves NaN codes)."""
    return torch.allclose(a, b, rtol=0, atol=0, equal_nan=True)


def norm_ws(cfg):
    return torch.empty(moe.moe_norm_workspace_size(cfg), dtype=torch.uint8, device=DEV)


def product_ws(cfg):
    return torch.zeros(moe.moe_product_workspace_size(cfg), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------ norms
@pytest.mark.parametrize("T,d", [(3, 7168), (1501, 7168), (4001, 1024), (700, 16384), (5003, 264)])
@pytest.mark.parametrize("gate", ["channel", "full"])
def test_forward_in_place(T, d, gate):
    r, y, w = randn(1, T, d), randn(2, T, d), randn(3, d)
    g = randn(4, d) if gate == "channel" else randn(4, T, d)
    cfg = moe.make_norm_config(T, d, gate=gate)
    want_r, want_h = torch.empty_like(r), torch.empty_like(r)
    moe.moe_block_norm(cfg, r, y, w, g, w, want_r, want_h, None)
    for place in ("y", "r"):
        a, b = r.clone(), y.clone()
        if place == "y":                         # r' over r, h over y
            moe.moe_block_norm(cfg, a, b, w, g, w, a, b, None)
            assert torch.equal(a, want_r) and torch.equal(b, want_h)
        else:                                    # h over r, r' not kept
            moe.moe_block_norm(cfg, a, b, w, g, w, None, a, None)
            assert torch.equal(a, want_h) and torch.equal(b, y)


@pytest.mark.parametrize("T,d", [(3, 7168), (1501, 7168), (4001, 1024), (300, 16384), (5003, 264)])
@pytest.mark.parametrize("gate", ["token", "full"])
def test_backward_in_place(T, d, gate):
    r, y, dh, dr, w = randn(1, T, d), randn(2, T, d), randn(5, T, d), randn(6, T, d), randn(3, d)
    g = randn(4, T) if gate == "token" else randn(4, T, d)
    cfg = moe.make_norm_config(T, d, gate=gate)
    ws = norm_ws(cfg)

    def call(y, dh, dr_out, dr_in, dy):
        dg = torch.empty_like(g, dtype=torch.float32 if gate == "token" else BF)
        dp, dq = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
        moe.moe_block_norm_backward(cfg, r, y, w, g, w, dh, dr_out, dr_in, dy, dg, dp, dq, ws)
        return dr_in, dy, dg, dp, dq
    want = call(y, dh, dr, torch.empty_like(r), torch.empty_like(y))
    a, b, c = y.clone(), dh.clone(), dr.clone()
    for got in (call(y, b, c, c, b), call(a, dh, dr, torch.empty_like(r), a)):
        for x, z in zip(got, want):
            assert torch.equal(x, z)


@pytest.mark.parametrize("T", [5, 2003])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_token_gates_and_scales_aligned_to_their_elements(T, dtype):
    d = 1024
    r, y, w, g = randn(1, T, d), randn(2, T, d), randn(3, d, dtype=dtype), randn(4, T, dtype=dtype)
    cfg = moe.make_norm_config(T, d, gate="token", weight="bf16" if dtype == BF else "f32", out="e4m3")
    got = []
    for gate, scale in ((g, torch.empty(T, d // 128, device=DEV)),
                        (shifted(g, 1), torch.empty(T * d // 128 + 1, device=DEV)[1:].view(T, d // 128))):
        h = torch.empty(T, d, device=DEV, dtype=torch.float8_e4m3fn)
        rp = torch.empty_like(r)
        moe.moe_block_norm(cfg, r, y, w, gate, w, rp, h, scale)
        dy, dr, dg = torch.empty_like(y), torch.empty_like(r), torch.empty(T + 1, device=DEV)[1:]
        moe.moe_block_norm_backward(cfg, rp, y, w, gate, w, y, r, dr, dy, dg, None, None, norm_ws(cfg))
        got.append((h.view(torch.uint8), scale, rp, dy, dr, dg))
    for x, z in zip(*got):
        assert torch.equal(x, z)


@pytest.mark.parametrize("T,d", [(7, 264), (2003, 7168)])
def test_norm_tensors_aligned_to_16_bytes(T, d):
    r, y, w, g = randn(1, T, d), randn(2, T, d), randn(3, d), randn(4, d)
    cfg = moe.make_norm_config(T, d, gate="channel")
    want = [torch.empty_like(r), torch.empty_like(r)]
    moe.moe_block_norm(cfg, r, y, w, g, w, *want, None)
    got = [shifted(torch.zeros_like(r), 8), shifted(torch.zeros_like(r), 24)]
    moe.moe_block_norm(cfg, shifted(r, 8), shifted(y, 40), shifted(w, 8), shifted(g, 16), shifted(w, 56), *got, None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------ products
def product(op, sizes, n, k, move=0, mark=None, out="bf16"):
    """One call; `move`: elements that every operand is moved by, `mark`: a row of NaN."""
    R, G = sum(sizes), len(sizes)
    fp8 = op == "fp8"
    cfg = moe.make_product_config(G, R, n, k, dtype="e4m3_fs" if fp8 else "bf16", out=out)
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    x, w = randn(1, R, n if op == "dgrad" else k), randn(2, G, n, k)
    dy = randn(5, R, n)
    sa = sw = None
    if fp8:
        x, w = (100 * x.float()).to(torch.float8_e4m3fn), (100 * w.float()).to(torch.float8_e4m3fn)
        sa = shifted(randn(6, R, -(-k // 128)).float(), move // 16)
        sw = shifted(randn(7, G, -(-n // 128), -(-k // 128)).float(), move // 16)
    if mark is not None:
        if fp8:
            x.view(torch.uint8)[mark] = 0x7F
        else:
            x[mark] = float("nan")
    x, w, dy = shifted(x, move), shifted(w, move), shifted(dy, move)
    shape = {"gemm": (R, n), "fp8": (R, n), "dgrad": (R, k), "wgrad": (G, n, k)}[op]
    y = shifted(torch.full(shape, -7.0, device=DEV, dtype=BF if out == "bf16" else torch.float32), move)
    ws = product_ws(cfg)
    if op == "dgrad":
        moe.moe_grouped_gemm_dgrad(cfg, off, x, w, y, ws)
    elif op == "wgrad":
        moe.moe_grouped_gemm_wgrad(cfg, off, dy, x, y, ws)
    else:
        moe.moe_grouped_gemm(cfg, off, x, sa, w, sw, y, ws)
    assert moe.moe_read_device_status(ws) == 0 and (ws[:256] == 0).all()
    return y


@pytest.mark.parametrize("op", ["gemm", "dgrad", "wgrad", "fp8"])
@pytest.mark.parametrize("sizes", [[1, 0, 6], [150, 3, 290]])
def test_operands_aligned_to_16_bytes(op, sizes):
    for out in ("bf16", "f32"):
        assert same(product(op, sizes, 264, 400, out=out), product(op, sizes, 264, 400, move=16, out=out))


@pytest.mark.parametrize("op", ["gemm", "dgrad", "fp8"])
@pytest.mark.parametrize("sizes,mark", [([3], 1), ([20, 0, 30], 25), ([300, 5], 140), ([90, 260], 91)])
def test_a_row_of_nan_stays_alone(op, sizes, mark):
    clean, got = product(op, sizes, 264, 400), product(op, sizes, 264, 400, mark=mark)
    assert torch.isnan(got[mark]).all()
    keep = [i for i in range(sum(sizes)) if i != mark]
    assert same(got[keep], clean[keep])


@pytest.mark.parametrize("op", ["gemm", "dgrad", "wgrad", "fp8"])
@pytest.mark.parametrize("rows", [1, 40])
def test_most_groups(op, rows):
    """1024 groups, most of them empty, against sums in 64 bits."""
    sizes = [0] * 1024
    for g in (0, 5, 511, 512, 1023):
        sizes[g] = rows
    n, k = 136, 64
    got = product(op, sizes, n, k, out="f32")
    R = sum(sizes)
    x, w = randn(1, R, n if op == "dgrad" else k), randn(2, 1024, n, k)
    lo = 0
    for g, m in enumerate(sizes):
        if op == "wgrad":
            if m == 0:
                assert (got[g] == 0).all()
                continue
            ref, mag = [f(randn(5, R, n)[lo:lo + m].double()).T @ f(x[lo:lo + m].double()) for f in (lambda v: v, abs)]
            inner, have = m, got[g]
        elif m == 0:
            continue
        elif op == "fp8":
            q, v = (100 * x.float()).to(torch.float8_e4m3fn), (100 * w[g].float()).to(torch.float8_e4m3fn)
            s = randn(6, R, 1).float().double()[lo:lo + m] * randn(7, 1024, 2, 1).float().double()[g].repeat_interleave(128, 0)[:n].T
            ref = (q[lo:lo + m].double() @ v.double().T) * s
            mag = (q[lo:lo + m].double().abs() @ v.double().T.abs()) * s.abs()
            inner, have = k, got[lo:lo + m]
        else:
            wm = w[g].double().T if op == "gemm" else w[g].double()
            ref, mag = x[lo:lo + m].double() @ wm, x[lo:lo + m].double().abs() @ wm.abs()
            inner, have = x.shape[1], got[lo:lo + m]
        lo += m
        # each of the inner + inner / 16 addends cut at 2^-23 of the largest; two scales: 3 roundings
        tol = ((inner + inner / 16 + 16) * 2.0 ** -23 + 3 * 2.0 ** -24) * mag + 2.0 ** -24 * ref.abs()
        assert (((have.double() - ref).abs() <= tol) | (torch.isnan(have) & torch.isnan(ref))).all(), g


# ------------------------------------------------------------------------------------ order
def test_each_call_waits_for_what_stands_before_it():
    """Launches overlap the kernel before them in the stream: what that one wrote is there all the
    same, behind copies, fills, kernels of others and work joined from another stream, eagerly and
    in a captured graph."""
    T, n, k = 300, 512, 2048
    x0, r0 = randn(1, T, k), randn(2, T, k)
    x1, r1 = randn(3, T, k), randn(4, T, k)
    w, w1, wn = randn(5, 1, n, k), randn(6, 1, k, n), randn(7, k)
    ncfg = moe.make_norm_config(T, k)
    pcfg, qcfg = moe.make_product_config(1, T, n, k), moe.make_product_config(1, T, k, n)
    ws, ws2 = product_ws(pcfg), product_ws(qcfg)
    x, r, h, y, z, out = (torch.empty(T, c, device=DEV, dtype=BF) for c in (k, k, k, n, k, k))
    side = torch.cuda.Stream()

    def chain(x_in, r_in):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            r.copy_(r_in)                        # a copy on another stream
        x.zero_()                                # a fill
        x.copy_(x_in)
        torch.cuda.current_stream().wait_stream(side)
        moe.moe_block_norm(ncfg, r, x, wn, None, wn, None, h, None)
        moe.moe_grouped_gemm(pcfg, None, h, None, w, None, y, ws)
        moe.moe_grouped_gemm(qcfg, None, y, None, w1, None, z, ws2)
        z.mul_(2.0 ** -11)                       # somebody else's kernel
        moe.moe_block_norm(ncfg, r, z, wn, None, wn, r, out, None)
        h.zero_()                                # behind the last reader
        return out

    def apart(x_in, r_in):
        """The same calls with the GPU idle between them."""
        torch.cuda.synchronize()
        a, b, c, d, e = (torch.empty_like(t) for t in (h, y, z, r, out))
        moe.moe_block_norm(ncfg, r_in, x_in, wn, None, wn, None, a, None)
        torch.cuda.synchronize()
        moe.moe_grouped_gemm(pcfg, None, a, None, w, None, b, ws)
        torch.cuda.synchronize()
        moe.moe_grouped_gemm(qcfg, None, b, None, w1, None, c, ws2)
        torch.cuda.synchronize()
        c.mul_(2.0 ** -11)
        torch.cuda.synchronize()
        moe.moe_block_norm(ncfg, r_in, c, wn, None, wn, d, e, None)
        torch.cuda.synchronize()
        return e
    want = apart(x0, r0), apart(x1, r1)
    for _ in range(20):
        for args, e in zip(((x0, r0), (x1, r1)), want):
            assert torch.equal(chain(*args), e)
    xs, rs = x0.clone(), r0.clone()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        chain(xs, rs)
    warm.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            chain(xs, rs)
    for _ in range(5):
        for args, e in zip(((x0, r0), (x1, r1)), want):
            xs.copy_(args[0])
            rs.copy_(args[1])
            graph.replay()
            assert torch.equal(out, e)
    assert moe.moe_read_device_status(ws) == 0 and moe.moe_read_device_status(ws2) == 0


@pytest.mark.parametrize("rows", [33, 64, 65, 96, 128, 129])
def test_block_scaled_product_between_its_kernels(rows):
    """Row counts on both sides of the choice of kernel, against sums in 64 bits."""
    n, k = 264, 2064
    many = product("fp8", [rows], n, k, out="f32")
    x, w = randn(1, rows, k), randn(2, 1, n, k)
    q, v = (100 * x.float()).to(torch.float8_e4m3fn), (100 * w.float()).to(torch.float8_e4m3fn)
    kb = -(-k // 128)
    s, t = randn(6, rows, kb).float(), randn(7, 1, -(-n // 128), kb).float()
    a = q.double() * s.double().repeat_interleave(128, 1)[:, :k]
    b = v[0].double() * t[0].double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    # 128 products and 8 steps per block cut at 2^-23 of the largest; kb blocks and scales round
    tol = ((128 + 8 + 16) * 2.0 ** -23 + (kb + 2) * 2.0 ** -24) * mag + 2.0 ** -24 * ref.abs()
    assert (((many.double() - ref).abs() <= tol) | (torch.isnan(many) & torch.isnan(ref))).all()


@pytest.mark.parametrize("op,rows,n,k", [("gemm", 3, 38400, 7168), ("gemm", 300, 10240, 7168), ("dgrad", 5, 7168, 38400),
                                         ("dgrad", 260, 7168, 10240), ("wgrad", 7168, 2048, 2560)])
def test_long_sums_in_fp32(op, rows, n, k):
    """fp32 outputs add up sums of 512 products (so many tiles that most are not cut).  Each step of
    the tensor cores leaves the sum so far short by up to a unit in its last place, half of one on
    average: 2^-24 of it, 32 steps in a sum of 512; those sums have random signs, and the 14 of them
    and up to 4 parts of a cut tile round once each.  So the root mean square of the errors is below
    32 + 18 times 2^-24 of the results'.  One sum of all 7168 is 448 steps long, and measured
    7.9e-6."""
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.randn(rows, n if op == "dgrad" else k, device=DEV, generator=g).to(BF)
    y = torch.randn(*((rows, n) if op == "wgrad" else (1, n, k)), device=DEV, generator=g).to(BF)
    cfg = moe.make_product_config(1, rows, n, k, out="f32")
    ws = product_ws(cfg)
    if op == "wgrad":
        out, ref = torch.empty(1, n, k, device=DEV), (y.double().T @ x.double())[None]
        moe.moe_grouped_gemm_wgrad(cfg, None, y, x, out, ws)
    elif op == "gemm":
        out, ref = torch.empty(rows, n, device=DEV), x.double() @ y[0].double().T
        moe.moe_grouped_gemm(cfg, None, x, None, y, None, out, ws)
    else:
        out, ref = torch.empty(rows, k, device=DEV), x.double() @ y[0].double()
        moe.moe_grouped_gemm_dgrad(cfg, None, x, y, out, ws)
    error, size = ((out.double() - ref).square().mean().sqrt(), ref.square().mean().sqrt())
    assert error <= 50 * 2.0 ** -24 * size, float(error / size)
