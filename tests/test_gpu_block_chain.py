"""The block norms and the grouped products as they are used together: a training step of one
expert block against 64-bit autograd, and the quantised rows of a norm as the input of the 8-bit
product and of the whole layer.  Also what one call may do to another: shared and separate
workspaces, several streams, tensors past 2^31 elements."""
import numpy as np
import pytest
import torch

import oracle
from sparse_expert_moe_b200 import inputs, moe

from helpers import dequant_fast, max_rel_err, oracle_layer, topk_gaps

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
# half a step of bf16, relative: what one rounding of a tensor can move it by, in the 2-norm too
STEP = torch.finfo(BF).eps / 2


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def ws_of(cfg):
    return torch.zeros(moe.moe_product_workspace_size(cfg), dtype=torch.uint8, device=DEV)


def test_training_step_of_an_expert_block():
    """r1, h = norm(r, y0); the experts' two products on h with SwiGLU between them, combined;
    r2, h2 = norm(r1, y): every gradient of sum(h2 * g) against autograd in 64 bits."""
    T, d, E, k, I = 200, 256, 8, 2, 128
    gen = torch.Generator(DEV).manual_seed(0)

    def rand(*s, scale=1.0, dt=BF):
        return (torch.randn(*s, device=DEV, generator=gen) * scale).to(dt)

    r, y0, g = rand(T, d, scale=2.0), rand(T, d), rand(T, d)
    wp0, wq0, wp1, wq1 = (1 + rand(d, scale=0.2) for _ in range(4))
    gate0, gate1 = 1 + rand(d, scale=0.2), torch.sigmoid(rand(T))
    w13, w2 = rand(E, 2 * I, d, scale=0.06), rand(E, d, I, scale=0.09)
    logits = rand(T, E, dt=torch.float32)
    R = T * k

    # ------------------------------------------------------------------ forward
    n0 = moe.make_norm_config(T, d, gate="channel", branch_scale=0.7)
    n1 = moe.make_norm_config(T, d, gate="token", branch_scale=0.9)
    r1, h, r2, h2 = (torch.empty(T, d, device=DEV, dtype=BF) for _ in range(4))
    moe.moe_block_norm(n0, r, y0, wp0, gate0, wq0, r1, h, None)
    cfg = moe.make_config(T, d, E, k, I, score="softmax")
    lws = torch.zeros(moe.moe_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    gates = torch.empty(T, k, device=DEV)
    moe.moe_route(cfg, logits, None, idx, gates)
    xp = torch.empty(R, d, device=DEV, dtype=BF)
    tok, inv = torch.empty(R, dtype=torch.int32, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    moe.moe_permute(cfg, idx, h, None, xp, None, tok, inv, off, lws)
    p1, p2 = moe.make_product_config(E, R, 2 * I, d), moe.make_product_config(E, R, d, I)
    p1w, p2w = moe.make_product_config(E, R, 2 * I, d, out="f32"), moe.make_product_config(E, R, d, I, out="f32")
    ws = ws_of(p1)
    z = torch.empty(R, 2 * I, device=DEV, dtype=BF)
    moe.moe_grouped_gemm(p1, off, xp, None, w13, None, z, ws)
    zg, zu = z[:, :I].float(), z[:, I:].float()
    a = (torch.nn.functional.silu(zg) * zu).to(BF)
    yp = torch.empty(R, d, device=DEV, dtype=BF)
    moe.moe_grouped_gemm(p2, off, a, None, w2, None, yp, ws)
    y = torch.empty(T, d, device=DEV, dtype=BF)
    moe.moe_combine(cfg, yp, inv, gates, None, y)
    moe.moe_block_norm(n1, r1, y, wp1, gate1, wq1, r2, h2, None)

    # ------------------------------------------------------------------ backward
    f32 = dict(device=DEV, dtype=torch.float32)
    nws = torch.empty(moe.moe_norm_workspace_size(n0), dtype=torch.uint8, device=DEV)
    dr1, dy = torch.empty_like(r1), torch.empty_like(y)
    dg1, dwp1, dwq1 = torch.empty(T, **f32), torch.empty(d, **f32), torch.empty(d, **f32)
    moe.moe_block_norm_backward(n1, r2, y, wp1, gate1, wq1, g, None, dr1, dy, dg1, dwp1, dwq1, nws)
    dyp = (gates.reshape(-1)[_slot_of_row(inv)][:, None] * dy[tok.long()].float()).to(BF)
    da, dw2 = torch.empty(R, I, device=DEV, dtype=BF), torch.empty(E, d, I, **f32)
    moe.moe_grouped_gemm_dgrad(p2, off, dyp, w2, da, ws)
    moe.moe_grouped_gemm_wgrad(p2w, off, dyp, a, dw2, ws)
    s = torch.sigmoid(zg)
    dz = torch.cat([da.float() * zu * s * (1 + zg * (1 - s)), da.float() * zg * s], 1).to(BF)
    dxp, dw13 = torch.empty(R, d, device=DEV, dtype=BF), torch.empty(E, 2 * I, d, **f32)
    moe.moe_grouped_gemm_dgrad(p1, off, dz, w13, dxp, ws)
    moe.moe_grouped_gemm_wgrad(p1w, off, dz, xp, dw13, ws)
    dh = torch.empty_like(h)
    moe.moe_combine(cfg, dxp, inv, torch.ones_like(gates), None, dh)
    dr, dy0 = torch.empty_like(r), torch.empty_like(y0)
    dg0, dwp0, dwq0 = (torch.empty(d, **f32) for _ in range(3))
    moe.moe_block_norm_backward(n0, r1, y0, wp0, gate0, wq0, dh, dr1, dr, dy0, dg0, dwp0, dwq0, nws)
    assert moe.moe_read_device_status(ws) == 0 and moe.moe_read_device_status(lws) == 0

    # ------------------------------------------------------------------ 64 bits
    L = {n: t.double().requires_grad_(True) for n, t in dict(
        r=r, y0=y0, wp0=wp0, wq0=wq0, gate0=gate0, w13=w13, w2=w2, wp1=wp1, wq1=wq1, gate1=gate1).items()}

    def norm(x, w):
        return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    R1 = L["r"] + 0.7 * L["gate0"] * norm(L["y0"], L["wp0"])
    H = norm(R1, L["wq0"])
    Y = torch.zeros(T, d, device=DEV, dtype=torch.float64)
    ig, gg = idx.long(), gates.double()
    for e in range(E):
        t, j = (ig == e).nonzero(as_tuple=True)
        Z = H[t] @ L["w13"][e].T
        O = (torch.nn.functional.silu(Z[:, :I]) * Z[:, I:]) @ L["w2"][e].T
        Y = Y.index_add(0, t, gg[t, j][:, None] * O)
    R2 = R1 + 0.9 * L["gate1"][:, None] * norm(Y, L["wp1"])
    (norm(R2, L["wq1"]) * g.double()).sum().backward()
    # bf16 roundings on the longest way to a gradient: r1, h, z, a, yp, y, r2 forward; dr1, dy, dyp,
    # da, dz, dxp, dh, dr backward
    bar = 15 * STEP
    got = dict(r=dr, y0=dy0, wp0=dwp0, wq0=dwq0, gate0=dg0, w13=dw13, w2=dw2, wp1=dwp1, wq1=dwq1, gate1=dg1)
    for n, t in got.items():
        assert rel(t, L[n].grad) < bar, (n, rel(t, L[n].grad))


def _slot_of_row(inv):
    """(token, slot) pair of each permuted row, as an index into the flattened pairs."""
    flat = inv.reshape(-1).long()
    out = torch.empty_like(flat)
    out[flat] = torch.arange(flat.numel(), device=flat.device)
    return out


def test_quantising_norm_feeds_the_block_scaled_product():
    """norm -> e4m3 rows and scales -> dense 8-bit product, against the product of the rows' values."""
    T, d, n = 75, 512, 384
    gen = torch.Generator(DEV).manual_seed(1)
    r, y = (torch.randn(T, d, device=DEV, generator=gen).to(BF) for _ in range(2))
    w_pre = torch.ones(d, device=DEV, dtype=BF)
    cfg = moe.make_norm_config(T, d, out="e4m3")
    r1, codes, scale = torch.empty_like(r), torch.empty(T, d, device=DEV, dtype=torch.float8_e4m3fn), torch.empty(T, d // 128, device=DEV)
    moe.moe_block_norm(cfg, r, y, None, None, w_pre, r1, codes, scale)
    w = torch.randn(1, n, d, device=DEV, generator=gen).mul_(100).to(torch.float8_e4m3fn)
    sw = torch.rand(1, n // 128, d // 128, device=DEV, generator=gen) * 1e-3
    out = torch.empty(T, n, device=DEV, dtype=BF)
    p = moe.make_product_config(1, T, n, d, dtype="e4m3_fs")
    moe.moe_grouped_gemm(p, None, codes, scale, w, sw, out, ws_of(p))
    x = codes.double() * scale.double().repeat_interleave(128, 1)
    v = w[0].double() * sw[0].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ref, mag = x @ v.T, x.abs() @ v.abs().T
    # two of the weights' draws pass 448 and become NaN codes: their columns are NaN, no others
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(out), nan) and nan.any(0).sum() == 2
    assert (((out.double() - ref).abs() <= STEP * ref.abs() + 200 * 2.0 ** -23 * mag) | nan).all()


def test_quantising_norm_feeds_the_layer():
    """The same rows as e4m3 activations of moe_layer_forward: accepted without a device fault, and
    the layer's output is the oracle's for those rows (tokens whose routing is decided by 1e-3)."""
    spec = inputs.custom_spec(T=96, d_model=256, E=8, top_k=2, d_ff=256, n_shared=1, act="e4m3", weight="e4m3")
    wl = inputs.make_workload(spec, 2, redraw=[], threads=4)
    gen = torch.Generator(DEV).manual_seed(2)
    r = torch.randn(96, 256, device=DEV, generator=gen).to(BF)
    cfg = moe.make_norm_config(96, 256, out="e4m3")
    codes, scale = torch.empty(96, 256, device=DEV, dtype=torch.float8_e4m3fn), torch.empty(96, 2, device=DEV)
    moe.moe_block_norm(cfg, r, None, None, None, torch.ones(256, device=DEV, dtype=BF), None, codes, scale)
    layer = moe.DeviceLayer.from_workload(wl, DEV)
    out = layer.forward(codes, scale)
    assert moe.moe_read_device_status(layer.ws) == 0
    wl.x, wl.x_scale = codes.cpu(), scale.cpu()
    x = dequant_fast(wl.x.view(torch.uint8).numpy(), wl.x_scale.numpy(), 1, 128)
    bias = None if wl.sel_bias is None else wl.sel_bias.double().numpy()
    keys = oracle.selection_keys(oracle.router_logits(x, wl.wr.double().numpy()), spec.score, bias)
    sure = topk_gaps(keys, spec.top_k) >= 1e-3
    assert sure.sum() > 60
    ref = oracle_layer(wl)
    assert max_rel_err(out.float().cpu().numpy()[sure], ref[sure]) < 6e-2


# ---------------------------------------------------------------------------------------
# calls next to one another
# ---------------------------------------------------------------------------------------

def _product_case(seed, sizes, n, k, dtype="bf16"):
    gen = torch.Generator(DEV).manual_seed(seed)
    G, R = len(sizes), sum(sizes)
    cfg = moe.make_product_config(G, R, n, k, dtype=dtype, out="f32")
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    x, w = torch.randn(R, k, device=DEV, generator=gen), torch.randn(G, n, k, device=DEV, generator=gen)
    sa = sw = None
    if dtype != "bf16":
        sa, sw = torch.rand(R, -(-k // 128), device=DEV), torch.rand(G, -(-n // 128), -(-k // 128), device=DEV)
    vt = BF if dtype == "bf16" else torch.float8_e4m3fn
    y = torch.zeros(R, n, device=DEV)
    return dict(cfg=cfg, off=off, x=x.to(vt), w=w.to(vt), sa=sa, sw=sw, y=y)


def _run(c, ws):
    moe.moe_grouped_gemm(c["cfg"], c["off"], c["x"], c["sa"], c["w"], c["sw"], c["y"], ws)


CASES = [([3], 512, 4096, "bf16"), ([200], 512, 4096, "bf16"), ([1], 512, 4096, "e4m3_fs"), ([150], 256, 7168, "e4m3_fs")]


def test_one_workspace_in_turn_and_two_graphs_that_share_it():
    """Calls of every kernel in turn on one workspace, eagerly and from two captured graphs that
    are replayed alternately, give what a workspace of their own gives."""
    cases = [_product_case(i, *c) for i, c in enumerate(CASES)]
    ws = ws_of(cases[0]["cfg"])
    want = []
    for c in cases:
        _run(c, ws_of(c["cfg"]))
        want.append(c["y"].clone())
        c["y"].zero_()
    for c in cases + cases[::-1]:
        _run(c, ws)
    for c, w in zip(cases, want):
        assert torch.equal(c["y"], w)
    graphs = []
    for part in (cases[:2], cases[2:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for c in part:
                _run(c, ws)
        graphs.append(g)
    for c in cases:
        c["y"].zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c["y"], w)
    assert (ws[:256] == 0).all()


def test_two_streams_with_workspaces_of_their_own():
    cases = [_product_case(10 + i, *c) for i, c in enumerate(CASES)]
    want = []
    for c in cases:
        _run(c, ws_of(c["cfg"]))
        want.append(c["y"].clone())
        c["y"].zero_()
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [ws_of(c["cfg"]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, ws in zip(cases, streams, spaces):
            moe.moe_grouped_gemm(c["cfg"], c["off"], c["x"], c["sa"], c["w"], c["sw"], c["y"], ws, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c["y"], w)


def test_workspace_of_a_layer_serves_the_products():
    """A zeroed workspace that the layer used before: same header, same results."""
    cfg = moe.make_config(64, 256, 8, 2, 256)
    c = _product_case(20, [200], 512, 4096)
    size = max(moe.moe_workspace_size(cfg), moe.moe_product_workspace_size(c["cfg"]))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    wl = inputs.make_workload(inputs.custom_spec(T=64, d_model=256, E=8, top_k=2, d_ff=256), 1, redraw=[], threads=2)
    layer = moe.DeviceLayer.from_workload(wl, DEV)
    layer.ws = ws
    a = layer.forward(wl.x.to(DEV))
    _run(c, ws)
    got = c["y"].clone()
    b = layer.forward(wl.x.to(DEV))
    _run(c, ws_of(c["cfg"]))
    assert torch.equal(got, c["y"]) and torch.equal(a, b)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.slow
def test_tensors_past_two_to_the_31_elements():
    """Rows, weights and outputs whose element offsets pass 32 bits."""
    T, d = 300_001, 7168
    r = torch.zeros(T, d, device=DEV, dtype=BF)
    y = torch.zeros(T, d, device=DEV, dtype=BF)
    r[-3:] = torch.randn(3, d, device=DEV).to(BF)
    y[-3:] = torch.randn(3, d, device=DEV).to(BF)
    w = torch.ones(d, device=DEV, dtype=BF)
    big, small = moe.make_norm_config(T, d), moe.make_norm_config(3, d)
    h, hs, rs = torch.empty_like(r), torch.empty(3, d, device=DEV, dtype=BF), torch.empty(3, d, device=DEV, dtype=BF)
    tail_r, tail_y = r[-3:].clone(), y[-3:].clone()
    moe.moe_block_norm(big, r, y, w, None, w, r, h, None)
    moe.moe_block_norm(small, tail_r, tail_y, w, None, w, rs, hs, None)
    # the two launches add a row's squares in different orders: within two roundings of each other
    assert ((h[-3:].float() - hs.float()).abs() <= 2 * STEP * hs.float().abs() + 1e-6).all()
    assert (h[:-3] == 0).all()
    del r, y, h
    torch.cuda.empty_cache()
    G, n, k = 80, 7168, 4096                                # 2.3e9 weights
    w = torch.zeros(G, n, k, device=DEV, dtype=BF)
    w[-1] = torch.randn(n, k, device=DEV).to(BF)
    sizes = [1] * (G - 1) + [5]
    R = sum(sizes)
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    x = torch.randn(R, k, device=DEV).to(BF)
    cfg = moe.make_product_config(G, R, n, k, out="f32")
    out = torch.empty(R, n, device=DEV)
    ws = ws_of(cfg)
    moe.moe_grouped_gemm(cfg, off, x, None, w, None, out, ws)
    ref = x[-5:].double() @ w[-1].double().T
    assert rel(out[-5:], ref) < 1e-4 and (out[:-5] == 0).all()
    del w
    torch.cuda.empty_cache()
    dw = torch.full((G, n, k), float("nan"), device=DEV, dtype=BF)
    cfg = moe.make_product_config(G, R, n, k)
    dy = torch.randn(R, n, device=DEV).to(BF)
    moe.moe_grouped_gemm_wgrad(cfg, off, dy, x, dw, ws)
    for g in (0, G - 2, G - 1):
        lo, hi = int(off[g]), int(off[g + 1])
        assert rel(dw[g], dy[lo:hi].double().T @ x[lo:hi].double()) < 2 * STEP
    assert moe.moe_read_device_status(ws) == 0
