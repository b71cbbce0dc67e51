"""moe_block_norm and moe_block_norm_backward against their formulas in 64 bits.

Tolerances per element, counted in roundings.  u32 = 2^-24 is half a step of fp32.  A sum of d
terms runs as chains of at most 32 terms per thread and at most 10 tree levels, so it is off
by at most 42 u32 of its terms' magnitudes; rsqrt and the few products around it add under 22:
64 u32 in all, of the magnitudes that enter (cancellation between them is not relative to the
result).  Each output then rounds once to its type: half a step, eps / 2 of its value."""
import numpy as np
import pytest
import torch

import oracle
from sparse_expert_moe_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24


def half_step(name):
    return torch.finfo(TYPES[name]).eps / 2


def tiny(name):
    """Half the spacing of the subnormals: what a rounding is off by below the normal range."""
    return torch.finfo(TYPES[name]).smallest_normal * torch.finfo(TYPES[name]).eps / 2


def make(T, d, gate="none", res="bf16", act="bf16", weight="bf16", post=True, pre=True, branch=True,
         seed=0):
    g = torch.Generator(DEV).manual_seed(seed * 1009 + T * 31 + d)

    def rand(*shape, dt):
        return torch.randn(*shape, device=DEV, generator=g).to(TYPES[dt])

    x = dict(r=2 * rand(T, d, dt=res), y=rand(T, d, dt=act) if branch else None)
    x["w_post"] = 1 + 0.2 * rand(d, dt=weight) if post and branch else None
    x["w_pre"] = 1 + 0.2 * rand(d, dt=weight) if pre else None
    shape = {"none": None, "channel": (d,), "token": (T,), "full": (T, d)}[gate]
    x["gate"] = None if shape is None else rand(*shape, dt=act if gate == "full" else weight)
    x["dh"] = rand(T, d, dt=act) if pre else None
    x["dr_out"] = rand(T, d, dt=res)
    return x


def f64(t):
    return None if t is None else t.double()


def gate64(x, gate):
    if x["gate"] is None:
        return torch.ones((), device=DEV, dtype=torch.float64)
    return f64(x["gate"])[:, None] if gate == "token" else f64(x["gate"])


def reference(x, gate, eps, a, b, off):
    """r', h and the magnitudes that r' was added from."""
    r = f64(x["r"]) * a
    mag = r.abs()
    if x["y"] is not None:
        u = f64(x["y"])
        if x["w_post"] is not None:
            u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * (f64(x["w_post"]) + off)
        br = b * gate64(x, gate) * u
        r, mag = r + br, mag + br.abs()
    h = hm = None
    if x["w_pre"] is not None:
        i = (r.square().mean(-1, keepdim=True) + eps).rsqrt()
        w = f64(x["w_pre"]) + off
        h, hm = r * i * w, mag * i * w.abs()
    return r, mag, h, hm


def forward(x, T, d, gate, res, act, weight, out, eps=1e-6, a=1.0, b=1.0, off=0.0, keep_r=True):
    cfg = moe.make_norm_config(T, d, gate=gate, res=res, act=act, weight=weight, out=out, eps=eps,
                               res_scale=a, branch_scale=b, w_offset=off)
    r_out = torch.full((T, d), float("nan"), device=DEV, dtype=TYPES[res]) if keep_r else None
    h = hs = None
    if x["w_pre"] is not None:
        if out == "e4m3":
            h = torch.zeros(T, d, device=DEV, dtype=torch.float8_e4m3fn)
            hs = torch.zeros(T, d // 128, device=DEV)
        else:
            h = torch.full((T, d), float("nan"), device=DEV, dtype=TYPES[out])
    moe.moe_block_norm(cfg, x["r"], x["y"], x["w_post"], x["gate"], x["w_pre"], r_out, h, hs)
    return r_out, h, hs


def check(got, ref, tol, what):
    bad = (got.double() - ref).abs() > tol
    assert torch.isfinite(got.float()).all(), what
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() / tol.clamp_min(1e-300)).max()))


SHAPES = [(1, 8), (1, 7168), (3, 16384), (5, 128), (67, 264), (300, 7168), (297, 520), (299, 16384),
          (1000, 1024), (513, 2056)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_forward_shapes_and_gates(T, d, gate):
    x = make(T, d, gate)
    r_out, h, _ = forward(x, T, d, gate, "bf16", "bf16", "bf16", "bf16", a=0.9, b=0.7)
    r, mag, hr, hm = reference(x, gate, 1e-6, np.float32(0.9).item(), np.float32(0.7).item(), 0.0)
    check(r_out, r, half_step("bf16") * r.abs() + 64 * U32 * mag + tiny("bf16"), "r_out")
    check(h, hr, half_step("bf16") * hr.abs() + 128 * U32 * hm + tiny("bf16"), "h")


@pytest.mark.parametrize("res,act,weight,out", [("f32", "bf16", "bf16", "bf16"), ("bf16", "f32", "f32", "f32"),
                                                ("f32", "f32", "bf16", "f32"), ("bf16", "bf16", "f32", "f32")])
@pytest.mark.parametrize("post,pre,branch", [(True, True, True), (False, True, True), (True, False, True),
                                             (False, False, True), (False, True, False)])
def test_forward_types_and_parts(res, act, weight, out, post, pre, branch):
    T, d, gate = 130, 640, "full" if branch else "none"
    x = make(T, d, gate, res, act, weight, post, pre, branch, seed=3)
    r_out, h, _ = forward(x, T, d, gate, res, act, weight, out, off=1.0, b=0.5)
    r, mag, hr, hm = reference(x, gate, 1e-6, 1.0, 0.5, 1.0)
    check(r_out, r, half_step(res) * r.abs() + 64 * U32 * mag + tiny(res), "r_out")
    if pre:
        check(h, hr, half_step(out) * hr.abs() + 128 * U32 * hm + tiny(out), "h")
    else:
        assert h is None


@pytest.mark.parametrize("T,d", [(1, 128), (3, 7168), (600, 256), (70, 16384)])
def test_quantised_rows_follow_the_permutations_rule(T, d):
    """The e4m3 rows are the oracle's quantisation of the fp32 h that the same call stores, and
    that h is the h of the formula."""
    x = make(T, d, "none", seed=5)
    x["r"][0, :128] = 0
    x["y"][0, :128] = 0                         # an all-zero block
    _, h32, _ = forward(x, T, d, "none", "bf16", "bf16", "bf16", "f32")
    _, codes, scale = forward(x, T, d, "none", "bf16", "bf16", "bf16", "e4m3", keep_r=False)
    want, ws = oracle.quantize_e4m3_blocks(h32.double().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), ws.astype(np.float32))
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want)


def test_zero_rows_and_huge_and_masked_values():
    """A row of zeros gives zeros; infinities and NaN stay in their own row."""
    T, d = 300, 1024
    x = make(T, d, "token", seed=7)
    clean, hc, _ = forward(x, T, d, "token", "bf16", "bf16", "bf16", "bf16")
    x["r"][1] = 0
    x["y"][1] = 0
    x["r"][2, 5] = float("inf")
    x["y"][3, 6] = float("nan")
    r_out, h, _ = forward(x, T, d, "token", "bf16", "bf16", "bf16", "bf16")
    assert (r_out[1] == 0).all() and (h[1] == 0).all()
    assert torch.isnan(h[3]).all()
    keep = [i for i in range(T) if i not in (1, 2, 3)]
    assert torch.equal(r_out[keep], clean[keep]) and torch.equal(h[keep], hc[keep])


def test_in_place():
    T, d = 400, 7168
    x = make(T, d, "channel", seed=8)
    want_r, want_h, _ = forward(x, T, d, "channel", "bf16", "bf16", "bf16", "bf16")
    cfg = moe.make_norm_config(T, d, gate="channel")
    moe.moe_block_norm(cfg, x["r"], x["y"], x["w_post"], x["gate"], x["w_pre"], x["r"], x["y"], None)
    assert torch.equal(x["r"], want_r) and torch.equal(x["y"], want_h)


# ---------------------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------------------

def backward(x, rp, T, d, gate, res, act, weight, a=1.0, b=1.0, off=0.0, eps=1e-6, skip=()):
    cfg = moe.make_norm_config(T, d, gate=gate, res=res, act=act, weight=weight, eps=eps, res_scale=a,
                               branch_scale=b, w_offset=off)
    ws = torch.full((moe.moe_norm_workspace_size(cfg),), 0xAB, dtype=torch.uint8, device=DEV)
    nan = dict(device=DEV)
    out = dict(dr=torch.full((T, d), float("nan"), dtype=TYPES[res], **nan), dy=None, dgate=None, dw_post=None,
               dw_pre=None)
    if x["y"] is not None:
        out["dy"] = torch.full((T, d), float("nan"), dtype=TYPES[act], **nan)
    if x["w_post"] is not None:
        out["dw_post"] = torch.full((d,), float("nan"), **nan)
    if x["w_pre"] is not None:
        out["dw_pre"] = torch.full((d,), float("nan"), **nan)
    if x["gate"] is not None:
        out["dgate"] = torch.full_like(x["gate"], float("nan"), dtype=TYPES[act] if gate == "full" else torch.float32)
    for k in skip:
        out[k] = None
    moe.moe_block_norm_backward(cfg, rp, x["y"], x["w_post"], x["gate"], x["w_pre"], x["dh"], x["dr_out"],
                                out["dr"], out["dy"], out["dgate"], out["dw_post"], out["dw_pre"], ws)
    return out


def pullback64(x, w, off, dout, tol_out, eps):
    """dx, dw terms of norm(x; w) for the gradient dout known to +- tol_out, with tolerances."""
    i = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    wv = w + off
    v = dout * wv
    m, ma = (v * x).mean(-1, keepdim=True), (v * x).abs().mean(-1, keepdim=True)
    dx = i * v - x * i ** 3 * m
    tol = 64 * U32 * (i * v.abs() + x.abs() * i ** 3 * ma)
    tol = tol + i * wv.abs() * tol_out + x.abs() * i ** 3 * (tol_out * wv.abs() * x.abs()).mean(-1, keepdim=True)
    return dx, tol, dout * x * i, (64 * U32 * dout.abs() + tol_out) * (x * i).abs(), x * i * wv


@pytest.mark.parametrize("T,d,gate,res,act,weight,post,pre,branch", [
    (1, 8, "channel", "bf16", "bf16", "bf16", True, True, True),
    (1, 7168, "token", "bf16", "bf16", "bf16", True, True, True),
    (2, 16384, "channel", "f32", "bf16", "f32", True, True, True),
    (149, 264, "full", "bf16", "bf16", "bf16", True, True, True),
    (1203, 520, "channel", "bf16", "f32", "f32", True, True, True),
    (301, 7168, "channel", "bf16", "bf16", "bf16", True, True, True),
    (150, 16384, "token", "bf16", "bf16", "bf16", True, True, True),
    (333, 4104, "full", "f32", "f32", "f32", False, True, True),
    (700, 128, "token", "bf16", "bf16", "bf16", True, False, True),
    (77, 1024, "none", "bf16", "bf16", "bf16", True, True, True),
    (640, 2048, "none", "bf16", "bf16", "bf16", False, True, False),
    (64, 9000, "channel", "bf16", "bf16", "bf16", False, False, True),
])
def test_backward_against_the_formula(T, d, gate, res, act, weight, post, pre, branch):
    a, b, off = np.float32(0.8).item(), np.float32(0.6).item(), 1.0
    x = make(T, d, gate, res, act, weight, post, pre, branch, seed=11)
    rp = x["r"]
    got = backward(x, rp, T, d, gate, res, act, weight, a, b, off)
    eps = 1e-6
    eps = np.float32(eps).item()
    G, tG = f64(x["dr_out"]), torch.zeros(T, d, device=DEV, dtype=torch.float64)
    if pre:
        dx, tG, dwp, tdwp, _ = pullback64(f64(rp), f64(x["w_pre"]), off, f64(x["dh"]), tG, eps)
        G = G + dx
        tG = tG + 4 * U32 * (G.abs() + dx.abs())
    check(got["dr"], a * G, half_step(res) * (a * G).abs() + a * tG + 2 * U32 * G.abs() + tiny(res), "dr")
    colsum = (T + 64) * U32                     # a column's chain over tokens, and the join
    if pre:
        check(got["dw_pre"], dwp.sum(0), tdwp.sum(0) + colsum * dwp.abs().sum(0), "dw_pre")
    if not branch:
        return
    g = gate64(x, gate)
    du, tdu = b * g * G, (b * g).abs() * (tG + 4 * U32 * G.abs())
    u = f64(x["y"])
    if post:
        dy, tdy, dwq, tdwq, u = pullback64(f64(x["y"]), f64(x["w_post"]), off, du, tdu, eps)
        check(got["dw_post"], dwq.sum(0), tdwq.sum(0) + colsum * dwq.abs().sum(0), "dw_post")
    else:
        dy, tdy = du, tdu
    check(got["dy"], dy, half_step(act) * dy.abs() + tdy + tiny(act), "dy")
    dg, tdg = b * G * u, b * u.abs() * (tG + 64 * U32 * G.abs())
    if gate == "channel":
        check(got["dgate"], dg.sum(0), tdg.sum(0) + colsum * dg.abs().sum(0), "dgate")
    elif gate == "token":
        check(got["dgate"], dg.sum(1), tdg.sum(1) + 42 * U32 * dg.abs().sum(1), "dgate")
    elif gate == "full":
        check(got["dgate"], dg, half_step(act) * dg.abs() + tdg + tiny(act), "dgate")


def test_backward_against_differences():
    """The gradients of sum(h dh) + sum(r' dr_out) by central differences of the formula in
    64 bits, along random directions of every input."""
    T, d, gate = 6, 64, "channel"
    x = make(T, d, gate, "f32", "f32", "f32", seed=13)
    eps, a, b = np.float32(1e-6).item(), 1.0, 0.5
    rp, _, _, _ = reference(x, gate, eps, a, b, 0.0)
    got = backward(x, rp.float(), T, d, gate, "f32", "f32", "f32", a, b)
    g = torch.Generator(DEV).manual_seed(1)
    for name, grad in (("r", "dr"), ("y", "dy"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("gate", "dgate")):
        v = torch.randn(x[name].shape, device=DEV, generator=g, dtype=torch.float64)

        def value(s):
            z = {k: f64(t) for k, t in x.items()}
            z[name] = z[name] + s * v
            r, _, h, _ = reference(z, gate, eps, a, b, 0.0)
            return float((h * z["dh"]).sum() + (r * z["dr_out"]).sum())
        step = 1e-5
        want = (value(step) - value(-step)) / (2 * step)
        have = float((got[grad].double() * v).sum())
        scale = float((got[grad].double() * v).abs().sum())
        # fp32 gradients (128 roundings of their terms), r' rounded to fp32, and the difference's
        # own error: step^2 of a third derivative of order one, 1e-16 / step of the values
        assert abs(have - want) < 1e-5 * max(1.0, scale), name


def test_backward_is_repeatable_and_parts_can_be_left_out():
    T, d, gate = 1000, 7168, "channel"
    x = make(T, d, gate, seed=17)
    one = backward(x, x["r"], T, d, gate, "bf16", "bf16", "bf16")
    two = backward(x, x["r"], T, d, gate, "bf16", "bf16", "bf16")
    less = backward(x, x["r"], T, d, gate, "bf16", "bf16", "bf16", skip=("dw_pre", "dgate"))
    for k in one:
        assert torch.equal(one[k], two[k]), k
        if less[k] is not None:
            assert torch.equal(one[k], less[k]), k


def test_backward_of_no_tokens_is_zero():
    cfg = moe.make_norm_config(0, 256, gate="channel")
    ws = torch.empty(moe.moe_norm_workspace_size(cfg), dtype=torch.uint8, device=DEV)
    e = torch.empty(0, 256, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(256, device=DEV, dtype=torch.bfloat16)
    dg, dp, dq = (torch.full((256,), float("nan"), device=DEV) for _ in range(3))
    moe.moe_block_norm_backward(cfg, e, e, w, w, w, e, e, e, e, dg, dp, dq, ws)
    assert (dg == 0).all() and (dp == 0).all() and (dq == 0).all()
    moe.moe_block_norm(cfg, e, e, w, w, w, e, e, None)
