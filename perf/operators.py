"""Timing cases of the operators that stand around the expert layer: the norms before and after
a block with its gate and residual scale (and their gradients), the experts' products one at a
time over ragged groups (forward and both gradients), and the 8-bit product with a scale for
each block of 128.

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true: the calls
a program makes of the library.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GATES = ("none", "channel", "token", "full")
EPS = 1e-6
RES_SCALE, BRANCH_SCALE, W_OFFSET = 1.0, 0.7, 0.0


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _norm(name, T, d, **kw):
    c = dict(name=name, op="norm", T=T, d=d, post=True, pre=True, gate="none", res="bf16", out="bf16")
    c.update(kw)
    return c


def _prod(name, op, G, rows, n, k, dtype="bf16", out="bf16", spare=0):
    return dict(name=name, op=op, G=G, rows=rows, n=n, k=k, dtype=dtype, out=out, spare=spare)


def listed():
    return [
        # one decoded token through a sandwich norm: pure latency
        _norm("norm_token", 1, 7168, gate="channel"),
        # a decode batch: residual add, pre-norm, rows quantised for 8-bit experts
        _norm("norm_quant_decode", 128, 7168, post=False, out="e4m3"),
        # a prefill batch: post-norm, per-token gate, residual add and the next pre-norm
        _norm("norm_prefill", 8192, 7168, gate="token"),
        # the training backward of the same block, every gradient, an odd number of tokens
        _norm("norm_backward", 4095, 7168, op="norm_bwd", gate="channel"),
        # one token's eight experts, the gate/up product: streams eight weight matrices
        _prod("gemm_token", "gemm", 64, 8, 4096, 7168),
        # a decode batch's down product: every expert holds a few rows
        _prod("gemm_decode", "gemm", 64, 1024, 7168, 2048, spare=5),
        # a prefill batch's gate/up product: ragged groups of some hundred rows
        _prod("gemm_prefill", "gemm", 32, 16384, 4096, 7168),
        # the gradient of the down product's input
        _prod("dgrad_prefill", "dgrad", 32, 8191, 7168, 2048, spare=3),
        # the gradient of the down product's weights, kept in 32 bits
        _prod("wgrad_prefill", "wgrad", 32, 8191, 7168, 2048, out="f32"),
        # one token through a dense 8-bit product: pure latency and weight streaming
        _prod("fp8_token", "gemm", 1, 1, 7168, 2048, dtype="e4m3"),
        # a decode batch over 8-bit experts
        _prod("fp8_decode", "gemm", 64, 1024, 4096, 7168, dtype="e4m3"),
        # a prefill batch through a dense 8-bit product
        _prod("fp8_prefill", "gemm", 1, 8192, 4096, 7168, dtype="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gemm", "dgrad", "wgrad", "fp8", "fp8"])
    if op in ("norm", "norm_bwd"):
        quant = op == "norm" and rng.random() < 0.3
        d = 128 * rng.randint(2, 64) if quant else 8 * _log_int(rng, 16, 1024)
        T = min(_log_int(rng, 1, 8192), max(1, 8192 * 7168 // d) if not quant else 1024)
        post = rng.random() < 0.6
        return dict(op=op, T=T, d=d, post=post, pre=quant or rng.random() < 0.8, gate=rng.choice(GATES),
                    res=rng.choice(["bf16", "bf16", "f32"]),
                    out="e4m3" if quant else ("bf16" if op == "norm_bwd" else rng.choice(["bf16", "bf16", "f32"])))
    n, k = 8 * _log_int(rng, 16, 896), 8 * _log_int(rng, 16, 896)
    if op == "fp8":
        G = rng.choice([1, 1, _log_int(rng, 2, 64)])
        k = 16 * _log_int(rng, 8, 448)
        rows = _log_int(rng, 1, 8192)
        return dict(op="gemm", G=G, rows=rows, n=n, k=k, dtype="e4m3", out=rng.choice(["bf16", "f32"]),
                    spare=rng.choice([0, 7]))
    G = _log_int(rng, 1, 64)
    out = rng.choice(["bf16", "f32"])
    rows = _log_int(rng, 1, 8192 if out == "bf16" else 4096)
    return dict(op=op, G=G, rows=rows, n=n, k=k, dtype="bf16", out=out, spare=rng.choice([0, 7]))


def group_sizes(case):
    """Rows of each expert: lognormal popularity, about one expert in eight without any."""
    G, rows = case["G"], case["rows"]
    if G == 1:
        return [rows]
    g = torch.Generator().manual_seed(1000003 * G + rows)
    p = torch.exp(0.5 * torch.randn(G, generator=g))
    p[torch.rand(G, generator=g) < 0.125] = 0.0
    if not bool((p > 0).any()):
        p[0] = 1.0
    if rows <= G:                       # a token's experts are different ones
        at = torch.multinomial(p + 1e-3, rows, replacement=False, generator=g)
    else:
        at = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(at, minlength=G).tolist()


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, device=DEV, generator=gen) * scale).to(dtype)


def _codes(gen, *shape):
    """e4m3 codes as amax-scaled blocks hold them: about four standard deviations below 448."""
    out = torch.empty(shape, device=DEV, dtype=torch.float8_e4m3fn)
    for part in (out if len(shape) == 3 else [out]):
        part.copy_((torch.randn(part.shape, device=DEV, generator=gen) * 110).clamp_(-448, 448))
    return out


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    if case["op"] in ("norm", "norm_bwd"):
        s = _prepare_norm(case, gen)
    else:
        s = _prepare_product(case, gen)
    s["case"] = case
    if own:
        _plan(s)
    return s


def _prepare_norm(case, gen):
    T, d = case["T"], case["d"]
    res = DT[case["res"]]
    s = {"r": _randn(gen, T, d, scale=2.0, dtype=res), "y": _randn(gen, T, d, scale=0.5)}
    s["w_post"] = (1 + _randn(gen, d, scale=0.1)) if case["post"] else None
    s["w_pre"] = (1 + _randn(gen, d, scale=0.1)) if case["pre"] else None
    s["gate"] = {"none": None,
                 "channel": lambda: 1 + _randn(gen, d, scale=0.2),
                 "token": lambda: torch.sigmoid(_randn(gen, T)),
                 "full": lambda: torch.sigmoid(_randn(gen, T, d))}[case["gate"]]
    s["gate"] = s["gate"] and s["gate"]()
    if case["op"] == "norm_bwd":
        s["dh"] = _randn(gen, T, d, scale=0.01) if case["pre"] else None
        s["dr_out"] = _randn(gen, T, d, scale=0.01, dtype=res)
        s["dr"], s["dy"] = torch.empty_like(s["r"]), torch.empty_like(s["y"])
        f32 = dict(device=DEV, dtype=torch.float32)
        s["dw_post"] = torch.empty(d, **f32) if case["post"] else None
        s["dw_pre"] = torch.empty(d, **f32) if case["pre"] else None
        s["dgate"] = {"none": None, "channel": (d,), "token": (T,), "full": (T, d)}[case["gate"]]
        if s["dgate"]:
            s["dgate"] = torch.empty(s["dgate"], device=DEV,
                                     dtype=torch.bfloat16 if case["gate"] == "full" else torch.float32)
        return s
    s["r_out"] = torch.empty_like(s["r"])
    s["h"], s["h_scale"] = None, None
    if case["pre"] and case["out"] == "e4m3":
        s["h"] = torch.empty(T, d, device=DEV, dtype=torch.float8_e4m3fn)
        s["h_scale"] = torch.empty(T, d // 128, device=DEV, dtype=torch.float32)
    elif case["pre"]:
        s["h"] = torch.empty(T, d, device=DEV, dtype=DT[case["out"]])
    return s


def _prepare_product(case, gen):
    G, n, k = case["G"], case["n"], case["k"]
    sizes = group_sizes(case)
    total = case["rows"] + case["spare"]        # buffers are longer than what the groups hold
    off = [0]
    for v in sizes:
        off.append(off[-1] + v)
    s = {"sizes": sizes, "most": max(sizes), "rows": total,
         "off": torch.tensor(off, dtype=torch.int32, device=DEV)}
    out = DT[case["out"]]
    if case["dtype"] == "e4m3":
        kb, nb = -(-k // 128), -(-n // 128)
        s["a"], s["w"] = _codes(gen, total, k), _codes(gen, G, n, k)
        s["a_scale"] = torch.rand(total, kb, device=DEV, generator=gen).mul_(0.015).add_(0.005)
        s["w_scale"] = torch.rand(G, nb, kb, device=DEV, generator=gen).mul_(2e-4).add_(1e-4)
    else:
        s["a_scale"] = s["w_scale"] = None
        if case["op"] != "dgrad":
            s["a"] = _randn(gen, total, k)
        if case["op"] != "gemm":
            s["dy"] = _randn(gen, total, n, scale=0.01)
        if case["op"] != "wgrad":
            s["w"] = torch.empty(G, n, k, device=DEV, dtype=torch.bfloat16)
            for part in s["w"]:
                part.copy_(_randn(gen, n, k, scale=0.02))
    shape = {"gemm": (total, n), "dgrad": (total, k), "wgrad": (G, n, k)}[case["op"]]
    s["out"] = torch.zeros(shape, device=DEV, dtype=out)
    return s


def _plan(s):
    """What a program keeps between calls: the sizes and a zeroed workspace."""
    from sparse_expert_moe_b200 import moe
    c = s["case"]
    if c["op"] in ("norm", "norm_bwd"):
        s["cfg"] = moe.make_norm_config(c["T"], c["d"], gate=c["gate"], res=c["res"], act="bf16", weight="bf16",
                                        out=c["out"], eps=EPS, res_scale=RES_SCALE,
                                        branch_scale=BRANCH_SCALE, w_offset=W_OFFSET)
        size = moe.moe_norm_workspace_size(s["cfg"])
    else:
        s["cfg"] = moe.make_product_config(c["G"], s["rows"], c["n"], c["k"],
                                           dtype="e4m3_fs" if c["dtype"] == "e4m3" else "bf16", out=c["out"])
        size = moe.moe_product_workspace_size(s["cfg"])
    s["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    s["moe"] = moe


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_backward(s)
    return _plain_product(s, op)


def _own(s, op):
    m = s["moe"]
    if op == "norm":
        m.moe_block_norm(s["cfg"], s["r"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["r_out"], s["h"],
                         s["h_scale"])
        return {"r_out": s["r_out"], "h": s["h"], "h_scale": s["h_scale"]}
    if op == "norm_bwd":
        m.moe_block_norm_backward(s["cfg"], s["r"], s["y"], s["w_post"], s["gate"], s["w_pre"], s["dh"],
                                  s["dr_out"], s["dr"], s["dy"], s["dgate"], s["dw_post"], s["dw_pre"], s["ws"])
        return {k: s[k] for k in ("dr", "dy", "dgate", "dw_post", "dw_pre")}
    if op == "gemm":
        m.moe_grouped_gemm(s["cfg"], s["off"], s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"], s["ws"])
    elif op == "dgrad":
        m.moe_grouped_gemm_dgrad(s["cfg"], s["off"], s["dy"], s["w"], s["out"], s["ws"])
    else:
        m.moe_grouped_gemm_wgrad(s["cfg"], s["off"], s["dy"], s["a"], s["out"], s["ws"])
    return s["out"]


def _gate_column(s):
    g = s["gate"]
    if g is None:
        return 1.0
    return g.float()[:, None] if s["case"]["gate"] == "token" else g.float()


def _plain_norm(s):
    """r' = a r + b gate * norm(y; w_post),  h = norm(r'; w_pre) (rounded, or e4m3 blocks of 128)."""
    r, u = s["r"].float(), s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * (s["w_post"].float() + W_OFFSET)
    r = RES_SCALE * r + BRANCH_SCALE * _gate_column(s) * u
    out = {"r_out": r.to(s["r"].dtype), "h": None, "h_scale": None}
    if s["w_pre"] is None:
        return out
    h = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * (s["w_pre"].float() + W_OFFSET)
    if s["h_scale"] is None:
        out["h"] = h.to(s["h"].dtype)
        return out
    # the smallest power of two that brings a block's largest value to 448 = 0.875 * 2^9 or below
    b = h.view(h.shape[0], -1, 128)
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m == 0, torch.zeros_like(e), torch.where(m <= 0.875, e - 9, e - 8)).clamp(-127, 127)
    scale = torch.exp2(e.double()).float()
    out["h"] = (b / scale[..., None]).to(torch.float8_e4m3fn).view(h.shape)
    out["h_scale"] = scale
    return out


def _norm_pullback(x, w, dout):
    """Gradients of x * rsqrt(mean(x^2) + eps) * w, per element of x and summed into w."""
    i = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    v = dout * (w.float() + W_OFFSET)
    dx = i * v - x * (i ** 3 * (v * x).mean(-1, keepdim=True))
    return dx, (dout * x * i).sum(0), x * i * (w.float() + W_OFFSET)


def _plain_norm_backward(s):
    """Gradients through the block's r' (given as r) and its branch y."""
    rp, y, G = s["r"].float(), s["y"].float(), s["dr_out"].float()
    out = {"dgate": None, "dw_post": None, "dw_pre": None}
    if s["w_pre"] is not None:
        dx, out["dw_pre"], _ = _norm_pullback(rp, s["w_pre"], s["dh"].float())
        G = G + dx
    out["dr"] = (RES_SCALE * G).to(s["r"].dtype)
    du = BRANCH_SCALE * _gate_column(s) * G
    u = y
    if s["w_post"] is not None:
        dy, out["dw_post"], u = _norm_pullback(y, s["w_post"], du)
    else:
        dy = du
    out["dy"] = dy.to(s["y"].dtype)
    dg = BRANCH_SCALE * G * u
    kind = s["case"]["gate"]
    if kind == "channel":
        out["dgate"] = dg.sum(0)
    elif kind == "token":
        out["dgate"] = dg.sum(1)
    elif kind == "full":
        out["dgate"] = dg.to(s["gate"].dtype)
    return out


def _blocks(scale, rows, cols, row_block):
    """A block scale spread over the values it stands for."""
    return scale.repeat_interleave(128, -1)[..., :cols].repeat_interleave(row_block, -2)[..., :rows, :]


def _padded(s, x):
    """Rows [R, c] as [G, most, c] with zeros behind each group's rows, and where they came from."""
    off = s["off"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=x.device)
    there = at < off[1:, None]
    at = torch.where(there, at, torch.zeros_like(at))
    return torch.where(there[..., None], x[at].float(), 0.0), at, there


def _plain_product(s, op):
    out = torch.zeros(s["out"].shape, device=DEV, dtype=s["out"].dtype)
    if op == "wgrad":
        dy, _, _ = _padded(s, s["dy"])
        a, _, _ = _padded(s, s["a"])
        return torch.bmm(dy.transpose(1, 2), a).to(out.dtype)
    x = s["a"] if op == "gemm" else s["dy"]
    w = s["w"].float()
    if s["a_scale"] is not None:
        w = w * _blocks(s["w_scale"], w.shape[-2], w.shape[-1], 128)
        x = x.float() * _blocks(s["a_scale"], x.shape[0], x.shape[1], 1)
    x, at, there = _padded(s, x)
    y = torch.bmm(x, w.transpose(1, 2) if op == "gemm" else w)
    out[at[there]] = y[there].to(out.dtype)
    return out


# ---------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(case, s)
    D = torch.float64
    out = torch.zeros(s["out"].shape, device=DEV, dtype=D)
    lo = 0
    for g, m in enumerate(s["sizes"]):
        hi = lo + m
        if m:
            if case["op"] == "wgrad":
                out[g] = s["dy"][lo:hi].to(D).T @ s["a"][lo:hi].to(D)
            elif case["op"] == "dgrad":
                out[lo:hi] = s["dy"][lo:hi].to(D) @ s["w"][g].to(D)
            elif case["dtype"] == "e4m3":
                for b in range(0, case["k"], 128):      # one block of 128 of the inner sum at a time
                    part = s["a"][lo:hi, b:b + 128].to(D) @ s["w"][g, :, b:b + 128].to(D).T
                    by = s["w_scale"][g, :, b // 128].to(D).repeat_interleave(128)[:case["n"]]
                    out[lo:hi] += part * s["a_scale"][lo:hi, b // 128, None].to(D) * by
            else:
                out[lo:hi] = s["a"][lo:hi].to(D) @ s["w"][g].to(D).T
        lo = hi
    return out


def _exact_norm(case, s):
    D = torch.float64
    f = {k: (None if s.get(k) is None else s[k].to(D)) for k in ("r", "y", "w_post", "w_pre", "gate", "dh", "dr_out")}
    if f["gate"] is not None and case["gate"] == "token":
        f["gate"] = f["gate"][:, None]
    back = case["op"] == "norm_bwd"
    leaf = {k: v.requires_grad_(True) for k, v in f.items() if back and v is not None and k not in ("dh", "dr_out")}

    def rms(x, w):
        return x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * (w + W_OFFSET)

    branch = f["y"] if f["w_post"] is None else rms(f["y"], f["w_post"])
    if f["gate"] is not None:
        branch = branch * f["gate"]
    if not back:
        new = RES_SCALE * f["r"] + BRANCH_SCALE * branch
        h = None if f["w_pre"] is None or case["out"] == "e4m3" else rms(new, f["w_pre"])
        return {"r_out": new, "h": h, "h_scale": None}
    # r' is an input of the backward pass: differentiate h(r') for it, then the branch
    up = f["dr_out"]
    if f["w_pre"] is not None:
        up = up + torch.autograd.grad(rms(leaf["r"], leaf["w_pre"]), leaf["r"], f["dh"])[0]
    got = {"dr": RES_SCALE * up, "dgate": None, "dw_post": None, "dw_pre": None}
    names = [k for k in ("y", "w_post", "gate") if k in leaf]
    grads = dict(zip(names, torch.autograd.grad(BRANCH_SCALE * branch, [leaf[k] for k in names], up)))
    got["dy"], got["dw_post"], got["dgate"] = (grads.get(k) for k in ("y", "w_post", "gate"))
    if got["dgate"] is not None and case["gate"] == "token":
        got["dgate"] = got["dgate"][:, 0]
    if f["w_pre"] is not None:
        got["dw_pre"] = torch.autograd.grad(rms(leaf["r"], leaf["w_pre"]), leaf["w_pre"], f["dh"])[0]
    return got


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "norm_bwd"):
        T, d, rb = case["T"], case["d"], 4 if case["res"] == "f32" else 2
        x = T * d
        vectors = 2 * d * (int(case["post"]) + int(case["pre"]))
        gate = {"none": 0, "channel": d, "token": T, "full": x}[case["gate"]]
        if case["op"] == "norm":
            h = {"bf16": 2 * x, "f32": 4 * x, "e4m3": x + x // 32}[case["out"]] if case["pre"] else 0
            return {"bytes": 2 * rb * x + 2 * x + h + vectors + 2 * gate, "flops": 12 * x}
        grads = 4 * d * (int(case["post"]) + int(case["pre"])) + (2 if case["gate"] == "full" else 4) * gate
        return {"bytes": 3 * rb * x + 4 * x + (2 * x if case["pre"] else 0) + vectors + 2 * gate + grads,
                "flops": 24 * x}
    G, n, k, m = case["G"], case["n"], case["k"], case["rows"]
    used = sum(v > 0 for v in group_sizes(case))
    ob = 4 if case["out"] == "f32" else 2
    flops = 2 * m * n * k
    if case["op"] == "wgrad":
        return {"bytes": 2 * m * (n + k) + ob * G * n * k, "flops": flops}
    if case["dtype"] == "e4m3":
        return {"bytes": m * k + used * n * k + ob * m * n + 4 * m * (k // 128) + 4 * used * (n // 128) * (k // 128),
                "flops": flops}
    inner, outer = (k, n) if case["op"] == "gemm" else (n, k)
    return {"bytes": 2 * m * inner + 2 * used * n * k + ob * m * outer, "flops": flops}
