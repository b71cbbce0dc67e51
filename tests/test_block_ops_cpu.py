"""Host checks of the block norms and the grouped products: refused calls launch nothing and
answer without a GPU (`FAKE` is an aligned address that none of these paths dereferences)."""
import ctypes
import os

import pytest
import torch

from sparse_expert_moe_b200 import moe

FAKE = 256


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from sparse_expert_moe_b200 import build
        build.build()
    return moe.load_library()


def refused(code, fn, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.code == code, (e.value.code, code)


# ------------------------------------------------------------------------------------ norms
NORM = dict(cfg={}, r=FAKE, y=FAKE, w_post=FAKE, gate=None, w_pre=FAKE, r_out=FAKE, h=FAKE, h_scale=None)


def norm_call(cfg=None, **kw):
    a = dict(NORM, **kw)
    a.pop("cfg")
    c = dict(T=4, d_model=256)
    c.update(cfg or {})
    config = moe.make_norm_config(c.pop("T"), c.pop("d_model"), **c)
    return (moe.moe_block_norm, config, a["r"], a["y"], a["w_post"], a["gate"], a["w_pre"], a["r_out"], a["h"],
            a["h_scale"])


@pytest.mark.parametrize("code,kw", [
    (1, dict(cfg=dict(T=-1))), (1, dict(cfg=dict(d_model=0))), (2, dict(cfg=dict(d_model=100))),
    (2, dict(cfg=dict(d_model=16392))), (2, dict(cfg=dict(T=(1 << 30) + 1))),
    (1, dict(cfg=dict(eps=0.0))), (1, dict(cfg=dict(eps=float("nan")))), (1, dict(cfg=dict(eps=float("inf")))),
    (1, dict(cfg=dict(res_scale=float("inf")))), (1, dict(cfg=dict(branch_scale=float("nan")))),
    (1, dict(cfg=dict(w_offset=float("nan")))),
    (2, dict(cfg=dict(res="e4m3"))), (2, dict(cfg=dict(act="e4m3"))), (2, dict(cfg=dict(weight="e2m1"))),
    (2, dict(cfg=dict(out="e2m1"))), (2, dict(cfg=dict(out="e4m3", d_model=264), h_scale=FAKE)),
    (1, dict(cfg=dict(out="e4m3"))),                     # no place for the scales
    (1, dict(h_scale=FAKE)),                             # scales of a bf16 h
    (1, dict(r=None)), (1, dict(y=None)),                # a post-norm of nothing
    (1, dict(gate=FAKE)), (1, dict(cfg=dict(gate="channel"))),
    (1, dict(h=None)), (1, dict(w_pre=None)), (1, dict(w_pre=None, h=None, r_out=None)),
    (1, dict(r=FAKE + 8)), (1, dict(h=FAKE + 2)), (1, dict(w_pre=FAKE + 4)),
    (1, dict(cfg=dict(gate="full"), gate=FAKE + 8)),
])
def test_norm_refusals(lib, code, kw):
    refused(code, *norm_call(**kw))


def test_norm_unknown_gate(lib):
    c = moe.make_norm_config(4, 256)
    c.gate = 7
    refused(1, moe.moe_block_norm, c, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, None)
    n = ctypes.c_size_t(0)
    assert lib.moe_norm_workspace_size(ctypes.byref(c), ctypes.byref(n)) == 1


def test_norm_of_no_tokens_is_a_no_op(lib):
    """Tensors without rows have null addresses: nothing about them is refused."""
    none = dict(r=None, y=None, r_out=None, h=None)
    for kw in (dict(cfg=dict(T=0), r=None), dict(cfg=dict(T=0), **none),
               dict(cfg=dict(T=0, out="e4m3"), h_scale=None, **none),
               dict(cfg=dict(T=0, gate="full"), **none)):
        fn, *args = norm_call(**kw)
        fn(*args, stream=0)


BWD = ("r_out", "y", "w_post", "gate", "w_pre", "dh", "dr_out", "dr", "dy", "dgate", "dw_post", "dw_pre")


@pytest.mark.parametrize("code,kw", [
    (1, dict(dh=None)), (1, dict(dr=None)), (1, dict(dy=None)), (1, dict(y=None)), (1, dict(r_out=None)),
    (1, dict(w_pre=None)), (1, dict(w_post=None)), (1, dict(dgate=FAKE)), (1, dict(gate=FAKE)),
    (1, dict(w_pre=None, dh=None, dw_pre=None, dr_out=None)),      # no gradient comes in
    (1, dict(dr=FAKE + 8)), (1, dict(dw_pre=FAKE + 4)), (1, dict(ws=None)), (3, dict(ws_bytes=1024)),
])
def test_norm_backward_refusals(lib, code, kw):
    a = {k: FAKE for k in BWD}
    a.update(gate=None, dgate=None)
    ws, size = kw.pop("ws", FAKE), kw.pop("ws_bytes", 1 << 30)
    a.update(kw)
    c = moe.make_norm_config(4, 256)
    assert lib.moe_block_norm_backward(ctypes.byref(c), *[a[k] for k in BWD], ws, size, None) == code


def test_norm_workspace_size(lib):
    # two fp32 partial sums per channel and SM at least
    for d in (8, 256, 7168, 16384):
        assert moe.moe_norm_workspace_size(moe.make_norm_config(10, d)) >= 256 + 148 * 2 * d * 4


# ------------------------------------------------------------------------------------ products
def product(**kw):
    c = dict(n_groups=4, n_rows=10, n=256, k=128)
    c.update(kw)
    return moe.make_product_config(**c)


def size_code(lib, c):
    n = ctypes.c_size_t(0)
    return lib.moe_product_workspace_size(ctypes.byref(c), ctypes.byref(n))


@pytest.mark.parametrize("code,kw", [
    (1, dict(n_groups=0)), (1, dict(n_rows=-1)), (1, dict(n=0)), (1, dict(k=-8)), (2, dict(n_groups=1025)),
    (2, dict(n=65544)), (2, dict(k=65544)), (2, dict(n=100)), (2, dict(k=100)), (2, dict(n_rows=(1 << 24) + 1)),
    (2, dict(dtype="f32")), (2, dict(dtype="e4m3")), (2, dict(out="e4m3")), (2, dict(dtype="e4m3_fs", k=136)),
    (0, dict(dtype="e4m3_fs", k=144)), (0, dict(n=8, k=8)), (0, dict(n_rows=0)),
])
def test_product_config(lib, code, kw):
    assert size_code(lib, product(**kw)) == code


def gemm_code(lib, c, off=FAKE, a=FAKE, sa=None, w=FAKE, sw=None, y=FAKE, ws=FAKE, size=1 << 30):
    return lib.moe_grouped_gemm(ctypes.byref(c), off, a, sa, w, sw, y, ws, size, None)


@pytest.mark.parametrize("code,kw", [
    (1, dict(off=None)), (1, dict(a=None)), (1, dict(w=None)), (1, dict(y=None)), (1, dict(ws=None)),
    (1, dict(a=FAKE + 8)), (1, dict(w=FAKE + 2)), (1, dict(y=FAKE + 4)), (1, dict(sa=FAKE)), (1, dict(sw=FAKE)),
    (3, dict(size=4096)),
])
def test_gemm_refusals(lib, code, kw):
    assert gemm_code(lib, product(), **kw) == code


def test_gemm_block_scales_are_required(lib):
    c = product(dtype="e4m3_fs")
    assert gemm_code(lib, c) == 1 and gemm_code(lib, c, sa=FAKE) == 1 and gemm_code(lib, c, sw=FAKE) == 1


def test_gradients_take_bf16_only(lib):
    c = product(dtype="e4m3_fs")
    for fn in (lib.moe_grouped_gemm_dgrad, lib.moe_grouped_gemm_wgrad):
        assert fn(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == 2
        for hole in range(4):
            args = [FAKE] * 4
            args[hole] = None
            assert fn(ctypes.byref(product()), *args, FAKE, 1 << 30, None) == 1
        assert fn(ctypes.byref(product()), FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 10, None) == 3
        assert fn(ctypes.byref(product()), FAKE, FAKE + 8, FAKE, FAKE, FAKE, 1 << 30, None) == 1


def test_no_rows_is_a_no_op(lib):
    c = product(n_rows=0)
    assert gemm_code(lib, c, a=None, w=None, y=None) == 0
    assert lib.moe_grouped_gemm_dgrad(ctypes.byref(c), FAKE, None, None, None, FAKE, 1 << 30, None) == 0


# ------------------------------------------------------------------------------------ binding
def test_binding_checks_tensors(lib):
    """Type, size, layout and device are checked before an address is taken."""
    c = moe.make_norm_config(4, 256)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="r is torch.float32"):
        moe.moe_block_norm(c, x.float(), FAKE, FAKE, None, FAKE, FAKE, FAKE, None, stream=0)
    with pytest.raises(ValueError, match="y must be contiguous with 1024"):
        moe.moe_block_norm(c, FAKE, x[:3], FAKE, None, FAKE, FAKE, FAKE, None, stream=0)
    with pytest.raises(ValueError, match="r must be contiguous"):
        moe.moe_block_norm(c, torch.zeros(256, 4, dtype=torch.bfloat16).T, FAKE, FAKE, None, FAKE, FAKE, FAKE, None,
                           stream=0)
    with pytest.raises(ValueError, match="not on the CUDA device"):
        moe.moe_block_norm(c, x, FAKE, FAKE, None, FAKE, FAKE, FAKE, None, stream=0)
    p, ws = product(), torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(TypeError, match="group_offsets"):
        moe.moe_grouped_gemm(p, torch.zeros(5, dtype=torch.int64), FAKE, None, FAKE, None, FAKE, ws, stream=0)
    with pytest.raises(TypeError, match="workspace"):
        moe.moe_grouped_gemm(p, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, stream=0)
    with pytest.raises(ValueError, match="ws is not on the CUDA device"):
        moe.moe_grouped_gemm(p, FAKE, FAKE, None, FAKE, None, FAKE, ws, stream=0)
