"""Calls of the block norms and the grouped products that have to be refused on the host, without a
GPU (`FAKE` is an aligned address that none of these paths dereferences)."""
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


BWD = ("r_out", "y", "w_post", "gate", "w_pre", "dh", "dr_out", "dr", "dy", "dgate", "dw_post", "dw_pre")


def backward_code(lib, config, **kw):
    a = {k: FAKE for k in BWD}
    a.update(kw)
    return lib.moe_block_norm_backward(ctypes.byref(config), *[a[k] for k in BWD], FAKE, 1 << 30, None)


@pytest.mark.parametrize("T", [0, 4])
def test_a_channel_gate_is_needed_without_rows_too(lib, T):
    """A [d] operand exists at every T; what has no rows may have no address."""
    c = moe.make_norm_config(T, 256, gate="channel")
    assert backward_code(lib, c, gate=None) == 1
    assert backward_code(lib, c, gate=None, dgate=None, dw_post=None, dw_pre=None) == 1


@pytest.mark.parametrize("gate", ["none", "token", "full"])
def test_backward_of_no_rows_has_no_addresses(lib, gate):
    """Nothing to compute, nothing to write: no launch, so the answer comes without a GPU."""
    c = moe.make_norm_config(0, 256, gate=gate)
    none = dict.fromkeys(("r_out", "y", "gate", "dh", "dr_out", "dr", "dy", "dgate", "dw_post", "dw_pre"))
    assert backward_code(lib, c, **none) == 0


def norm_code(lib, config, gate=None, h_scale=None):
    return lib.moe_block_norm(ctypes.byref(config), FAKE, FAKE, FAKE, gate, FAKE, FAKE, FAKE, h_scale, None)


@pytest.mark.parametrize("weight,gate", [("bf16", FAKE + 1), ("f32", FAKE + 1), ("f32", FAKE + 2)])
def test_token_gates_have_their_elements_alignment(lib, weight, gate):
    c = moe.make_norm_config(4, 256, gate="token", weight=weight)
    assert norm_code(lib, c, gate=gate) == 1
    assert backward_code(lib, c, gate=gate) == 1
    assert backward_code(lib, c, dgate=FAKE + 2) == 1


def test_scales_and_offsets_have_their_elements_alignment(lib):
    for odd in (1, 2):
        assert norm_code(lib, moe.make_norm_config(4, 256, out="e4m3"), h_scale=FAKE + odd) == 1
    c, f8 = (moe.make_product_config(4, 10, 256, 128, dtype=t) for t in ("bf16", "e4m3_fs"))
    size = moe.moe_product_workspace_size(c)

    def gemm(config, off=FAKE, sa=None, sw=None):
        return lib.moe_grouped_gemm(ctypes.byref(config), off, FAKE, sa, FAKE, sw, FAKE, FAKE, size, None)
    assert gemm(c, off=FAKE + 2) == 1
    assert gemm(f8, sa=FAKE + 2, sw=FAKE) == 1 and gemm(f8, sa=FAKE, sw=FAKE + 1) == 1
    for fn in (lib.moe_grouped_gemm_dgrad, lib.moe_grouped_gemm_wgrad):
        assert fn(ctypes.byref(c), FAKE + 2, FAKE, FAKE, FAKE, FAKE, size, None) == 1


def test_matrices_of_products_are_told_from_their_transposes(lib):
    """A contiguous [G, k, n] has the elements of a [G, n, k] and is refused; flat tensors, rows split
    into more dimensions and groups joined with rows are the same memory and pass (to the check of the
    device, the last one, which these tensors on the host fail)."""
    G, R, n, k = 4, 10, 256, 128
    c, ws = moe.make_product_config(G, R, n, k), torch.zeros(16, dtype=torch.uint8)
    f8 = moe.make_product_config(G, R, n, 256, dtype="e4m3_fs")

    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype)

    def calls(w):
        yield lambda: moe.moe_grouped_gemm(c, FAKE, FAKE, None, w, None, FAKE, ws, stream=0)
        yield lambda: moe.moe_grouped_gemm_dgrad(c, FAKE, FAKE, w, FAKE, ws, stream=0)
        yield lambda: moe.moe_grouped_gemm_wgrad(c, FAKE, FAKE, FAKE, w, ws, stream=0)
    for shape in ((G, k, n), (k, G * n), (G * k, n), (k, G, n)):
        for call in calls(t(*shape)):
            with pytest.raises(ValueError, match="rows of 128 elements"):
                call()
    for shape in ((G, n, k), (G * n, k), (G * n * k,), (G, n, 2, k // 2), (G, 2, n // 2, k), (G, n, k, 1)):
        for call in calls(t(*shape)):
            with pytest.raises(ValueError, match="not on the CUDA device"):
                call()
    for bad in (dict(a=t(k, R)), dict(y=t(n, R))):
        a = dict(dict(a=FAKE, y=FAKE), **bad)
        with pytest.raises(ValueError, match="rows of"):
            moe.moe_grouped_gemm(c, FAKE, a["a"], None, FAKE, None, a["y"], ws, stream=0)
    f32 = torch.float32
    for bad in (dict(sa=t(2, R, dtype=f32)), dict(sw=t(2, G, 2, dtype=f32).view(2, G * 2))):
        s = dict(dict(sa=FAKE, sw=FAKE), **bad)
        with pytest.raises(ValueError, match="rows of 2 elements"):
            moe.moe_grouped_gemm(f8, FAKE, FAKE, s["sa"], FAKE, s["sw"], FAKE, ws, stream=0)
    one = moe.make_product_config(1, R, 128, 128, dtype="e4m3_fs")          # rows of one scale
    for shape in ((R, 1), (1, R), (R,)):
        with pytest.raises(ValueError, match="not on the CUDA device"):
            moe.moe_grouped_gemm(one, FAKE, FAKE, t(*shape, dtype=f32), FAKE, FAKE, FAKE, ws, stream=0)
