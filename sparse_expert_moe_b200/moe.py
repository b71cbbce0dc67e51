"""Python binding of the C ABI in ``include/moe.h`` (argument marshalling only).

Every function keeps the C name and argument order; tensors are passed as
device pointers (``tensor.data_ptr()``), ``None`` as NULL, and the stream
defaults to PyTorch's current stream.  All arithmetic happens in the CUDA
library ``libmoe_b200.so``; if it is missing the import fails loudly -- there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe.h")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
                4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_INDEX", 6: "MOE_ERR_TIMEOUT",
                7: "MOE_ERR_DEVICE_VALUE"}
SCORE = {"softmax": 0, "sigmoid_bias": 1}
GATE = {"none": 0, "channel": 1, "token": 2, "full": 3}
DTYPE = {"f32": 0, "bf16": 1, "e4m3": 2, "e2m1": 3, "e4m3_fs": 4}


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(code, code)}")
        self.code = code


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("E", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("score", ctypes.c_int), ("act", ctypes.c_int),
                ("weight", ctypes.c_int), ("out", ctypes.c_int)]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("wr", "sel_bias", "w13", "w2", "w13_s", "w2_s",
                                                "ws13", "ws2", "ws13_s", "ws2_s")]


class MoeNormConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("gate", ctypes.c_int),
                ("res", ctypes.c_int), ("act", ctypes.c_int), ("weight", ctypes.c_int),
                ("out", ctypes.c_int), ("eps", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("w_offset", ctypes.c_float)]


class MoeProductConfig(ctypes.Structure):
    _fields_ = [("n_groups", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("in_", ctypes.c_int), ("out", ctypes.c_int)]


_lib: Optional[ctypes.CDLL] = None


def load_library() -> ctypes.CDLL:
    """Load libmoe_b200.so (built by ``python -m sparse_expert_moe_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_expert_moe_b200.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    cfgp = ctypes.POINTER(MoeConfig)
    sigs = {
        "moe_workspace_size": [cfgp, ctypes.POINTER(SZ)],
        "moe_route": [cfgp, P, P, P, P, P],
        "moe_permute": [cfgp, P, P, P, P, P, P, P, P, P, SZ, P],
        "moe_permute_noalloc": [cfgp, P, P, P, P, P, P, P, P, P],
        "moe_grouped_ffn": [cfgp, I32, P, I32, P, P, P, P, P, P, P, P, SZ, P],
        "moe_combine": [cfgp, P, P, P, P, P, P],
        "moe_layer_forward": [cfgp, ctypes.POINTER(MoeWeights), P, P, P, P, P, P, SZ, P],
        "moe_layer_forward_staged": [cfgp, ctypes.POINTER(MoeWeights), P, P, P, P, P, P, SZ, P,
                                     ctypes.POINTER(ctypes.c_void_p)],
        "moe_read_device_status": [P, P, ctypes.POINTER(ctypes.c_int)],
        "moe_reset_device_status": [P, P],
        "moe_selftest_bounded_wait": [P, ctypes.c_longlong, P],
        "moe_layer_graph_create": [cfgp, ctypes.POINTER(MoeWeights), P, P, P, P, P, P, SZ,
                                   ctypes.POINTER(ctypes.c_void_p)],
        "moe_layer_graph_launch": [P, P],
        "moe_layer_graph_destroy": [P],
        "moe_norm_workspace_size": [ctypes.POINTER(MoeNormConfig), ctypes.POINTER(SZ)],
        "moe_block_norm": [ctypes.POINTER(MoeNormConfig)] + [P] * 9,
        "moe_block_norm_backward": [ctypes.POINTER(MoeNormConfig)] + [P] * 13 + [SZ, P],
        "moe_product_workspace_size": [ctypes.POINTER(MoeProductConfig), ctypes.POINTER(SZ)],
        "moe_grouped_gemm": [ctypes.POINTER(MoeProductConfig)] + [P] * 7 + [SZ, P],
        "moe_grouped_gemm_dgrad": [ctypes.POINTER(MoeProductConfig)] + [P] * 5 + [SZ, P],
        "moe_grouped_gemm_wgrad": [ctypes.POINTER(MoeProductConfig)] + [P] * 5 + [SZ, P],
    }
    for name, argtypes in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def declared_symbols():
    """Names of the entry points include/moe.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text, flags=re.M)


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _p(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name: str, code: int):
    if code != MOE_OK:
        raise MoeError(name, code)


def make_config(T, d_model, E, top_k, d_ff, n_shared=0, score="sigmoid_bias", act="bf16",
                weight="bf16", out="bf16") -> MoeConfig:
    return MoeConfig(T, d_model, E, top_k, d_ff, n_shared, d_ff if n_shared else 0, SCORE[score],
                     DTYPE[act], DTYPE[weight], DTYPE[out])


def config_from_spec(spec, T: Optional[int] = None) -> MoeConfig:
    return make_config(spec.T if T is None else T, spec.d_model, spec.E, spec.top_k, spec.d_ff,
                       spec.n_shared, spec.score, spec.act, spec.weight, spec.out)


# ---------------------------------------------------------------------------
# the C entry points
# ---------------------------------------------------------------------------

def moe_workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_workspace_size", load_library().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def moe_route(cfg, logits, sel_bias, topk_idx, topk_w, stream=None):
    _check("moe_route", load_library().moe_route(ctypes.byref(cfg), _p(logits), _p(sel_bias),
                                                 _p(topk_idx), _p(topk_w), _stream(stream)))


def moe_permute(cfg, topk_idx, x, x_scale, x_perm, x_perm_scale, perm_token, inv_perm,
                group_offsets, ws, stream=None):
    _check("moe_permute", load_library().moe_permute(
        ctypes.byref(cfg), _p(topk_idx), _p(x), _p(x_scale), _p(x_perm), _p(x_perm_scale),
        _p(perm_token), _p(inv_perm), _p(group_offsets), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_permute_noalloc(cfg, topk_idx, x, x_scale, x_perm, x_perm_scale, perm_token, inv_perm,
                        group_offsets, stream=None):
    """moe_permute without a workspace (scratch inside the library; see include/moe.h)."""
    _check("moe_permute_noalloc", load_library().moe_permute_noalloc(
        ctypes.byref(cfg), _p(topk_idx), _p(x), _p(x_scale), _p(x_perm), _p(x_perm_scale),
        _p(perm_token), _p(inv_perm), _p(group_offsets), _stream(stream)))


def moe_grouped_ffn(cfg, n_groups, group_offsets, n_rows, a, a_scale, w13, w13_s, w2, w2_s, y, ws,
                    stream=None):
    _check("moe_grouped_ffn", load_library().moe_grouped_ffn(
        ctypes.byref(cfg), n_groups, _p(group_offsets), n_rows, _p(a), _p(a_scale), _p(w13),
        _p(w13_s), _p(w2), _p(w2_s), _p(y), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_combine(cfg, y_perm, inv_perm, topk_w, y_shared, y, stream=None):
    _check("moe_combine", load_library().moe_combine(
        ctypes.byref(cfg), _p(y_perm), _p(inv_perm), _p(topk_w), _p(y_shared), _p(y),
        _stream(stream)))


def make_weights(wr, sel_bias, w13, w2, ws13=None, ws2=None, w13_s=None, w2_s=None, ws13_s=None,
                 ws2_s=None) -> MoeWeights:
    return MoeWeights(_p(wr), _p(sel_bias), _p(w13), _p(w2), _p(w13_s), _p(w2_s), _p(ws13), _p(ws2),
                      _p(ws13_s), _p(ws2_s))


def moe_layer_forward(cfg, weights: MoeWeights, x, x_scale, y, topk_idx_out, topk_w_out, ws,
                      stream=None):
    _check("moe_layer_forward", load_library().moe_layer_forward(
        ctypes.byref(cfg), ctypes.byref(weights), _p(x), _p(x_scale), _p(y), _p(topk_idx_out),
        _p(topk_w_out), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


STAGES = ("router_gemm", "route", "permute", "plan", "ffn1", "ffn2", "combine")


def moe_layer_forward_staged(cfg, weights: MoeWeights, x, x_scale, y, topk_idx_out, topk_w_out, ws,
                             events, stream=None):
    """``events``: 8 recorded-once ``torch.cuda.Event(enable_timing=True)`` objects."""
    handles = (ctypes.c_void_p * 8)(*[ev.cuda_event for ev in events])
    _check("moe_layer_forward_staged", load_library().moe_layer_forward_staged(
        ctypes.byref(cfg), ctypes.byref(weights), _p(x), _p(x_scale), _p(y), _p(topk_idx_out),
        _p(topk_w_out), _p(ws), ws.numel() * ws.element_size(), _stream(stream), handles))


class LayerGraph:
    """moe_layer_graph_create / _launch / _destroy: the layer recorded once for fixed
    tensors (x, y, routing outputs, workspace) and replayed with one graph launch."""

    def __init__(self, cfg, weights: MoeWeights, x, x_scale, y, topk_idx_out, topk_w_out, ws):
        h = ctypes.c_void_p(0)
        _check("moe_layer_graph_create", load_library().moe_layer_graph_create(
            ctypes.byref(cfg), ctypes.byref(weights), _p(x), _p(x_scale), _p(y), _p(topk_idx_out),
            _p(topk_w_out), _p(ws), ws.numel() * ws.element_size(), ctypes.byref(h)))
        self._h = h
        self._keep = (cfg, weights, x, x_scale, y, topk_idx_out, topk_w_out, ws)

    def launch(self, stream=None):
        _check("moe_layer_graph_launch", load_library().moe_layer_graph_launch(self._h, _stream(stream)))

    def close(self):
        if self._h:
            _check("moe_layer_graph_destroy", load_library().moe_layer_graph_destroy(self._h))
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_read_device_status(ws, stream=None) -> int:
    v = ctypes.c_int(0)
    _check("moe_read_device_status",
           load_library().moe_read_device_status(_p(ws), _stream(stream), ctypes.byref(v)))
    return v.value


def moe_reset_device_status(ws, stream=None):
    _check("moe_reset_device_status", load_library().moe_reset_device_status(_p(ws), _stream(stream)))


def moe_selftest_bounded_wait(ws, budget_cycles, stream=None):
    _check("moe_selftest_bounded_wait",
           load_library().moe_selftest_bounded_wait(_p(ws), int(budget_cycles), _stream(stream)))


def moe_status_string(code: int) -> str:
    return load_library().moe_status_string(code).decode()


# ---------------------------------------------------------------------------
# norms around a block; products grouped by expert
# ---------------------------------------------------------------------------

_VALUE_TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float8_e4m3fn, 4: torch.float8_e4m3fn}


def _device_of(*tensors) -> int:
    """Index of the CUDA device of the first tensor among them (-1: only addresses)."""
    for t in tensors:
        if t is not None and type(t) is not int:
            d = t.get_device()
            return d if d >= 0 else -2
    return -1


def _in_rows(t, row: int) -> bool:
    """Whether a tensor's last dimensions are `row` elements together, or it is flat."""
    if t.dim() < 2:
        return True
    n = 1
    for size in reversed(t.shape):
        if n == row:
            return True
        n *= size
    return n == row or n == 0                    # one row, or no elements


def _addr(fn: str, name: str, t, want, numel: int, device: int, row: int = 0):
    """Device address of a tensor of one call, checked: its type (None: any), element count,
    contiguity and device, and (matrices of a product) the length of its rows, which is what tells a
    weight from its transpose.  None and plain integers (device addresses) pass."""
    if t is None or type(t) is int:
        return t
    if (t.dtype is want or want is None) and t.numel() == numel and t.is_contiguous() and \
            t.get_device() == device and (not row or t.shape[-1] == row or _in_rows(t, row)):
        return t.data_ptr()
    if want is torch.float8_e4m3fn and t.dtype is torch.uint8:       # codes as bytes
        return _addr(fn, name, t, torch.uint8, numel, device, row)
    if want is not None and t.dtype is not want:
        raise TypeError(f"{fn}: {name} is {t.dtype}, not {want}")
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous with {numel} elements, got shape "
                         f"{tuple(t.shape)}, strides {t.stride()}")
    if row and not _in_rows(t, row):
        raise ValueError(f"{fn}: {name} must have rows of {row} elements, got shape {tuple(t.shape)}")
    raise ValueError(f"{fn}: {name} is not on the CUDA device of the other tensors")


def _workspace(fn: str, ws, device: int):
    if ws is None or type(ws) is int:
        raise TypeError(f"{fn}: the workspace is a tensor")
    n = ws.numel()
    return _addr(fn, "ws", ws, None, n, device), n * ws.element_size()


def _call(fn: str, device: int, stream, *args):
    """The C call on the tensors' device, on `stream` or that device's current stream."""
    f = getattr(_lib or load_library(), fn)
    if device < 0:
        code = f(*args, _stream(stream))
    elif device == torch._C._cuda_getDevice():       # its tensors have initialised CUDA
        code = f(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(device):
            code = f(*args, _stream(stream))
    if code != MOE_OK:
        raise MoeError(fn, code)


def make_norm_config(T, d_model, gate="none", res="bf16", act="bf16", weight="bf16", out="bf16", eps=1e-6,
                     res_scale=1.0, branch_scale=1.0, w_offset=0.0) -> MoeNormConfig:
    return MoeNormConfig(T, d_model, GATE[gate], DTYPE[res], DTYPE[act], DTYPE[weight], DTYPE[out], eps,
                         res_scale, branch_scale, w_offset)


def moe_norm_workspace_size(cfg: MoeNormConfig) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_norm_workspace_size",
           load_library().moe_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def _gate_shape(cfg: MoeNormConfig):
    """(elements, type code) of the gate."""
    if cfg.gate == 3:
        return cfg.T * cfg.d_model, cfg.act
    return (cfg.T if cfg.gate == 2 else cfg.d_model), cfg.weight


def moe_block_norm(cfg: MoeNormConfig, r, y, w_post, gate, w_pre, r_out, h, h_scale, stream=None):
    """r_out = res_scale r + branch_scale gate norm(y; w_post), h = norm(r_out; w_pre); see
    include/moe.h for what may be None."""
    fn, D = "moe_block_norm", _VALUE_TYPES.get
    dev = _device_of(r, y, w_post, gate, w_pre, r_out, h, h_scale)
    d, n = cfg.d_model, cfg.T * cfg.d_model
    res, act, wt = D(cfg.res), D(cfg.act), D(cfg.weight)
    gn, gt = _gate_shape(cfg)
    _call(fn, dev, stream, ctypes.byref(cfg), _addr(fn, "r", r, res, n, dev), _addr(fn, "y", y, act, n, dev),
          _addr(fn, "w_post", w_post, wt, d, dev), _addr(fn, "gate", gate, D(gt), gn, dev),
          _addr(fn, "w_pre", w_pre, wt, d, dev), _addr(fn, "r_out", r_out, res, n, dev),
          _addr(fn, "h", h, D(cfg.out), n, dev), _addr(fn, "h_scale", h_scale, torch.float32, n // 128, dev))


def moe_block_norm_backward(cfg: MoeNormConfig, r_out, y, w_post, gate, w_pre, dh, dr_out, dr, dy, dgate,
                            dw_post, dw_pre, ws, stream=None):
    """Gradients of moe_block_norm (dr, dy and, where not None, dgate, dw_post, dw_pre)."""
    fn, D, f32 = "moe_block_norm_backward", _VALUE_TYPES.get, torch.float32
    dev = _device_of(r_out, y, w_post, gate, w_pre, dh, dr_out, dr, dy, dgate, dw_post, dw_pre, ws)
    d, n = cfg.d_model, cfg.T * cfg.d_model
    res, act, wt = D(cfg.res), D(cfg.act), D(cfg.weight)
    gn, gt = _gate_shape(cfg)
    _call(fn, dev, stream, ctypes.byref(cfg), _addr(fn, "r_out", r_out, res, n, dev),
          _addr(fn, "y", y, act, n, dev), _addr(fn, "w_post", w_post, wt, d, dev),
          _addr(fn, "gate", gate, D(gt), gn, dev), _addr(fn, "w_pre", w_pre, wt, d, dev),
          _addr(fn, "dh", dh, act, n, dev), _addr(fn, "dr_out", dr_out, res, n, dev),
          _addr(fn, "dr", dr, res, n, dev), _addr(fn, "dy", dy, act, n, dev),
          _addr(fn, "dgate", dgate, act if cfg.gate == 3 else f32, gn, dev),
          _addr(fn, "dw_post", dw_post, f32, d, dev), _addr(fn, "dw_pre", dw_pre, f32, d, dev),
          *_workspace(fn, ws, dev))


def make_product_config(n_groups, n_rows, n, k, dtype="bf16", out="bf16") -> MoeProductConfig:
    return MoeProductConfig(n_groups, n_rows, n, k, DTYPE[dtype], DTYPE[out])


def moe_product_workspace_size(cfg: MoeProductConfig) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_product_workspace_size",
           load_library().moe_product_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def moe_grouped_gemm(cfg: MoeProductConfig, group_offsets, a, a_scale, w, w_scale, y, ws, stream=None):
    """y[r] = a[r] W_g^T for the rows r of group g (bf16, or e4m3 with block scales)."""
    fn, f32 = "moe_grouped_gemm", torch.float32
    dev = _device_of(a, w, y, group_offsets, a_scale, w_scale, ws)
    G, R, n, k, vt = cfg.n_groups, cfg.n_rows, cfg.n, cfg.k, _VALUE_TYPES.get(cfg.in_)
    kb = (k + 127) // 128
    _call(fn, dev, stream, ctypes.byref(cfg),
          _addr(fn, "group_offsets", group_offsets, torch.int32, G + 1, dev), _addr(fn, "a", a, vt, R * k, dev, k),
          _addr(fn, "a_scale", a_scale, f32, R * kb, dev, kb), _addr(fn, "w", w, vt, G * n * k, dev, k),
          _addr(fn, "w_scale", w_scale, f32, G * ((n + 127) // 128) * kb, dev, kb),
          _addr(fn, "y", y, _VALUE_TYPES.get(cfg.out), R * n, dev, n), *_workspace(fn, ws, dev))


def moe_grouped_gemm_dgrad(cfg: MoeProductConfig, group_offsets, dy, w, da, ws, stream=None):
    """da[r] = dy[r] W_g: the gradient of moe_grouped_gemm's rows."""
    fn = "moe_grouped_gemm_dgrad"
    dev = _device_of(dy, w, da, group_offsets, ws)
    G, R, n, k, vt = cfg.n_groups, cfg.n_rows, cfg.n, cfg.k, _VALUE_TYPES.get(cfg.in_)
    _call(fn, dev, stream, ctypes.byref(cfg),
          _addr(fn, "group_offsets", group_offsets, torch.int32, G + 1, dev), _addr(fn, "dy", dy, vt, R * n, dev, n),
          _addr(fn, "w", w, vt, G * n * k, dev, k), _addr(fn, "da", da, _VALUE_TYPES.get(cfg.out), R * k, dev, k),
          *_workspace(fn, ws, dev))


def moe_grouped_gemm_wgrad(cfg: MoeProductConfig, group_offsets, dy, a, dw, ws, stream=None):
    """dw_g = sum of dy[r]^T a[r] over the rows of group g: the gradient of the weights."""
    fn = "moe_grouped_gemm_wgrad"
    dev = _device_of(dw, dy, a, group_offsets, ws)
    G, R, n, k, vt = cfg.n_groups, cfg.n_rows, cfg.n, cfg.k, _VALUE_TYPES.get(cfg.in_)
    _call(fn, dev, stream, ctypes.byref(cfg),
          _addr(fn, "group_offsets", group_offsets, torch.int32, G + 1, dev), _addr(fn, "dy", dy, vt, R * n, dev, n),
          _addr(fn, "a", a, vt, R * k, dev, k), _addr(fn, "dw", dw, _VALUE_TYPES.get(cfg.out), G * n * k, dev, k),
          *_workspace(fn, ws, dev))


# ---------------------------------------------------------------------------
# a resident layer: weights and workspace on the device
# ---------------------------------------------------------------------------

_TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
                "e4m3_fs": torch.float8_e4m3fn}


@dataclass
class DeviceLayer:
    """One layer's weights and workspace held in device memory."""
    cfg: MoeConfig
    tensors: dict
    weights: MoeWeights
    ws: torch.Tensor

    @classmethod
    def from_workload(cls, wl, device="cuda", T: Optional[int] = None):
        spec = wl.spec
        cfg = config_from_spec(spec, T)
        names = ("wr", "sel_bias", "w13", "w2", "w13_s", "w2_s", "ws13", "ws2", "ws13_s", "ws2_s")
        ten = {}
        for n in names:
            t = getattr(wl, n)
            ten[n] = None if t is None else t.to(device, non_blocking=False)
        weights = make_weights(ten["wr"], ten["sel_bias"], ten["w13"], ten["w2"], ten["ws13"],
                               ten["ws2"], ten["w13_s"], ten["w2_s"], ten["ws13_s"], ten["ws2_s"])
        ws = torch.zeros(moe_workspace_size(cfg), dtype=torch.uint8, device=device)
        return cls(cfg, ten, weights, ws)

    def output(self, device="cuda"):
        dt = torch.float32 if self.cfg.out == DTYPE["f32"] else torch.bfloat16
        return torch.empty((self.cfg.T, self.cfg.d_model), dtype=dt, device=device)

    def forward(self, x, x_scale=None, y=None, topk_idx=None, topk_w=None, stream=None):
        if y is None:
            y = self.output(x.device)
        moe_layer_forward(self.cfg, self.weights, x, x_scale, y, topk_idx, topk_w, self.ws, stream)
        return y
