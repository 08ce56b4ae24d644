"""ButterflyMoE expert forward on B200: a thin Python binding of libbfmoe.so.

Functions carry the C ABI's names (include/bfmoe.h) and take torch tensors
that live on the current CUDA device; torch only provides device memory and
streams.  Every compute step runs in the library's CUDA kernels, and a missing
library raises instead of falling back.  A call with ``stream`` runs on that
stream and makes its outputs and scratch as under ``torch.cuda.stream(stream)``;
ordering it with the streams that made its inputs and use its outputs is the
caller's part.

Each expert is W_i = B(phi_i) . W_base . B(theta_i)^T with one shared ternary
base (ButterflyMoE technical summary, gist.science, section 2.1); inference
applies B(theta)^T, the ternary product and B(phi) without forming W_i
(section 2.3).
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional

from . import capi
from .capi import BFMOE_BF16, BFMOE_F32, BfmoeError

__all__ = [
    "BfmoeError", "Layer", "ButterflyMoE", "bfmoe_pack_base", "bfmoe_unpack_base", "bfmoe_router_topk",
    "bfmoe_router_topk_noalloc", "bfmoe_moe_forward", "bfmoe_moe_workspace_size", "bfmoe_prepare_layer",
    "bfmoe_layer_tables_size", "bfmoe_prepare_gate", "bfmoe_gate_parts_size", "bfmoe_backward", "bfmoe_backward_workspace_size",
    "bfmoe_forward", "bfmoe_decode_forward", "bfmoe_materialize_expert", "bfmoe_workspace_size", "bfmoe_router_scratch_size", "bfmoe_check_device_error",
    "Scoring", "GradList", "bfmoe_router_logits", "bfmoe_route", "bfmoe_route_backward", "bfmoe_balance_loss",
    "bfmoe_route_workspace_size", "bfmoe_expert_backward", "bfmoe_grad_norm", "bfmoe_grad_clip",
    "bfmoe_grad_workspace_size",
    "bfmoe_launch_count", "bfmoe_profile_enable", "bfmoe_profile_collect", "bfmoe_last_error", "workspace",
]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream=None):
    """The stream's handle as an integer.  torch.cuda.current_stream() builds an
    object (3 us); the handle alone is there for generated kernels."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _made(stream, make, *args, **kw):
    """make(*args): the tensors of a call on ``stream``, None for the current
    one.  They come from the memory pool of the stream that the call runs on: a
    block of another stream's pool may still be in use there, by work that this
    call is not ordered behind.  The caller, on the current stream, uses them
    too, so they are not reused before that stream is done."""
    if stream is None:
        return make(*args, **kw)
    cuda = _torch().cuda
    here = cuda.current_stream()
    with cuda.stream(stream):
        made = make(*args, **kw)
    for t in made.values() if isinstance(made, dict) else made if isinstance(made, tuple) else (made,):
        if t is not None:
            t.record_stream(here)
    return made


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype=None, cuda=True, contiguous=True):
    if t is None:
        raise ValueError(f"{name} is required")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BFMOE_BF16
    if t.dtype == torch.float32:
        return BFMOE_F32
    raise ValueError(f"x must be float32 or bfloat16, got {t.dtype}")


def words_per_row(d: int) -> int:
    return max(1, (d + 15) // 16)


def bfmoe_last_error() -> str:
    return capi.lib().bfmoe_last_error().decode(errors="replace")


def bfmoe_launch_count() -> int:
    return int(capi.lib().bfmoe_launch_count())


def bfmoe_workspace_size(d: int, n_experts: int, T: int, k: int, x_dtype: int) -> int:
    return int(capi.lib().bfmoe_workspace_size(d, n_experts, T, k, x_dtype))


def bfmoe_router_scratch_size(d: int, n_experts: int, T: int, k: int, x_dtype: int) -> int:
    """Scratch bytes the router alone uses (what bfmoe_router_topk_noalloc checks)."""
    return int(capi.lib().bfmoe_router_scratch_size(d, n_experts, T, k, x_dtype))


def workspace(d: int, n_experts: int, T: int, k: int, x_dtype: int, device=None):
    """A device scratch buffer of bfmoe_workspace_size bytes."""
    torch = _torch()
    n = bfmoe_workspace_size(d, n_experts, T, k, x_dtype)
    if n == 0 and T > 0:
        raise ValueError("invalid sizes for a workspace")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def bfmoe_pack_base(w, out=None, stream=None):
    """int8 [d][d] ternary -> uint32 2-bit codes [d][max(1, d/16)] (synchronises)."""
    torch = _torch()
    _need(w, "w", torch.int8)
    d = w.shape[1]
    if w.dim() != 2 or w.shape[0] != d:
        raise ValueError("w must be [d][d]")
    if out is None:
        out = _made(stream, torch.empty, (d, words_per_row(d)), dtype=torch.int32, device=w.device)
    capi.check(capi.lib().bfmoe_pack_base(_ptr(w), d, _ptr(out), _stream(stream)))
    return out


def bfmoe_unpack_base(w_packed, d: int, out=None, stream=None):
    """Packed codes -> the exact bf16 matrix [d][d] the tensor-core product uses."""
    torch = _torch()
    _need(w_packed, "w_packed")
    if out is None:
        out = _made(stream, torch.empty, (d, d), dtype=torch.bfloat16, device=w_packed.device)
    capi.check(capi.lib().bfmoe_unpack_base(_ptr(w_packed), d, _ptr(out), _stream(stream)))
    return out


def _routing_buffers(T, N, k, dev, buckets=True):
    """(idx, gates, counts, offsets, rows)."""
    torch = _torch()
    out = (torch.empty((T, k), dtype=torch.int32, device=dev),
           torch.empty((T, k), dtype=torch.float32, device=dev))
    return out + ((torch.empty((N,), dtype=torch.int32, device=dev),
                   torch.empty((N + 1,), dtype=torch.int32, device=dev),
                   torch.empty((T * k,), dtype=torch.int32, device=dev)) if buckets else (None, None, None))


def bfmoe_router_topk(x, w_gate, bias, k: int, ws, out=None, stream=None, buckets: bool = True):
    """Returns (idx [T,k] int32, gates [T,k] f32, counts [N], offsets [N+1], rows [T*k]);
    with ``buckets=False`` the last three are None and are not built."""
    torch = _torch()
    _need(x, "x")
    _need(w_gate, "w_gate", torch.float32)
    if bias is not None:
        _need(bias, "bias", torch.float32)
    T, d = x.shape
    N = w_gate.shape[0]
    dev = x.device
    if out is None:
        out = _made(stream, _routing_buffers, T, N, k, dev, buckets)
    idx, gates, counts, offsets, rows = out
    capi.check(capi.lib().bfmoe_router_topk(
        _ptr(x), _dtype_code(x), T, d, _ptr(w_gate), _ptr(bias), N, k, _ptr(idx), _ptr(gates),
        _ptr(counts), _ptr(offsets), _ptr(rows), _ptr(ws), ws.numel() if ws is not None else 0,
        _stream(stream)))
    return out


def bfmoe_router_topk_noalloc(x, w_gate, bias, k: int, out=None, stream=None):
    """bfmoe_router_topk for callers that cannot allocate device memory at
    call time: no workspace argument, the library's built-in scratch array is
    used instead (see include/bfmoe.h for its size and sharing rules).  The
    outputs must be provided by the caller (``out``) to allocate nothing here;
    without ``out`` this wrapper allocates them with torch for convenience."""
    torch = _torch()
    _need(x, "x")
    _need(w_gate, "w_gate", torch.float32)
    if bias is not None:
        _need(bias, "bias", torch.float32)
    T, d = x.shape
    N = w_gate.shape[0]
    dev = x.device
    if out is None:
        out = _made(stream, _routing_buffers, T, N, k, dev)
    idx, gates, counts, offsets, rows = out
    capi.check(capi.lib().bfmoe_router_topk_noalloc(
        _ptr(x), _dtype_code(x), T, d, _ptr(w_gate), _ptr(bias), N, k, _ptr(idx), _ptr(gates),
        _ptr(counts), _ptr(offsets), _ptr(rows), _stream(stream)))
    return out


class Layer:
    """Device weights of one ButterflyMoE layer (packed base, alpha, angles)."""

    def __init__(self, w_packed, alpha: float, theta, phi):
        torch = _torch()
        _need(w_packed, "w_packed")
        _need(theta, "theta", torch.float32)
        _need(phi, "phi", torch.float32)
        self.n_experts, L, half = theta.shape
        self.d = 2 * half
        if L != int(round(math.log2(self.d))) or phi.shape != theta.shape:
            raise ValueError("theta and phi must be [N][log2 d][d/2]")
        self.w_packed, self.theta, self.phi = w_packed, theta, phi
        self.alpha = float(alpha)
        self.c = capi.BfmoeLayer(self.d, self.n_experts, w_packed.data_ptr(), ctypes.c_float(alpha),
                                 theta.data_ptr(), phi.data_ptr(), None, None)
        self.tables = None
        self.gate_parts = None

    def prepare(self, stream=None):
        """Build the weight tables once (bfmoe_prepare_layer); later calls with
        this layer read them instead of rebuilding them per call."""
        torch = _torch()
        n = bfmoe_layer_tables_size(self.d, self.n_experts)
        self.tables = _made(stream, torch.empty, max(n, 256), dtype=torch.uint8, device=self.theta.device)
        self.c.tables = None
        bfmoe_prepare_layer(self, self.tables, stream=stream)
        self.c.tables = self.tables.data_ptr()
        return self

    def unprepare(self):
        """Go back to building the tables per call."""
        self.c.tables = None
        self.tables = None
        return self

    def prepare_gate(self, w_gate, stream=None):
        """Split the router weights once (bfmoe_prepare_gate); the combined
        calls with this layer and the same w_gate then skip the split."""
        torch = _torch()
        _need(w_gate, "w_gate", torch.float32)
        N, d = w_gate.shape
        n = int(capi.lib().bfmoe_gate_parts_size(N, d))
        self.gate_parts = _made(stream, torch.empty, max(n, 256), dtype=torch.uint8, device=w_gate.device)
        capi.check(capi.lib().bfmoe_prepare_gate(_ptr(w_gate), N, d, _ptr(self.gate_parts), self.gate_parts.numel(),
                                                _stream(stream)))
        self.c.gate_parts = self.gate_parts.data_ptr()
        return self

    def unprepare_gate(self):
        """Go back to splitting the router weights per call."""
        self.c.gate_parts = None
        self.gate_parts = None
        return self

    @classmethod
    def from_host(cls, w_base, alpha, theta, phi, device="cuda", stream=None):
        """Pack an int8 ternary base and upload float32 angles."""
        torch = _torch()
        w = torch.as_tensor(w_base, dtype=torch.int8).to(device).contiguous()
        packed = bfmoe_pack_base(w, stream=stream)
        th = torch.as_tensor(theta, dtype=torch.float32).to(device).contiguous()
        ph = torch.as_tensor(phi, dtype=torch.float32).to(device).contiguous()
        return cls(packed, float(alpha), th, ph)


def bfmoe_gate_parts_size(n_experts: int, d: int) -> int:
    return int(capi.lib().bfmoe_gate_parts_size(n_experts, d))


def bfmoe_prepare_gate(w_gate, parts, stream=None):
    """Write the exact bf16 split of w_gate [N][d] into parts (device bytes)."""
    N, d = w_gate.shape
    capi.check(capi.lib().bfmoe_prepare_gate(_ptr(w_gate), N, d, _ptr(parts), parts.numel(), _stream(stream)))
    return parts


def bfmoe_layer_tables_size(d: int, n_experts: int) -> int:
    return int(capi.lib().bfmoe_layer_tables_size(d, n_experts))


def bfmoe_prepare_layer(layer: "Layer", tables, stream=None):
    """Write the layer's weight tables (cos/sin of the angles, bf16 base) into
    ``tables`` (a device byte tensor of bfmoe_layer_tables_size bytes)."""
    _need(tables, "tables")
    capi.check(capi.lib().bfmoe_prepare_layer(ctypes.byref(layer.c), _ptr(tables), tables.numel(), _stream(stream)))
    return tables


def bfmoe_forward(layer: Layer, x, k: int, idx, gates, offsets, rows, ws, y=None, stream=None):
    """y [T][d] (dtype of x) = sum_j g_j B(phi) (alpha W_base (B(theta)^T x))."""
    _need(x, "x")
    T, d = x.shape
    if d != layer.d:
        raise ValueError(f"x has width {d}, layer has d={layer.d}")
    if y is None:
        y = _made(stream, _torch().empty_like, x)
    capi.check(capi.lib().bfmoe_forward(
        ctypes.byref(layer.c), _ptr(x), _dtype_code(x), T, k, _ptr(idx), _ptr(gates), _ptr(offsets),
        _ptr(rows), _ptr(y), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))
    return y


def bfmoe_decode_forward(layer: Layer, x, k: int, idx, gates, y=None, stream=None):
    """Add-only small-batch forward: y [T][d] (dtype of x) from the routing
    idx / gates, the ternary product done by signed sums, float32 inside."""
    torch = _torch()
    _need(x, "x")
    T, d = x.shape
    if d != layer.d:
        raise ValueError(f"x has width {d}, layer has d={layer.d}")
    _need(idx, "idx", torch.int32)
    _need(gates, "gates", torch.float32)
    if y is None:
        y = _made(stream, _torch().empty_like, x)
    capi.check(capi.lib().bfmoe_decode_forward(
        ctypes.byref(layer.c), _ptr(x), _dtype_code(x), T, k, _ptr(idx), _ptr(gates), _ptr(y), _stream(stream)))
    return y


def bfmoe_backward_workspace_size(d: int, n_experts: int, T: int, k: int) -> int:
    return int(capi.lib().bfmoe_backward_workspace_size(d, n_experts, T, k))


def bfmoe_backward(layer: Layer, x, k: int, w_gate, routing, gy, bias_grad: bool = True, ws=None, stream=None):
    """Gradients of the layer for dL/dy = gy (float32 [T][d]), with the
    forward's routing (idx, gates, counts, offsets, rows).  Returns a dict of
    float32 tensors dx, dtheta, dphi, dw_base, dalpha, dw_gate and dbias
    (None when bias_grad is False)."""
    torch = _torch()
    _need(x, "x")
    _need(w_gate, "w_gate", torch.float32)
    _need(gy, "gy", torch.float32)
    T, d = x.shape
    if d != layer.d or tuple(gy.shape) != (T, d):
        raise ValueError("x and gy must be [T][d] with the layer's d")
    N = layer.n_experts
    idx, gates, _counts, offsets, rows = routing
    dev = x.device
    if ws is None:
        ws = _scratch(bfmoe_backward_workspace_size(d, N, T, k), dev, stream)
    f = dict(dtype=torch.float32, device=dev)
    out = _made(stream, lambda: {
        "dx": torch.empty((T, d), **f), "dtheta": torch.empty_like(layer.theta),
        "dphi": torch.empty_like(layer.phi), "dw_base": torch.empty((d, d), **f),
        "dalpha": torch.empty((1,), **f), "dw_gate": torch.empty((N, d), **f),
        "dbias": torch.empty((N,), **f) if bias_grad else None})
    capi.check(capi.lib().bfmoe_backward(
        ctypes.byref(layer.c), _ptr(x), _dtype_code(x), T, k, _ptr(w_gate), _ptr(idx), _ptr(gates), _ptr(offsets),
        _ptr(rows), _ptr(gy), _ptr(out["dx"]), _ptr(out["dtheta"]), _ptr(out["dphi"]), _ptr(out["dw_base"]),
        _ptr(out["dalpha"]), _ptr(out["dw_gate"]), _ptr(out["dbias"]), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bfmoe_moe_workspace_size(d: int, n_experts: int, T: int, k: int, x_dtype: int) -> int:
    return int(capi.lib().bfmoe_moe_workspace_size(d, n_experts, T, k, x_dtype))


def bfmoe_moe_forward(layer: Layer, x, w_gate, bias, k: int, ws, routing=None, y=None, stream=None):
    """Router + forward in one call (weight-only work overlaps the router on a
    side stream).  Returns (y, (idx, gates, counts, offsets, rows))."""
    torch = _torch()
    _need(x, "x")
    _need(w_gate, "w_gate", torch.float32)
    if bias is not None:
        _need(bias, "bias", torch.float32)
    T, d = x.shape
    if d != layer.d:
        raise ValueError(f"x has width {d}, layer has d={layer.d}")
    N = layer.n_experts
    dev = x.device
    if routing is None:
        routing = _made(stream, _routing_buffers, T, N, k, dev)
    if y is None:
        y = _made(stream, _torch().empty_like, x)
    idx, gates, counts, offsets, rows = routing
    capi.check(capi.lib().bfmoe_moe_forward(
        ctypes.byref(layer.c), _ptr(x), _dtype_code(x), T, _ptr(w_gate), _ptr(bias), k, _ptr(idx), _ptr(gates),
        _ptr(counts), _ptr(offsets), _ptr(rows), _ptr(y), _ptr(ws), ws.numel() if ws is not None else 0,
        _stream(stream)))
    return y, routing


def bfmoe_moe_host_workspace_size(d: int, n_experts: int, T: int, k: int, x_dtype: int, chunk: int = 0) -> int:
    return int(capi.lib().bfmoe_moe_host_workspace_size(d, n_experts, T, k, x_dtype, chunk))


def bfmoe_moe_forward_host(layer: Layer, x_host, w_gate, bias, k: int, y_host, ws, chunk: int = 0, stream=None):
    """Router + forward from and to host memory (pinned CPU tensors), the
    copies overlapped with the work in chunks of ``chunk`` tokens.  ``y_host``
    is complete once ``stream`` has been synchronised.  Returns y_host."""
    torch = _torch()
    for t, name in ((x_host, "x_host"), (y_host, "y_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    if y_host.shape != x_host.shape or y_host.dtype != x_host.dtype:
        raise ValueError("y_host must match x_host in shape and dtype")
    _need(w_gate, "w_gate", torch.float32)
    if bias is not None:
        _need(bias, "bias", torch.float32)
    T, d = x_host.shape
    if d != layer.d:
        raise ValueError(f"x has width {d}, layer has d={layer.d}")
    capi.check(capi.lib().bfmoe_moe_forward_host(
        ctypes.byref(layer.c), ctypes.c_void_p(x_host.data_ptr()), _dtype_code(x_host), T, _ptr(w_gate), _ptr(bias),
        k, ctypes.c_void_p(y_host.data_ptr()), chunk, _ptr(ws), ws.numel() if ws is not None else 0,
        _stream(stream)))
    return y_host


class Scoring:
    """How logits become experts and gates (bfmoe_scoring in include/bfmoe.h):
    ``score`` "softmax" or "sigmoid"; ``n_groups`` groups of consecutive
    experts of which ``top_groups`` are kept by their largest value
    (``group_score`` "max") or their two best scores ("top2"); gates over
    their sum (``renormalize``) or as the scores are; times ``scale``."""

    SCORES = {"softmax": capi.BFMOE_SCORE_SOFTMAX, "sigmoid": capi.BFMOE_SCORE_SIGMOID}
    GROUP_SCORES = {"max": capi.BFMOE_GROUP_MAX, "top2": capi.BFMOE_GROUP_TOP2}

    def __init__(self, score: str = "softmax", n_groups: int = 1, top_groups: int = 1, group_score: str = "max",
                 renormalize: bool = True, scale: float = 1.0):
        self.c = capi.BfmoeScoring()   # holds every field, so that calls see a changed one
        self.ref = ctypes.byref(self.c)
        self.score, self.n_groups, self.top_groups, self.group_score = score, n_groups, top_groups, group_score
        self.renormalize, self.scale = renormalize, scale

    @staticmethod
    def _code(codes, name, value):
        if value not in codes:
            raise ValueError(f"{name} must be one of {sorted(codes)}, got {value!r}")
        return codes[value]

    @property
    def score(self) -> str:
        return next(s for s, code in self.SCORES.items() if code == self.c.score)

    @score.setter
    def score(self, value):
        self.c.score = self._code(self.SCORES, "score", value)

    @property
    def group_score(self) -> str:
        return next(s for s, code in self.GROUP_SCORES.items() if code == self.c.group_score)

    @group_score.setter
    def group_score(self, value):
        self.c.group_score = self._code(self.GROUP_SCORES, "group_score", value)

    n_groups = property(lambda self: self.c.n_groups, lambda self, value: setattr(self.c, "n_groups", value))
    top_groups = property(lambda self: self.c.top_groups, lambda self, value: setattr(self.c, "top_groups", value))
    renormalize = property(lambda self: bool(self.c.renormalize),
                           lambda self, value: setattr(self.c, "renormalize", int(bool(value))))

    @property
    def scale(self) -> float:
        return self._scale

    @scale.setter
    def scale(self, value):
        self._scale = float(value)
        self.c.scale = self._scale

    def __repr__(self):
        return (f"Scoring(score={self.score!r}, n_groups={self.n_groups}, top_groups={self.top_groups}, "
                f"group_score={self.group_score!r}, renormalize={self.renormalize}, scale={self.scale})")


def _here(stream, *named):
    """The stream handle of a call whose tensors (name, tensor or None, ...)
    must all live on the current CUDA device."""
    dev = _torch().cuda.current_device()
    for i in range(1, len(named), 2):
        t = named[i]
        if t is not None and t.get_device() != dev:
            name = named[i - 1]
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    return _stream(stream)


def _need_shape(t, name, dtype, *shape):
    if t is not None and (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}, got {t.dtype} "
                         f"{tuple(t.shape)}")


def _logits(t, name="logits"):
    """(dtype code, T, N, row stride) of logits: rows of consecutive elements."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T][N]")
    T, N = t.shape
    ld, one = t.stride()
    if N > 1 and one != 1:
        raise ValueError(f"{name} must have consecutive elements in a row")
    if T <= 1:
        ld = N
    elif ld < N:
        raise ValueError(f"the rows of {name} overlap (stride {ld} for {N} experts)")
    torch = _torch()
    if t.dtype is torch.float32:
        return BFMOE_F32, T, N, ld
    if t.dtype is torch.bfloat16:
        return BFMOE_BF16, T, N, ld
    raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def bfmoe_route_workspace_size(n_experts: int, T: int, k: int) -> int:
    return int(capi.lib().bfmoe_route_workspace_size(n_experts, T, k))


def _scratch(n, dev, stream):
    """A workspace of one call, freed when the call returns (see _made)."""
    torch = _torch()
    if stream is None:
        return torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(max(n, 256), dtype=torch.uint8, device=dev)


def bfmoe_router_logits(x, w_gate, bias=None, logits=None, ws=None, stream=None):
    """Router logits x W_g^T (+ b) alone, float32 [T][N] (bfmoe_router_logits)."""
    torch = _torch()
    _need(x, "x")
    _need(w_gate, "w_gate", torch.float32)
    if x.dim() != 2 or w_gate.dim() != 2 or x.shape[1] != w_gate.shape[1]:
        raise ValueError("x must be [T][d] and w_gate [N][d]")
    T, d = x.shape
    N = w_gate.shape[0]
    _need_shape(bias, "bias", torch.float32, N)
    code = _dtype_code(x)
    if logits is None:
        logits = _made(stream, torch.empty, (T, N), dtype=torch.float32, device=x.device)
    _need_shape(logits, "logits", torch.float32, T, N)
    s = _here(stream, "x", x, "w_gate", w_gate, "bias", bias, "logits", logits, "ws", ws)
    if ws is None:
        ws = _scratch(bfmoe_workspace_size(d, N, T, 1, code), x.device, stream)
    capi.check(capi.lib().bfmoe_router_logits(_ptr(x), code, T, d, _ptr(w_gate), _ptr(bias), N, _ptr(logits),
                                              _ptr(ws), ws.numel(), s))
    return logits


def _route_outputs(logits, T, N, k, buckets):
    new, i32 = logits.new_empty, _torch().int32
    out = (new((T, k), dtype=i32), new((T, k), dtype=_torch().float32))
    return out + ((new(N, dtype=i32), new(N + 1, dtype=i32), new(T * k, dtype=i32)) if buckets else (None, None, None))


def bfmoe_route(logits, k: int, scoring: Scoring, balance_bias=None, ws=None, out=None, buckets: bool = True,
                stream=None):
    """Experts and gates from logits [T][N] (float32 or bfloat16, rows may be
    strided).  Returns (idx [T,k] int32, gates [T,k] f32, counts [N],
    offsets [N+1], rows [T*k]); with ``buckets=False`` the last three are None
    and are not built."""
    torch = _torch()
    code, T, N, ld = _logits(logits)
    _need_shape(balance_bias, "balance_bias", torch.float32, N)
    if out is None:
        out = _made(stream, _route_outputs, logits, T, N, k, buckets)
        idx, gates, counts, offsets, rows = out
        s = _here(stream, "logits", logits, "balance_bias", balance_bias, "ws", ws)
    else:
        idx, gates, counts, offsets, rows = out
        _need_shape(idx, "idx", torch.int32, T, k)
        _need_shape(gates, "gates", torch.float32, T, k)
        _need_shape(counts, "counts", torch.int32, N)
        _need_shape(offsets, "offsets", torch.int32, N + 1)
        _need_shape(rows, "rows", torch.int32, T * k)
        s = _here(stream, "logits", logits, "balance_bias", balance_bias, "idx", idx, "gates", gates,
                  "counts", counts, "offsets", offsets, "rows", rows, "ws", ws)
    if counts is not None and ws is None:
        ws = _scratch(bfmoe_route_workspace_size(N, T, k), logits.device, stream)
    capi.check(capi.lib().bfmoe_route(
        logits.data_ptr(), code, T, ld, N, k, scoring.ref, _ptr(balance_bias), _ptr(idx), _ptr(gates),
        _ptr(counts), _ptr(offsets), _ptr(rows), _ptr(ws), ws.nbytes if ws is not None else 0, s))
    return out


def bfmoe_balance_loss(logits, idx, score: str = "softmax", ws=None, out=None, stream=None):
    """The load-balance and z losses of the routing idx [T,k] of logits [T][N]:
    (loss float32 [2], load int32 [N+1]: slots of each expert, then the rows
    that have an expert left)."""
    torch = _torch()
    code, T, N, ld = _logits(logits)
    if score not in Scoring.SCORES:
        raise ValueError(f"score must be one of {sorted(Scoring.SCORES)}, got {score!r}")
    if idx.dim() != 2:
        raise ValueError("idx must be [T][k]")
    k = idx.shape[1]
    _need_shape(idx, "idx", torch.int32, T, k)
    if out is None:
        out = (_made(stream, logits.new_empty, 2, dtype=torch.float32),
               _made(stream, logits.new_empty, N + 1, dtype=torch.int32))
    loss, load = out
    _need_shape(loss, "loss", torch.float32, 2)
    _need_shape(load, "load", torch.int32, N + 1)
    s = _here(stream, "logits", logits, "idx", idx, "loss", loss, "load", load, "ws", ws)
    if ws is None:
        ws = _scratch(bfmoe_route_workspace_size(N, T, k), logits.device, stream)
    capi.check(capi.lib().bfmoe_balance_loss(logits.data_ptr(), code, T, ld, N, k, Scoring.SCORES[score], _ptr(idx),
                                             loss.data_ptr(), load.data_ptr(), ws.data_ptr(), ws.nbytes, s))
    return out


def bfmoe_route_backward(logits, idx, scoring: Scoring, dgates=None, load=None, dloss=None, dlogits=None,
                         balance_bias=None, stream=None):
    """Gradient of the logits [T][N] (their dtype) from ``dgates`` [T,k], the
    gradient of bfmoe_route's gates, and from ``dloss`` [2], that of
    bfmoe_balance_loss's losses, with its ``load``.  ``balance_bias`` is needed
    where it masks experts (-inf)."""
    torch = _torch()
    code, T, N, ld = _logits(logits)
    if idx.dim() != 2:
        raise ValueError("idx must be [T][k]")
    k = idx.shape[1]
    _need_shape(idx, "idx", torch.int32, T, k)
    _need_shape(dgates, "dgates", torch.float32, T, k)
    _need_shape(load, "load", torch.int32, N + 1)
    _need_shape(dloss, "dloss", torch.float32, 2)
    _need_shape(balance_bias, "balance_bias", torch.float32, N)
    if dlogits is None:
        dlogits, ldd = _made(stream, logits.new_empty, (T, N)), N
    else:
        if dlogits.dtype is not logits.dtype or dlogits.shape != logits.shape:
            raise ValueError("dlogits must match logits in shape and dtype")
        ldd = _logits(dlogits, "dlogits")[3]
    s = _here(stream, "logits", logits, "idx", idx, "dgates", dgates, "load", load, "dloss", dloss, "dlogits", dlogits,
              "balance_bias", balance_bias)
    capi.check(capi.lib().bfmoe_route_backward(
        logits.data_ptr(), code, T, ld, N, k, scoring.ref, _ptr(balance_bias), _ptr(idx), _ptr(dgates), _ptr(load), _ptr(dloss),
        dlogits.data_ptr(), ldd, s))
    return dlogits


def bfmoe_expert_backward(layer: "Layer", x, k: int, routing, gy, ws=None, stream=None):
    """bfmoe_backward without the router: float32 dx (the experts' part),
    dtheta, dphi, dw_base, dalpha and dgates [T,k], the gradient of the gates
    for bfmoe_route_backward."""
    torch = _torch()
    _need(x, "x")
    T, d = x.shape
    N = layer.n_experts
    if d != layer.d:
        raise ValueError(f"x has width {d}, layer has d={layer.d}")
    idx, gates, _counts, offsets, rows = routing
    _need_shape(gy, "gy", torch.float32, T, d)
    _need_shape(idx, "idx", torch.int32, T, k)
    _need_shape(gates, "gates", torch.float32, T, k)
    for t, name, n in ((offsets, "offsets", N + 1), (rows, "rows", T * k)):
        if t is None:
            raise ValueError(f"{name} is required")
        _need_shape(t, name, torch.int32, n)
    s = _here(stream, "x", x, "gy", gy, "idx", idx, "gates", gates, "offsets", offsets, "rows", rows,
              "theta", layer.theta, "ws", ws)
    if ws is None:
        ws = _scratch(bfmoe_backward_workspace_size(d, N, T, k), x.device, stream)
    f = dict(dtype=torch.float32, device=x.device)
    out = _made(stream, lambda: {
        "dx": torch.empty((T, d), **f), "dtheta": torch.empty_like(layer.theta),
        "dphi": torch.empty_like(layer.phi), "dw_base": torch.empty((d, d), **f),
        "dalpha": torch.empty((1,), **f), "dgates": torch.empty((T, k), **f)})
    capi.check(capi.lib().bfmoe_expert_backward(
        ctypes.byref(layer.c), _ptr(x), _dtype_code(x), T, k, _ptr(idx), _ptr(gates), _ptr(offsets), _ptr(rows),
        _ptr(gy), _ptr(out["dx"]), _ptr(out["dtheta"]), _ptr(out["dphi"]), _ptr(out["dw_base"]), _ptr(out["dalpha"]),
        _ptr(out["dgates"]), _ptr(ws), ws.numel(), s))
    return out


def bfmoe_grad_workspace_size() -> int:
    return int(capi.lib().bfmoe_grad_workspace_size())


class GradList:
    """A list of gradients (float32 or bfloat16, contiguous) for bfmoe_grad_norm
    and bfmoe_grad_clip, with its workspace: made once, used every step while
    the gradients are these very tensors.  (bfmoe_backward and
    bfmoe_expert_backward return new ones each time: their list is made anew,
    or the call is given the tensors themselves.)  ``out``: tensors of the same shapes that
    bfmoe_grad_clip writes instead of scaling in place (None entries: in place).
    Calls that overlap on the GPU need a list each (they share its workspace,
    which is made on the stream that is current here)."""

    def __init__(self, grads, out=None):
        torch = _torch()
        self.grads = list(grads)
        self.out = list(out) if out is not None else [None] * len(self.grads)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.out)} outputs for {len(self.grads)} gradients")
        codes = {torch.float32: BFMOE_F32, torch.bfloat16: BFMOE_BF16}
        n = len(self.grads)
        dev = self.grads[0].get_device() if n else torch.cuda.current_device()
        fields = []
        for g, o in zip(self.grads, self.out):
            code = codes.get(g.dtype)
            if code is None or g.get_device() != dev or dev < 0 or not g.is_contiguous():
                self._refuse(len(fields) // 5, g, "gradient", dev)
            if o is None:
                fields += (g.data_ptr(), 0, g.numel(), code, code)
            else:
                out_code = codes.get(o.dtype)
                if out_code is None or o.get_device() != dev or not o.is_contiguous() or o.shape != g.shape:
                    self._refuse(len(fields) // 5, o, "output", dev, g)
                fields += (g.data_ptr(), o.data_ptr(), g.numel(), code, out_code)
        # (one structure made for each tensor took 1.7 us a tensor)
        packed = struct.pack("=" + "QQqii" * n, *fields) or bytes(ctypes.sizeof(capi.BfmoeGrad))
        self.c = (capi.BfmoeGrad * max(n, 1)).from_buffer_copy(packed)
        self.n = n
        self.device = torch.device("cuda", dev)
        self.ws = torch.empty(bfmoe_grad_workspace_size(), dtype=torch.uint8, device=self.device)

    @staticmethod
    def _refuse(i, t, name, dev, grad=None):
        name = f"{name} {i}"
        _need(t, name)
        if t.dtype not in (_torch().float32, _torch().bfloat16):
            raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, gradient 0 on cuda:{dev}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, its gradient {tuple(grad.shape)}")


def _grad_call(grads, norm, stream):
    """(GradList, norm, stream handle) of a call on the current device."""
    torch = _torch()
    g = grads
    if stream is not None:
        if not isinstance(g, GradList):
            with torch.cuda.stream(stream):  # the list's workspace goes when the call returns
                g = GradList(grads)
        else:
            g.ws.record_stream(stream)
    elif not isinstance(g, GradList):
        g = GradList(grads)
    if norm is None:
        norm = _made(stream, g.ws.new_empty, 1, dtype=torch.float32)
    else:
        _need_shape(norm, "norm", torch.float32, 1)
    return g, norm, _here(stream, "the gradients", g.ws, "norm", norm)


def bfmoe_grad_norm(grads, norm=None, stream=None):
    """The global norm (float32 [1]) of a GradList or of a sequence of tensors."""
    g, norm, s = _grad_call(grads, norm, stream)
    capi.check(capi.lib().bfmoe_grad_norm(g.c, g.n, norm.data_ptr(), g.ws.data_ptr(), g.ws.nbytes, s))
    return norm


def bfmoe_grad_clip(grads, max_norm: float, norm=None, stream=None):
    """Scale a GradList (or a sequence of tensors, in place) by
    min(1, max_norm / norm); returns the norm before it (float32 [1]).  An
    infinity or a NaN among the gradients leaves them as they are; a norm beyond
    float32 comes back as inf, too, but scales them."""
    g, norm, s = _grad_call(grads, norm, stream)
    capi.check(capi.lib().bfmoe_grad_clip(g.c, g.n, max_norm, norm.data_ptr(), g.ws.data_ptr(), g.ws.nbytes, s))
    return norm


def bfmoe_materialize_expert(layer: Layer, e: int, out=None, stream=None):
    """alpha * B(phi_e) . W_base . B(theta_e)^T as float32 [d][d] (checking aid)."""
    torch = _torch()
    if out is None:
        out = _made(stream, torch.empty, (layer.d, layer.d), dtype=torch.float32, device=layer.theta.device)
    capi.check(capi.lib().bfmoe_materialize_expert(ctypes.byref(layer.c), e, _ptr(out), _stream(stream)))
    return out


def bfmoe_check_device_error(stream=None) -> None:
    capi.check(capi.lib().bfmoe_check_device_error(_stream(stream)))


def bfmoe_profile_enable(on: bool = True) -> None:
    capi.check(capi.lib().bfmoe_profile_enable(1 if on else 0))


def bfmoe_profile_collect():
    """{kernel name: (launches, total ms)} since profiling was enabled."""
    buf = (capi.BfmoeKernelTime * 64)()
    n = ctypes.c_int(0)
    capi.check(capi.lib().bfmoe_profile_collect(buf, 64, ctypes.byref(n)))
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n.value)}


class ButterflyMoE:
    """Router + expert forward of one layer, with its own buffers.

    ``__call__(x)`` runs on device tensors; ``forward_host(x_host, y_host)``
    is the end-to-end call: pinned host tokens in, pinned host outputs back.

    With ``scoring`` the experts and gates come from bfmoe_route (on the logits
    x W_g^T + bias, ranked with ``balance_bias``) instead of the plain softmax
    router; the logits of the last call are in ``logits[:T]``.  forward_host
    then has no form.
    """

    def __init__(self, layer: Layer, w_gate, bias, k: int, max_tokens: int, x_dtype,
                 scoring: Optional[Scoring] = None, balance_bias=None):
        torch = _torch()
        if balance_bias is not None and scoring is None:
            raise ValueError("balance_bias needs a scoring")
        self.layer, self.w_gate, self.bias, self.k = layer, w_gate, bias, k
        self.scoring, self.balance_bias = scoring, balance_bias
        self.dtype = x_dtype
        code = BFMOE_BF16 if x_dtype == torch.bfloat16 else BFMOE_F32
        dev = layer.theta.device
        N, d = layer.n_experts, layer.d
        self.ws = workspace(d, N, max_tokens, k, code, dev)
        n = bfmoe_moe_workspace_size(d, N, max_tokens, k, code)
        self.ws_moe = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
        self.max_tokens = max_tokens
        self.idx = torch.empty((max_tokens, k), dtype=torch.int32, device=dev)
        self.gates = torch.empty((max_tokens, k), dtype=torch.float32, device=dev)
        self.counts = torch.empty((N,), dtype=torch.int32, device=dev)
        self.offsets = torch.empty((N + 1,), dtype=torch.int32, device=dev)
        self.rows = torch.empty((max_tokens * k,), dtype=torch.int32, device=dev)
        self.y_dev = torch.empty((max_tokens, d), dtype=x_dtype, device=dev)
        if scoring is not None:
            self.logits = torch.empty((max_tokens, N), dtype=torch.float32, device=dev)
            # the logits' and the routing's scratch, one after the other
            n = max(bfmoe_workspace_size(d, N, max_tokens, 1, code), bfmoe_route_workspace_size(N, max_tokens, k))
            self.ws_route = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)

    def _scored(self, x, out, stream):
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError("more tokens than the buffers hold")
        logits = bfmoe_router_logits(x, self.w_gate, self.bias, logits=self.logits[:T], ws=self.ws_route,
                                     stream=stream)
        return bfmoe_route(logits, self.k, self.scoring, balance_bias=self.balance_bias, ws=self.ws_route, out=out,
                           stream=stream)

    def route(self, x, stream=None):
        T = x.shape[0]
        if self.scoring is not None:
            return self._scored(x, (self.idx[:T], self.gates[:T], self.counts, self.offsets, self.rows[:T * self.k]),
                                stream)
        out = (self.idx[:T], self.gates[:T], self.counts, self.offsets, self.rows[:T * self.k])
        return bfmoe_router_topk(x, self.w_gate, self.bias, self.k, self.ws, out=out, stream=stream)

    def __call__(self, x, y=None, stream=None):
        """Router + forward of x (device) through bfmoe_moe_forward."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError("more tokens than the buffers hold")
        if y is None:
            y = self.y_dev[:T]
        if self.scoring is not None:
            idx, gates, _, offsets, rows = self.route(x, stream=stream)
            return bfmoe_forward(self.layer, x, self.k, idx, gates, offsets, rows, self.ws, y=y, stream=stream)
        routing = (self.idx[:T], self.gates[:T], self.counts, self.offsets, self.rows[:T * self.k])
        y, _ = bfmoe_moe_forward(self.layer, x, self.w_gate, self.bias, self.k, self.ws_moe, routing=routing, y=y,
                                 stream=stream)
        return y

    def decode(self, x, y=None, stream=None):
        """Router (no buckets) + the add-only small-batch forward
        (bfmoe_decode_forward)."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError("more tokens than the buffers hold")
        if y is None:
            y = self.y_dev[:T]
        idx, gates = self.idx[:T], self.gates[:T]
        if self.scoring is not None:
            self._scored(x, (idx, gates, None, None, None), stream)
            return bfmoe_decode_forward(self.layer, x, self.k, idx, gates, y=y, stream=stream)
        bfmoe_router_topk(x, self.w_gate, self.bias, self.k, self.ws, out=(idx, gates, None, None, None),
                          stream=stream)
        return bfmoe_decode_forward(self.layer, x, self.k, idx, gates, y=y, stream=stream)

    def forward_host(self, x_host, y_host, chunk: int = 0, stream=None):
        """The end-to-end call: pinned host tokens in, pinned host outputs back,
        through bfmoe_moe_forward_host (copies overlapped with the work in
        token chunks).  Synchronise ``stream`` before reading y_host."""
        torch = _torch()
        if self.scoring is not None:
            raise ValueError("forward_host routes by the plain softmax router only")
        T = x_host.shape[0]
        key = (T, chunk)
        if getattr(self, "_host_key", None) != key:
            code = BFMOE_BF16 if self.dtype == torch.bfloat16 else BFMOE_F32
            n = bfmoe_moe_host_workspace_size(self.layer.d, self.layer.n_experts, T, self.k, code, chunk)
            self.ws_host = _made(stream, torch.empty, max(n, 256), dtype=torch.uint8, device=self.layer.theta.device)
            self._host_key = key
        elif stream is not None:
            self.ws_host.record_stream(stream)
        return bfmoe_moe_forward_host(self.layer, x_host, self.w_gate, self.bias, self.k, y_host, self.ws_host,
                                      chunk=chunk, stream=stream)
