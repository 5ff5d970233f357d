"""torch-facing binding of the C ABI (argument marshalling only).

torch supplies device memory and the current HIP stream; every computation
is a kernel of libmoe_route.so.  Shapes are fixed per ``Dispatcher`` (the
handle is initialised once, like a static-shape buffer), and no call reads a
device value back to the host.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import NamedTuple, Optional

import torch

from . import _abi as A

_FMT = {"dense_i16": A.ROUTE_DENSE_I16, "dense_i32": A.ROUTE_DENSE_I32, "sparse_bool": A.ROUTE_SPARSE_BOOL}
_FMT_DTYPES = {A.ROUTE_DENSE_I16: (torch.int16,), A.ROUTE_DENSE_I32: (torch.int32,),
               A.ROUTE_SPARSE_BOOL: (torch.uint8, torch.bool, torch.int8)}
_DT = {"bf16": A.BF16, "fp8": A.FP8E4M3_B128, "int4": A.INT4_G128}
_ROW_DT = {torch.bfloat16: A.BF16, torch.float32: A.F32}
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)
_SCORE = {"softmax": A.GATE_SOFTMAX, "sigmoid": A.GATE_SIGMOID}
_ROUTING_OUT = {A.ROUTE_DENSE_I16: torch.int16, A.ROUTE_DENSE_I32: torch.int32, A.ROUTE_SPARSE_BOOL: torch.uint8}
_FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()      # c_void_p arguments take addresses as they are


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _stream():
    # the current stream's handle, without building a Stream object (2.9 us of a call that launches in 4)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def make_desc(T: int, H: int, E: int, K: int, route_fmt: str = "dense_i16", payload: str = "bf16",
              pad_multiple: int = 1, capacity: Optional[int] = None, out_rows: int = 0) -> A.MoeDesc:
    return A.MoeDesc(T=T, H=H, E=E, K=K, route_fmt=_FMT[route_fmt], payload=_DT[payload],
                     pad_multiple=pad_multiple, capacity=-1 if capacity is None else int(capacity),
                     out_rows=int(out_rows))


def out_rows_bound(T: int, H: int, E: int, K: int, pad_multiple: int = 1, capacity: Optional[int] = None,
                   route_fmt: str = "dense_i16", payload: str = "bf16") -> int:
    d = make_desc(T, H, E, K, route_fmt, payload, pad_multiple, capacity)
    return int(A.lib().moe_out_rows_bound(C.byref(d)))


def routing_bytes(T: int, E: int, K: int, route_fmt: str = "dense_i16") -> int:
    d = make_desc(T, 8, E, K, route_fmt)
    return int(A.lib().moe_routing_bytes(C.byref(d)))


def capacity_from_rows(rows: int, factor: float) -> int:
    return int(A.lib().moe_capacity_from_rows(int(rows), float(factor)))


def assert_no_overflow(flag: torch.Tensor) -> None:
    """Device-side assert that the overflow flag is clear; the host does not
    wait for it (the failure surfaces at the next synchronisation)."""
    torch._assert_async(flag[0] == 0)


# The checks below run on every call of a few microseconds: messages are only
# put together where a check fails.
def _check_rows(t, name, shape, dtypes):
    if t.dtype not in dtypes or t.shape != shape:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)} {list(shape)}, got {t.dtype} "
                         f"{list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_aligned(**tensors):
    """The calls' own condition on addresses, for checks ahead of them."""
    for name, t in tensors.items():
        if t is not None and t.data_ptr() % 16:
            raise ValueError(f"{name} must start at a multiple of 16 bytes")


def _check_current_device(tensors):
    """``tensors``: (name, tensor or None) pairs."""
    current = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None     # a CPU tensor's is -1
    for name, t in tensors:
        if t is not None and t.get_device() != current:
            raise ValueError(f"{name} must live on the current GPU")


def _check_norm_params(H, **params):
    """The parameters' common dtype (float32 where there are none)."""
    kind = None
    for name, p in params.items():
        if p is not None:
            _check_rows(p, name, (H,), _ROW_DT)
            _need(kind is None or p.dtype == kind, "weight and bias must share their dtype")
            kind = p.dtype
    return A.F32 if kind is None else _ROW_DT[kind]


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, *, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None):
    """Layer norm of rows x [T,H] (bf16 or fp32; weight and bias [H] of one of
    these types): (out [T,H], mean [T], rstd [T]), the last two fp32, for
    layer_norm_backward.  ``out`` is of ``out_dtype`` (default: x's).  Rows,
    weight and bias start at a multiple of 16 bytes, rows of any width follow
    each other without gaps."""
    _need(x.dim() == 2, "x must be [T,H]")
    T, H = x.shape
    _check_rows(x, "x", (T, H), _ROW_DT)
    wdt = _check_norm_params(H, weight=weight, bias=bias)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype or x.dtype, device=x.device)
    _check_rows(out, "out", (T, H), _ROW_DT)
    _need(out_dtype is None or out.dtype == out_dtype, "out must be of out_dtype")
    if mean is None:
        mean = torch.empty(T, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    _check_rows(mean, "mean", (T,), _F32)
    _check_rows(rstd, "rstd", (T,), _F32)
    _check_current_device((("x", x), ("weight", weight), ("bias", bias), ("out", out), ("mean", mean),
                           ("rstd", rstd)))
    A.check(A.lib().moe_layer_norm(T, H, _ROW_DT[x.dtype], _ROW_DT[out.dtype], wdt, _ptr(x), _ptr(weight), _ptr(bias),
                                   float(eps), _ptr(out), _ptr(mean), _ptr(rstd), _stream()), "moe_layer_norm")
    return out, mean, rstd


def layer_norm_backward_scratch_bytes(T: int, H: int) -> int:
    return int(A.lib().moe_layer_norm_backward_scratch_bytes(int(T), int(H)))


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
                        grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None,
                        scratch: Optional[torch.Tensor] = None, want_params: bool = True):
    """Gradients of a layer norm: (grad_x [T,H] of x's dtype, grad_weight [H],
    grad_bias [H]), the last two fp32, or None without ``want_params``.
    mean and rstd are the forward's."""
    _need(x.dim() == 2, "x must be [T,H]")
    T, H = x.shape
    _check_rows(x, "x", (T, H), _ROW_DT)
    _check_rows(grad_y, "grad_y", (T, H), _ROW_DT)
    _check_rows(mean, "mean", (T,), _F32)
    _check_rows(rstd, "rstd", (T,), _F32)
    wdt = _check_norm_params(H, weight=weight)
    if out is None:
        out = torch.empty_like(x)
    _check_rows(out, "out", (T, H), (x.dtype,))
    if want_params:
        if grad_weight is None:
            grad_weight = torch.empty(H, dtype=torch.float32, device=x.device)
        if grad_bias is None:
            grad_bias = torch.empty(H, dtype=torch.float32, device=x.device)
        _check_rows(grad_weight, "grad_weight", (H,), _F32)
        _check_rows(grad_bias, "grad_bias", (H,), _F32)
        need = layer_norm_backward_scratch_bytes(T, H)
        if need == 0:
            raise ValueError(f"rows of {H} elements are outside 1..{A.NORM_MAX_H}")
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=x.device)
        _need(scratch.is_contiguous(), "scratch must be contiguous")
        if _nbytes(scratch) < need:
            raise ValueError(f"scratch holds fewer than the {need} bytes needed")
    else:
        _need(grad_weight is None and grad_bias is None, "grad_weight and grad_bias need want_params")
    _check_current_device((("grad_y", grad_y), ("x", x), ("mean", mean), ("rstd", rstd), ("weight", weight),
                           ("out", out), ("grad_weight", grad_weight), ("grad_bias", grad_bias),
                           ("scratch", scratch)))
    nbytes = 0 if scratch is None else _nbytes(scratch)
    A.check(A.lib().moe_layer_norm_backward(T, H, _ROW_DT[x.dtype], _ROW_DT[grad_y.dtype], wdt, _ptr(grad_y), _ptr(x),
                                            _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(out), _ptr(grad_weight),
                                            _ptr(grad_bias), _ptr(scratch), nbytes, _stream()),
            "moe_layer_norm_backward")
    return out, grad_weight, grad_bias


class RmsNorm(NamedTuple):
    """What rms_norm gives; None where it was not asked for."""
    out: Optional[torch.Tensor]      # normalised rows [T,H]
    codes: Optional[torch.Tensor]    # the same as e4m3 codes [T,H] ...
    scales: Optional[torch.Tensor]   # ... with fp32 scales [T,H/128]
    total: Optional[torch.Tensor]    # x + residual [T,H]
    rstd: torch.Tensor               # [T] fp32


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
             residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
             want_rows: bool = True, quantize: bool = False, out: Optional[torch.Tensor] = None,
             codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
             total: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None) -> RmsNorm:
    """RMS norm of x + residual, rows [T,H] of bf16 or fp32 each (weight [H]
    likewise).  The normalised rows come as ``out`` (of ``out_dtype``, default
    x's; not with ``want_rows=False``), with ``quantize`` also or only as e4m3
    codes and scales, as a Dispatcher with fp8 payload takes them.  ``total``,
    of the residual's type, may be the residual itself (or x, where the types
    are the same); without a residual it is written only where it is given."""
    # a single token's call is bound by the host (4.1 us for the launch alone): what is in order is seen inline, the
    # helpers that put messages together are called where something is not (9.6 -> 8.7 us per call)
    shape = x.shape
    if len(shape) != 2 or x.dtype not in _ROW_DT or not x.is_contiguous():
        _need(x.dim() == 2, "x must be [T,H]")
        _check_rows(x, "x", shape, _ROW_DT)
    T, H = shape
    wdt = A.F32
    if weight is not None:
        if weight.dtype not in _ROW_DT or weight.shape != (H,) or not weight.is_contiguous():
            _check_rows(weight, "weight", (H,), _ROW_DT)
        wdt = _ROW_DT[weight.dtype]
    if residual is not None:
        if residual.dtype not in _ROW_DT or residual.shape != shape or not residual.is_contiguous():
            _check_rows(residual, "residual", shape, _ROW_DT)
        if total is None:
            total = torch.empty_like(residual)
        elif total is not residual and (total.dtype != residual.dtype or total.shape != shape
                                        or not total.is_contiguous()):
            _check_rows(total, "total", shape, (residual.dtype,))
    elif total is not None:
        _check_rows(total, "total", shape, _ROW_DT)
    if want_rows:
        if out is None:
            out = torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
        elif out.dtype not in _ROW_DT or out.shape != shape or not out.is_contiguous():
            _check_rows(out, "out", shape, _ROW_DT)
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out must be of out_dtype")
        ydt = _ROW_DT.get(out.dtype)
        _need(ydt is not None, "out must be bf16 or fp32")
    else:
        _need(quantize, "rms_norm without rows needs quantize")
        _need(out is None and out_dtype is None, "out and out_dtype need want_rows")
        ydt = A.BF16
    if quantize:
        if H % 128:
            raise ValueError(f"8-bit rows need a width that is a multiple of 128, got {H}")
        if codes is None:
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
        elif codes.dtype not in _FP8_DTYPES or codes.shape != shape or not codes.is_contiguous():
            _check_rows(codes, "codes", shape, _FP8_DTYPES)
        if scales is None:
            scales = torch.empty((T, H // 128), dtype=torch.float32, device=x.device)
        elif scales.dtype != torch.float32 or scales.shape != (T, H // 128) or not scales.is_contiguous():
            _check_rows(scales, "scales", (T, H // 128), _F32)
    else:
        _need(codes is None and scales is None, "codes and scales need quantize")
    if rstd is None:
        rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    elif rstd.dtype != torch.float32 or rstd.shape != (T,) or not rstd.is_contiguous():
        _check_rows(rstd, "rstd", (T,), _F32)
    here = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None     # a CPU tensor's is -1
    for t in (x, weight, residual, out, codes, scales, total, rstd):
        if t is not None and t.get_device() != here:
            _check_current_device((("x", x), ("weight", weight), ("residual", residual), ("out", out),
                                   ("codes", codes), ("scales", scales), ("total", total), ("rstd", rstd)))
    status = A.lib().moe_rms_norm(
        T, H, _ROW_DT[x.dtype], _ROW_DT[(x if total is None else total).dtype], ydt, wdt, x.data_ptr(),
        None if residual is None else residual.data_ptr(), None if weight is None else weight.data_ptr(), eps,
        None if out is None else out.data_ptr(), None if codes is None else codes.data_ptr(),
        None if scales is None else scales.data_ptr(), None if total is None else total.data_ptr(), rstd.data_ptr(),
        torch._C._cuda_getCurrentRawStream(here))
    if status:
        A.check(status, "moe_rms_norm")
    return RmsNorm(out, codes, scales, total, rstd)


def rms_norm_backward_scratch_bytes(T: int, H: int) -> int:
    return int(A.lib().moe_rms_norm_backward_scratch_bytes(int(T), int(H)))


def rms_norm_backward(grad_y: torch.Tensor, total: torch.Tensor, rstd: torch.Tensor,
                      weight: Optional[torch.Tensor] = None, *, grad_total: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, grad_weight: Optional[torch.Tensor] = None,
                      scratch: Optional[torch.Tensor] = None, want_weight: bool = True):
    """Gradients of an RMS norm: (grad [T,H] of total's dtype, grad_weight [H]
    fp32 or None without ``want_weight``).  ``total`` and ``rstd`` are the
    forward's (x where there was no residual).  ``grad`` is the gradient of x
    and of the residual alike; ``grad_total``, of total's dtype, is what
    reaches the sum along the residual stream and may be ``out``."""
    # checks inline as in rms_norm: two launches and 13 us of a small call on the host
    shape = total.shape
    if len(shape) != 2 or total.dtype not in _ROW_DT or not total.is_contiguous():
        _need(total.dim() == 2, "total must be [T,H]")
        _check_rows(total, "total", shape, _ROW_DT)
    T, H = shape
    if grad_y.dtype not in _ROW_DT or grad_y.shape != shape or not grad_y.is_contiguous():
        _check_rows(grad_y, "grad_y", shape, _ROW_DT)
    if rstd.dtype != torch.float32 or rstd.shape != (T,) or not rstd.is_contiguous():
        _check_rows(rstd, "rstd", (T,), _F32)
    wdt = A.F32
    if weight is not None:
        if weight.dtype not in _ROW_DT or weight.shape != (H,) or not weight.is_contiguous():
            _check_rows(weight, "weight", (H,), _ROW_DT)
        wdt = _ROW_DT[weight.dtype]
    same = (total.dtype,)
    if grad_total is not None and (grad_total.dtype not in same or grad_total.shape != shape
                                   or not grad_total.is_contiguous()):
        _check_rows(grad_total, "grad_total", shape, same)
    if out is None:
        out = torch.empty_like(total)
    elif out.dtype not in same or out.shape != shape or not out.is_contiguous():
        _check_rows(out, "out", shape, same)
    nbytes = 0
    if want_weight:
        if grad_weight is None:
            grad_weight = torch.empty(H, dtype=torch.float32, device=total.device)
        elif grad_weight.dtype != torch.float32 or grad_weight.shape != (H,) or not grad_weight.is_contiguous():
            _check_rows(grad_weight, "grad_weight", (H,), _F32)
        need = A.lib().moe_rms_norm_backward_scratch_bytes(T, H)
        if need == 0:
            raise ValueError(f"rows of {H} elements are outside 1..{A.NORM_MAX_H}")
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=total.device)
        elif not scratch.is_contiguous():
            raise ValueError("scratch must be contiguous")
        nbytes = _nbytes(scratch)
        if nbytes < need:
            raise ValueError(f"scratch holds fewer than the {need} bytes needed")
    else:
        _need(grad_weight is None, "grad_weight needs want_weight")
    here = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else None     # a CPU tensor's is -1
    for t in (grad_y, total, rstd, weight, grad_total, out, grad_weight, scratch):
        if t is not None and t.get_device() != here:
            _check_current_device((("grad_y", grad_y), ("total", total), ("rstd", rstd), ("weight", weight),
                                   ("grad_total", grad_total), ("out", out), ("grad_weight", grad_weight),
                                   ("scratch", scratch)))
    status = A.lib().moe_rms_norm_backward(
        T, H, _ROW_DT[total.dtype], _ROW_DT[grad_y.dtype], wdt, grad_y.data_ptr(), total.data_ptr(), rstd.data_ptr(),
        None if weight is None else weight.data_ptr(), None if grad_total is None else grad_total.data_ptr(),
        out.data_ptr(), None if grad_weight is None else grad_weight.data_ptr(),
        None if scratch is None else scratch.data_ptr(), nbytes, torch._C._cuda_getCurrentRawStream(here))
    if status:
        A.check(status, "moe_rms_norm_backward")
    return out, grad_weight


class Dispatcher:
    """One fixed-shape dispatch/MLP/combine problem with its workspace."""

    def __init__(self, T: int, H: int, E: int, K: int, *, route_fmt: str = "dense_i16",
                 payload: str = "bf16", pad_multiple: int = 1, capacity: Optional[int] = None,
                 out_rows: int = 0, device=None):
        L = A.lib()
        self.device = torch.device(device if device is not None else "cuda")
        self._cuda = self.device.type == "cuda"
        self._scratch_need = {}
        self.desc = make_desc(T, H, E, K, route_fmt, payload, pad_multiple, capacity, out_rows)
        ws_bytes = int(L.moe_workspace_bytes(C.byref(self.desc)))
        if ws_bytes == 0:
            raise A.MoeError(A.MOE_ESHAPE, "moe_workspace_bytes")
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device)
        self.h = A.MoeHandle()
        A.check(L.moe_handle_init(C.byref(self.desc), _ptr(self.ws), ws_bytes, C.byref(self.h)), "moe_handle_init")
        self.T, self.H, self.E, self.K = T, H, E, K
        self.R = int(self.h.desc.out_rows)
        self.route_fmt = self.desc.route_fmt
        self.payload = self.desc.payload
        self.tokens_per_expert = torch.empty(E, dtype=torch.int32, device=self.device)
        self.flag = torch.empty(1, dtype=torch.int32, device=self.device)

    # ---- views of the handle's device metadata ------------------------------
    def _view(self, field: str, dtype: torch.dtype, n: int) -> torch.Tensor:
        off = int(getattr(self.h, field)) - int(self.h.ws)
        nb = n * torch.empty(0, dtype=dtype).element_size()
        return self.ws[off:off + nb].view(dtype)

    @property
    def row_id(self):
        return self._view("row_id", torch.int32, self.T * self.K).view(self.T, self.K)

    @property
    def copy_prob(self):
        return self._view("copy_prob", torch.float32, self.T * self.K).view(self.T, self.K)

    @property
    def seg_off(self):
        return self._view("seg_off", torch.int64, self.E + 1)

    @property
    def kept(self):
        return self._view("kept", torch.int32, self.E)

    @property
    def src_row(self):
        return self._view("src_row", torch.int32, self.R)

    @property
    def rows_needed(self):
        return self._view("rows_needed", torch.int64, 1)

    # ---- checks ------------------------------------------------------------------
    def _dev(self, t: torch.Tensor, name: str):
        index = t.get_device()               # -1 on the CPU
        if not (self._cuda and index >= 0 and (index == self.device.index or index == torch._C._cuda_getDevice())
                or t.device == self.device):
            raise ValueError(f"{name} must live on {self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _check_here(self):
        # the workspace on the current GPU leaves _dev the current GPU alone to accept
        _check_current_device((("the Dispatcher's workspace", self.ws),))

    def _check_routing(self, routing, probs, T_live):
        self._dev(routing, "routing")
        if routing.dtype not in _FMT_DTYPES[self.route_fmt]:
            raise ValueError(f"routing dtype {routing.dtype} does not match the format")
        shape = self._routing_shape()
        if routing.shape != shape:
            raise ValueError(f"routing shape {tuple(routing.shape)} != {shape}")
        if probs is not None:
            self._dev(probs, "probs")
            _need(probs.dtype == torch.float32 and probs.shape == shape, "probs must be float32 shaped like routing")
        if T_live is not None:
            self._dev(T_live, "T_live")
            _need(T_live.dtype == torch.int32 and T_live.numel() == 1, "T_live must be one int32")

    # ---- gate --------------------------------------------------------------------
    def _routing_shape(self):
        return (self.T, self.E) if self.route_fmt == A.ROUTE_SPARSE_BOOL else (self.T, self.K)

    def _check_gate(self, logits, score):
        _check_rows(logits, "logits", (self.T, self.E), _ROW_DT)
        if score not in _SCORE:
            raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}")

    def _check_gate_options(self, bias=None, *, score="softmax", normalize=False, scale=1.0, routing=None, probs=None):
        """What gate() refuses of its keyword arguments, for calls that have no logits yet."""
        if score not in _SCORE:
            raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}")
        _need(math.isfinite(C.c_float(scale).value), "scale must be finite in fp32")
        shape = self._routing_shape()
        spans = []
        for name, t, want, dtypes in (("bias", bias, (self.E,), _F32), ("probs", probs, shape, _F32),
                                      ("routing", routing, shape, _FMT_DTYPES[self.route_fmt])):
            if t is not None:
                _check_rows(t, name, want, dtypes)
                if self._cuda:
                    _check_current_device(((name, t),))
                spans.append((t.data_ptr(), t.data_ptr() + _nbytes(t)))
        _need(all(a[1] <= b[0] or b[1] <= a[0] for i, a in enumerate(spans) for b in spans[:i]),
              "bias, routing and probs must not overlap")
        _check_aligned(routing=routing)

    def gate(self, logits: torch.Tensor, bias: Optional[torch.Tensor] = None, *, score: str = "softmax",
             normalize: bool = False, scale: float = 1.0, routing: Optional[torch.Tensor] = None,
             probs: Optional[torch.Tensor] = None):
        """The top-k experts of each token and their weights from router logits
        [T,E] (bf16 or fp32): (routing, probs) in this Dispatcher's routing
        format, as preprocess and dispatch take them.  ``bias`` [E] (fp32)
        steers the choice only; -inf logits switch experts off.  Logits and
        routing start at a multiple of 16 bytes."""
        self._check_gate(logits, score)
        if bias is not None:
            _check_rows(bias, "bias", (self.E,), _F32)
        shape = self._routing_shape()
        if routing is None:
            routing = torch.empty(shape, dtype=_ROUTING_OUT[self.route_fmt], device=self.device)
        else:
            _check_rows(routing, "routing", shape, _FMT_DTYPES[self.route_fmt])
        if probs is None:
            probs = torch.empty(shape, dtype=torch.float32, device=self.device)
        else:
            _check_rows(probs, "probs", shape, _F32)
        _check_current_device((("logits", logits), ("bias", bias), ("routing", routing), ("probs", probs)))
        A.check(A.lib().moe_gate(C.byref(self.h), _ptr(logits), _ROW_DT[logits.dtype], _ptr(bias), _SCORE[score],
                                 1 if normalize else 0, float(scale), _ptr(routing), _ptr(probs), _stream()),
                "moe_gate")
        return routing, probs

    def gate_backward(self, grad_probs: torch.Tensor, logits: torch.Tensor, routing: torch.Tensor, *,
                      score: str = "softmax", normalize: bool = False, scale: float = 1.0,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Gradient of the gate's weights (grad_probs, in the routing's shape,
        as combine_backward gives it) to the logits [T,E], in their dtype.
        ``out`` may be the logits."""
        self._check_gate(logits, score)
        shape = self._routing_shape()
        _check_rows(routing, "routing", shape, _FMT_DTYPES[self.route_fmt])
        _check_rows(grad_probs, "grad_probs", shape, _F32)
        if out is None:
            out = torch.empty_like(logits)
        else:
            _check_rows(out, "out", logits.shape, (logits.dtype,))
        _check_current_device((("grad_probs", grad_probs), ("logits", logits), ("routing", routing), ("out", out)))
        A.check(A.lib().moe_gate_backward(C.byref(self.h), _ptr(grad_probs), _ptr(logits), _ROW_DT[logits.dtype],
                                          _ptr(routing), _SCORE[score], 1 if normalize else 0, float(scale),
                                          _ptr(out), _stream()), "moe_gate_backward")
        return out

    # ---- calls -------------------------------------------------------------------
    def preprocess(self, routing: torch.Tensor, probs: Optional[torch.Tensor] = None,
                   T_live: Optional[torch.Tensor] = None, out_probs: Optional[torch.Tensor] = None):
        self._check_routing(routing, probs, T_live)
        if out_probs is not None:
            self._dev(out_probs, "out_probs")
            _need(out_probs.dtype == torch.float32 and out_probs.numel() >= self.R, "out_probs must hold R floats")
        A.check(A.lib().moe_route_preprocess(C.byref(self.h), _ptr(routing), _ptr(probs), _ptr(T_live),
                                             _ptr(self.tokens_per_expert), _ptr(out_probs), _ptr(self.flag),
                                             _stream()), "moe_route_preprocess")
        return self.tokens_per_expert, self.flag

    def _alloc_out(self, x, out, x_scales, out_scales):
        if out is None:
            out = torch.empty((self.R, self.H), dtype=x.dtype, device=self.device)
        self._dev(out, "out")
        _need((out.dtype == x.dtype or (x.dtype in _FP8_DTYPES and out.dtype in _FP8_DTYPES))
              and tuple(out.shape) == (self.R, self.H), "out must be [R,H] like x")
        if self.payload == A.FP8E4M3_B128:
            _need(x_scales is not None, "fp8 payload needs x_scales")
            self._dev(x_scales, "x_scales")
            _need(x_scales.dtype == torch.float32 and tuple(x_scales.shape) == (self.T, self.H // 128),
                  "x_scales must be float32 [T, H/128]")
            if out_scales is None:
                out_scales = torch.empty((self.R, self.H // 128), dtype=torch.float32, device=self.device)
            self._dev(out_scales, "out_scales")
            _need(out_scales.dtype == torch.float32 and tuple(out_scales.shape) == (self.R, self.H // 128),
                  "out_scales must be float32 [R, H/128]")
        return out, out_scales

    def _check_x(self, x):
        self._dev(x, "x")
        _need(tuple(x.shape) == (self.T, self.H), f"x shape {tuple(x.shape)} != {(self.T, self.H)}")
        if self.payload == A.BF16:
            _need(x.dtype == torch.bfloat16, "bf16 payload expects a bfloat16 x")
        else:
            _need(x.dtype in _FP8_DTYPES, "fp8 payload expects uint8 / float8_e4m3fn codes")

    def permute(self, x: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None):
        self._check_x(x)
        out, out_scales = self._alloc_out(x, out, x_scales, out_scales)
        A.check(A.lib().moe_permute(C.byref(self.h), _ptr(x), _ptr(x_scales), _ptr(out), _ptr(out_scales),
                                    _stream()), "moe_permute")
        return (out, out_scales) if self.payload == A.FP8E4M3_B128 else out

    def permute_quantize(self, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                         out_scales: Optional[torch.Tensor] = None):
        """Quantise-on-dispatch (handle with fp8 payload): bf16 token rows x
        [T,H] -> e4m3 codes [R,H] and 1x128 fp32 scales [R,H/128] at every
        kept copy's row.  Returns (codes, scales)."""
        _need(self.payload == A.FP8E4M3_B128, "quantise-on-dispatch needs a handle with fp8 payload")
        self._dev(x, "x")
        _need(x.dtype == torch.bfloat16 and tuple(x.shape) == (self.T, self.H), "x must be bf16 [T,H]")
        if out is None:
            out = torch.empty((self.R, self.H), dtype=torch.uint8, device=self.device)
        if out_scales is None:
            out_scales = torch.empty((self.R, self.H // 128), dtype=torch.float32, device=self.device)
        self._dev(out, "out")
        self._dev(out_scales, "out_scales")
        _need(out.dtype in _FP8_DTYPES and tuple(out.shape) == (self.R, self.H), "out must be e4m3 codes [R,H]")
        _need(out_scales.dtype == torch.float32 and tuple(out_scales.shape) == (self.R, self.H // 128),
              "out_scales must be float32 [R, H/128]")
        A.check(A.lib().moe_permute_quantize(C.byref(self.h), _ptr(x), _ptr(out), _ptr(out_scales), _stream()),
                "moe_permute_quantize")
        return out, out_scales

    def dispatch(self, x: torch.Tensor, routing: torch.Tensor, probs: Optional[torch.Tensor] = None, *,
                 x_scales=None, out=None, out_scales=None, out_probs=None, T_live=None):
        """preprocess + permute.  Returns (permuted, tokens_per_expert, flag,
        out_probs, out_scales); out_probs / out_scales are None unless given
        / fp8."""
        self._check_x(x)
        self._check_routing(routing, probs, T_live)
        out, out_scales = self._alloc_out(x, out, x_scales, out_scales)
        if out_probs is not None:
            self._dev(out_probs, "out_probs")
            _need(out_probs.dtype == torch.float32 and out_probs.numel() >= self.R, "out_probs must hold R floats")
        A.check(A.lib().moe_dispatch(C.byref(self.h), _ptr(routing), _ptr(probs), _ptr(T_live), _ptr(x),
                                     _ptr(x_scales), _ptr(out), _ptr(out_scales), _ptr(out_probs),
                                     _ptr(self.tokens_per_expert), _ptr(self.flag), _stream()), "moe_dispatch")
        return out, self.tokens_per_expert, self.flag, out_probs, out_scales

    def mlp_scratch_bytes(self, F: int, wdtype: str = "bf16") -> int:
        return int(A.lib().moe_mlp_scratch_bytes(C.byref(self.h), int(F), _DT[wdtype]))

    def alloc_mlp_scratch(self, F: int, wdtype: str = "bf16") -> torch.Tensor:
        n = self.mlp_scratch_bytes(F, wdtype)
        _need(n > 0, "invalid F / wdtype for the MLP scratch")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def _check_perm(self, perm, perm_scales):
        self._dev(perm, "perm")
        if self.payload == A.FP8E4M3_B128:
            _need(perm.dtype in _FP8_DTYPES and tuple(perm.shape) == (self.R, self.H),
                  "perm must be e4m3 codes [R,H] (quantised on dispatch)")
            _need(perm_scales is not None, "fp8 permuted rows need their scales")
            self._dev(perm_scales, "perm_scales")
            _need(perm_scales.dtype == torch.float32 and tuple(perm_scales.shape) == (self.R, self.H // 128),
                  "perm_scales must be float32 [R, H/128]")
        else:
            _need(perm.dtype == torch.bfloat16 and perm.shape == (self.R, self.H), "perm must be bf16 [R,H]")
            _need(perm_scales is None, "bf16 permuted rows take no scales")

    def _check_w1(self, w1: torch.Tensor, w1_scales: Optional[torch.Tensor]):
        """FC1 weights [E, 2F, H] (bf16, or e4m3 codes with [E, 2F/128, H/128]
        float32 block scales, or packed 4-bit codes [E, 2F, H/2] with
        [E, 2F, H/128] float32 scales) on this device; returns (F, wdtype)."""
        self._dev(w1, "w1")
        if self._is_int4(w1, w1_scales):
            experts, rows, packed = w1.shape
            if not (experts == self.E and 2 * packed == self.H and rows % 2 == 0 and rows > 0):
                raise ValueError(f"4-bit w1 must be [E, 2F, H/2] = [{self.E}, 2F, {self.H // 2}], "
                                 f"got {tuple(w1.shape)}")
            return rows // 2, self._check_int4(rows, 2 * packed, w1_scales, "w1")
        _need(w1.dim() == 3 and w1.shape[0] == self.E and w1.shape[2] == self.H and w1.shape[1] % 2 == 0
              and w1.shape[1] > 0, f"w1 must be [E, 2F, H] = [{self.E}, 2F, {self.H}], got {tuple(w1.shape)}")
        F = int(w1.shape[1]) // 2
        return F, self._check_wdtype(w1, w1_scales, "w1", (self.E, 2 * F // 128, self.H // 128))

    def _check_w2(self, w2: torch.Tensor, w2_scales: Optional[torch.Tensor]):
        """FC2 weights [E, H, F] (bf16, or e4m3 codes with [E, H/128, F/128]
        float32 block scales, or packed 4-bit codes [E, H, F/2] with
        [E, H, F/128] float32 scales) on this device; returns (F, wdtype)."""
        self._dev(w2, "w2")
        if self._is_int4(w2, w2_scales):
            experts, rows, packed = w2.shape
            if not (experts == self.E and rows == self.H and packed > 0):
                raise ValueError(f"4-bit w2 must be [E, H, F/2] = [{self.E}, {self.H}, F/2], got {tuple(w2.shape)}")
            return 2 * packed, self._check_int4(rows, 2 * packed, w2_scales, "w2")
        _need(w2.dim() == 3 and w2.shape[0] == self.E and w2.shape[1] == self.H and w2.shape[2] > 0,
              f"w2 must be [E, H, F] = [{self.E}, {self.H}, F], got {tuple(w2.shape)}")
        F = int(w2.shape[2])
        return F, self._check_wdtype(w2, w2_scales, "w2", (self.E, self.H // 128, F // 128))

    @staticmethod
    def _is_int4(w, scales) -> bool:
        """Byte weights are packed 4-bit codes where every weight row has its
        own scales; e4m3 codes share a scale among 128 rows."""
        return (w.dtype == torch.uint8 and w.dim() == 3 and scales is not None and scales.dim() == 3
                and scales.shape[1] == w.shape[1])

    def _check_int4(self, rows, cols, scales, name) -> str:
        if self.H % 128 or rows % 128 or cols % 128:
            raise ValueError(f"4-bit {name} needs dimensions that are multiples of 128")
        shape = (self.E, rows, cols // 128)
        self._dev(scales, name + "_scales")
        if scales.dtype != torch.float32 or scales.shape != shape:
            raise ValueError(f"{name}_scales must be float32 {shape}, got {scales.dtype} {tuple(scales.shape)}")
        return "int4"

    def _check_wdtype(self, w, scales, name, scale_shape):
        if w.dtype in _FP8_DTYPES:
            _need(self.H % 128 == 0 and w.shape[1] % 128 == 0 and w.shape[2] % 128 == 0,
                  f"fp8 {name} needs dimensions that are multiples of 128")
            _need(scales is not None, f"fp8 {name} needs its 128x128 block scales")
            self._dev(scales, f"{name}_scales")
            _need(scales.dtype == torch.float32 and tuple(scales.shape) == scale_shape,
                  f"{name}_scales must be float32 {scale_shape}, got {scales.dtype} {tuple(scales.shape)}")
            return "fp8"
        _need(w.dtype == torch.bfloat16, f"{name} must be bfloat16 or e4m3 codes, got {w.dtype}")
        _need(scales is None, f"bf16 {name} takes no block scales")
        return "bf16"

    def _check_scratch(self, scratch: torch.Tensor, F: int, wdtype: str):
        self._dev(scratch, "scratch")
        need = self._scratch_need.get((F, wdtype))      # a function of the fixed shape alone
        if need is None:
            need = self._scratch_need[F, wdtype] = self.mlp_scratch_bytes(F, wdtype)
        if need <= 0:
            raise ValueError(f"invalid FFN width {F} for {wdtype} weights")
        if _nbytes(scratch) < need:
            raise ValueError(f"scratch holds fewer than the {need} bytes needed")

    def _check_expert_out(self, out: torch.Tensor):
        self._dev(out, "out")
        if out.dtype != torch.bfloat16 or out.shape != (self.R, self.H):
            raise ValueError(f"out must be bf16 [R, H] = [{self.R}, {self.H}]")

    def grouped_mlp(self, perm: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, *,
                    w1_scales: Optional[torch.Tensor] = None, w2_scales: Optional[torch.Tensor] = None,
                    scratch: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    perm_scales: Optional[torch.Tensor] = None):
        """Grouped SwiGLU MLP over the permuted rows.  w1 [E,2F,H], w2 [E,H,F]
        (bf16, or e4m3 codes with 128x128 block scales, or packed 4-bit codes
        w1 [E,2F,H/2], w2 [E,H,F/2] with scales [E,2F,H/128], [E,H,F/128]: see
        _check_w1).  With 4-bit weights, rows of ``out`` that hold no kept copy
        are left as they were.  With a handle of fp8 payload, perm is e4m3
        codes quantised on dispatch plus perm_scales (fp8 weights only)."""
        F, wdtype = self._check_w1(w1, w1_scales)
        F2, wdtype2 = self._check_w2(w2, w2_scales)
        _need(F2 == F and wdtype2 == wdtype, "w1 and w2 must share the FFN width and dtype")
        self._check_perm(perm, perm_scales)
        if scratch is None:
            scratch = self.alloc_mlp_scratch(F, wdtype)
        self._check_scratch(scratch, F, wdtype)
        if out is None:
            out = torch.empty((self.R, self.H), dtype=torch.bfloat16, device=self.device)
        self._check_expert_out(out)
        if wdtype == "int4":
            self._check_here()
        A.check(A.lib().moe_grouped_swiglu_mlp(C.byref(self.h), F, _DT[wdtype], _ptr(perm), _ptr(perm_scales), _ptr(w1),
                                               _ptr(w1_scales), _ptr(w2), _ptr(w2_scales), _ptr(scratch),
                                               _nbytes(scratch), _ptr(out), _stream()),
                "moe_grouped_swiglu_mlp")
        return out

    def grouped_mlp_noalloc(self, perm: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, *,
                            w1_scales: Optional[torch.Tensor] = None, w2_scales: Optional[torch.Tensor] = None,
                            out: torch.Tensor, perm_scales: Optional[torch.Tensor] = None):
        """grouped_mlp without a scratch argument and without any allocation:
        the activations live in the library's fixed device array
        (A.NOALLOC_SCRATCH_BYTES per GPU, shared by every call on that GPU).
        ``out`` is required."""
        F, wdtype = self._check_w1(w1, w1_scales)
        F2, wdtype2 = self._check_w2(w2, w2_scales)
        _need(F2 == F and wdtype2 == wdtype, "w1 and w2 must share the FFN width and dtype")
        self._check_perm(perm, perm_scales)
        self._check_expert_out(out)
        if wdtype == "int4":
            self._check_here()
        A.check(A.lib().moe_grouped_swiglu_mlp_noalloc(C.byref(self.h), F, _DT[wdtype], _ptr(perm), _ptr(perm_scales),
                                                       _ptr(w1), _ptr(w1_scales), _ptr(w2), _ptr(w2_scales), _ptr(out),
                                                       _stream()), "moe_grouped_swiglu_mlp_noalloc")
        return out

    def fc1(self, perm: torch.Tensor, w1: torch.Tensor, scratch: torch.Tensor, w1_scales=None,
            perm_scales=None) -> None:
        """FC1 + SwiGLU of every kept row into ``scratch`` (the first half of
        grouped_mlp).  The FFN width and weight dtype are remembered: fc2 on
        this scratch must use the same."""
        F, wdtype = self._check_w1(w1, w1_scales)
        self._check_perm(perm, perm_scales)
        self._check_scratch(scratch, F, wdtype)
        if wdtype == "int4":
            self._check_here()
        A.check(A.lib().moe_grouped_fc1_swiglu(C.byref(self.h), F, _DT[wdtype], _ptr(perm), _ptr(perm_scales), _ptr(w1),
                                               _ptr(w1_scales), _ptr(scratch), _nbytes(scratch), _stream()),
                "moe_grouped_fc1_swiglu")
        self._fc1_done = (F, wdtype, scratch.data_ptr())

    def _check_after_fc1(self, F: int, wdtype: str, scratch: torch.Tensor):
        prev = getattr(self, "_fc1_done", None)
        _need(prev is not None, "fc2 needs an fc1 on this Dispatcher first")
        _need(prev == (F, wdtype, scratch.data_ptr()),
              f"fc2 with FFN width {F} ({wdtype}) on scratch {scratch.data_ptr():#x} does not match the last fc1 "
              f"(width {prev[0]} ({prev[1]}) on scratch {prev[2]:#x})")

    def fc2(self, w2: torch.Tensor, scratch: torch.Tensor, out: torch.Tensor, w2_scales=None) -> torch.Tensor:
        """FC2 from ``scratch`` into the caller-owned ``out`` (the second half
        of grouped_mlp)."""
        F, wdtype = self._check_w2(w2, w2_scales)
        self._check_scratch(scratch, F, wdtype)
        self._check_after_fc1(F, wdtype, scratch)
        self._check_expert_out(out)
        if wdtype == "int4":
            self._check_here()
        A.check(A.lib().moe_grouped_fc2(C.byref(self.h), F, _DT[wdtype], _ptr(w2), _ptr(w2_scales), _ptr(scratch),
                                        _nbytes(scratch), _ptr(out), _stream()), "moe_grouped_fc2")
        return out

    def fc2_fp8out(self, w2: torch.Tensor, scratch: torch.Tensor, out: Optional[torch.Tensor] = None,
                   out_scales: Optional[torch.Tensor] = None):
        """FC2 (bf16 weights) into the fp8 combine format: returns (codes
        [R,H] uint8, scales [R,H/128] float32)."""
        F, wdtype = self._check_w2(w2, None)
        _need(wdtype == "bf16", "the fp8 combine format is written from bf16 weights")
        self._check_scratch(scratch, F, wdtype)
        self._check_after_fc1(F, wdtype, scratch)
        if out is None:
            out = torch.empty((self.R, self.H), dtype=torch.uint8, device=self.device)
        if out_scales is None:
            out_scales = torch.empty((self.R, self.H // 128), dtype=torch.float32, device=self.device)
        self._dev(out, "out")
        self._dev(out_scales, "out_scales")
        _need(out.dtype in _FP8_DTYPES and tuple(out.shape) == (self.R, self.H), "out must be e4m3 codes [R,H]")
        _need(out_scales.dtype == torch.float32 and tuple(out_scales.shape) == (self.R, self.H // 128),
              "out_scales must be float32 [R, H/128]")
        A.check(A.lib().moe_grouped_fc2_fp8out(C.byref(self.h), F, A.BF16, _ptr(w2), None, _ptr(scratch),
                                               _nbytes(scratch), _ptr(out), _ptr(out_scales), _stream()),
                "moe_grouped_fc2_fp8out")
        return out, out_scales

    def combine_fp8(self, expert_out_q: torch.Tensor, expert_out_scales: torch.Tensor, apply_probs: bool = True,
                    out: Optional[torch.Tensor] = None):
        """Combine from fp8 expert-output rows (codes [R,H], scales [R,H/128])."""
        self._dev(expert_out_q, "expert_out_q")
        self._dev(expert_out_scales, "expert_out_scales")
        _need(expert_out_q.dtype in _FP8_DTYPES and tuple(expert_out_q.shape) == (self.R, self.H),
              "expert_out_q must be e4m3 codes [R,H]")
        _need(expert_out_scales.dtype == torch.float32 and tuple(expert_out_scales.shape) == (self.R, self.H // 128),
              "expert_out_scales must be float32 [R, H/128]")
        if out is None:
            out = torch.empty((self.T, self.H), dtype=torch.bfloat16, device=self.device)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.T, self.H), "out must be bf16 [T,H]")
        A.check(A.lib().moe_combine_fp8(C.byref(self.h), _ptr(expert_out_q), _ptr(expert_out_scales),
                                        1 if apply_probs else 0, _ptr(out), _stream()), "moe_combine_fp8")
        return out

    def combine(self, expert_out: torch.Tensor, apply_probs: bool = True, out: Optional[torch.Tensor] = None):
        self._dev(expert_out, "expert_out")
        _need(expert_out.dtype == torch.bfloat16 and tuple(expert_out.shape) == (self.R, self.H),
              "expert_out must be bf16 [R,H]")
        if out is None:
            out = torch.empty((self.T, self.H), dtype=torch.bfloat16, device=self.device)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.T, self.H), "out must be bf16 [T,H]")
        A.check(A.lib().moe_combine(C.byref(self.h), _ptr(expert_out), 1 if apply_probs else 0, _ptr(out),
                                    _stream()), "moe_combine")
        return out

    # ---- backward ---------------------------------------------------------------
    def _probs_grad_shape(self):
        return (self.T, self.E) if self.route_fmt == A.ROUTE_SPARSE_BOOL else (self.T, self.K)

    def _grad_probs_out(self, grad_probs):
        if grad_probs is None:
            grad_probs = torch.empty(self._probs_grad_shape(), dtype=torch.float32, device=self.device)
        self._dev(grad_probs, "grad_probs")
        _need(grad_probs.dtype == torch.float32 and tuple(grad_probs.shape) == self._probs_grad_shape(),
              "grad_probs must be float32 in the routing's shape")
        return grad_probs

    def dispatch_backward(self, grad_out: torch.Tensor, grad_out_probs: Optional[torch.Tensor] = None, *,
                          out: Optional[torch.Tensor] = None, grad_probs: Optional[torch.Tensor] = None):
        """Gradients of a dispatch: (grad_x [T,H] bf16, grad_probs or None).
        grad_probs (routing-shaped fp32) is produced when grad_out_probs [R]
        is given."""
        self._dev(grad_out, "grad_out")
        _need(grad_out.dtype == torch.bfloat16 and tuple(grad_out.shape) == (self.R, self.H),
              "grad_out must be bf16 [R,H]")
        if out is None:
            out = torch.empty((self.T, self.H), dtype=torch.bfloat16, device=self.device)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.T, self.H), "out must be bf16 [T,H]")
        if grad_out_probs is not None:
            self._dev(grad_out_probs, "grad_out_probs")
            _need(grad_out_probs.dtype == torch.float32 and grad_out_probs.numel() >= self.R,
                  "grad_out_probs must hold R floats")
            grad_probs = self._grad_probs_out(grad_probs)
        else:
            _need(grad_probs is None, "grad_probs needs grad_out_probs")
        A.check(A.lib().moe_dispatch_backward(C.byref(self.h), _ptr(grad_out), _ptr(grad_out_probs), _ptr(out),
                                              _ptr(grad_probs), _stream()), "moe_dispatch_backward")
        return out, grad_probs

    def combine_backward(self, grad_y: torch.Tensor, expert_out: Optional[torch.Tensor] = None,
                         apply_probs: bool = True, *, out: Optional[torch.Tensor] = None,
                         grad_probs: Optional[torch.Tensor] = None, want_probs: bool = True):
        """Gradients of a combine: (grad_expert_out [R,H] bf16, grad_probs or
        None).  The probability gradient needs the forward's expert_out."""
        self._dev(grad_y, "grad_y")
        _need(grad_y.dtype == torch.bfloat16 and tuple(grad_y.shape) == (self.T, self.H), "grad_y must be bf16 [T,H]")
        if out is None:
            out = torch.empty((self.R, self.H), dtype=torch.bfloat16, device=self.device)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.R, self.H), "out must be bf16 [R,H]")
        if expert_out is not None:
            self._dev(expert_out, "expert_out")
            _need(expert_out.dtype == torch.bfloat16 and tuple(expert_out.shape) == (self.R, self.H),
                  "expert_out must be bf16 [R,H]")
        if want_probs or grad_probs is not None:
            _need(expert_out is not None or not apply_probs, "the probability gradient needs expert_out")
            grad_probs = self._grad_probs_out(grad_probs)
        A.check(A.lib().moe_combine_backward(C.byref(self.h), _ptr(grad_y), _ptr(expert_out), 1 if apply_probs else 0,
                                             _ptr(out), _ptr(grad_probs), _stream()), "moe_combine_backward")
        return out, grad_probs

    # ---- expert products of a training step --------------------------------------
    def _check_expert_weight(self, w, name, shape=None):
        if w.dtype != torch.bfloat16 or w.dim() != 3 or w.shape[0] != self.E or (shape and w.shape != shape):
            want = list(shape) if shape else f"[{self.E}, N, M]"
            raise ValueError(f"{name} must be bf16 {want}, got {w.dtype} {list(w.shape)}")
        if not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def grouped_product(self, rows: torch.Tensor, w: torch.Tensor, *, transpose: bool = False,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The product of every kept row with its expert's weight w [E,N,M]
        (bf16, N and M multiples of 8): rows [R,M] -> out [R,N], or with
        ``transpose`` rows [R,N] -> out [R,M], the gradient of the former to
        its rows.  Rows of ``out`` that hold no kept copy are left as they
        were."""
        self._check_expert_weight(w, "w")
        N, M = w.shape[1:]
        cols, width = (N, M) if transpose else (M, N)
        _check_rows(rows, "rows", (self.R, cols), _BF16)
        if out is None:
            out = torch.empty((self.R, width), dtype=torch.bfloat16, device=self.device)
        _check_rows(out, "out", (self.R, width), _BF16)
        _check_current_device((("the Dispatcher's workspace", self.ws), ("rows", rows), ("w", w), ("out", out)))
        A.check(A.lib().moe_grouped_product(C.byref(self.h), N, M, 1 if transpose else 0, _ptr(rows), _ptr(w),
                                            _ptr(out), _stream()), "moe_grouped_product")
        return out

    def grouped_weight_grad(self, grad: torch.Tensor, rows: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                            out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False) -> torch.Tensor:
        """The gradient of grouped_product to its weights: out [E,N,M] (bf16 or
        fp32) = sum over an expert's kept rows of grad [R,N] times rows [R,M],
        zeros for an expert without rows; with ``accumulate`` added to
        ``out``."""
        _need(grad.dim() == 2 and rows.dim() == 2, "grad and rows must be [R,N] and [R,M]")
        N, M = grad.shape[1], rows.shape[1]
        _check_rows(grad, "grad", (self.R, N), _BF16)
        _check_rows(rows, "rows", (self.R, M), _BF16)
        _need(out is not None or not accumulate, "accumulate needs out")
        if out is None:
            out = torch.empty((self.E, N, M), dtype=out_dtype, device=self.device)
        _check_rows(out, "out", (self.E, N, M), _ROW_DT)
        _check_current_device((("the Dispatcher's workspace", self.ws), ("grad", grad), ("rows", rows), ("out", out)))
        A.check(A.lib().moe_grouped_weight_grad(C.byref(self.h), N, M, _ROW_DT[out.dtype], 1 if accumulate else 0,
                                                _ptr(grad), _ptr(rows), _ptr(out), _stream()),
                "moe_grouped_weight_grad")
        return out

    def grouped_mlp_keep(self, perm: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, *,
                         h: Optional[torch.Tensor] = None, scratch: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None):
        """grouped_mlp with bf16 weights (H and F multiples of 8) for a training
        step: (out [R,H], h [R,2F]), with h, FC1's pre-activations, for
        grouped_mlp_backward.  The activations are rounded to bf16 once between
        the two products, as in grouped_mlp.  ``scratch`` is grouped_mlp's."""
        F = self._check_mlp_pair(w1, w2)
        _check_rows(perm, "perm", (self.R, self.H), _BF16)
        if h is None:
            h = torch.empty((self.R, 2 * F), dtype=torch.bfloat16, device=self.device)
        if out is None:
            out = torch.empty((self.R, self.H), dtype=torch.bfloat16, device=self.device)
        if scratch is None:
            scratch = self.alloc_mlp_scratch(F)
        _check_rows(h, "h", (self.R, 2 * F), _BF16)
        _check_rows(out, "out", (self.R, self.H), _BF16)
        self._check_scratch(scratch, F, "bf16")
        _check_current_device((("the Dispatcher's workspace", self.ws), ("perm", perm), ("w1", w1), ("w2", w2),
                               ("h", h), ("out", out), ("scratch", scratch)))
        A.check(A.lib().moe_grouped_mlp_keep(C.byref(self.h), F, _ptr(perm), _ptr(w1), _ptr(w2), _ptr(scratch),
                                             _nbytes(scratch), _ptr(h), _ptr(out), _stream()), "moe_grouped_mlp_keep")
        return out, h

    def _check_mlp_pair(self, w1, w2) -> int:
        self._check_expert_weight(w1, "w1")
        F = w1.shape[1] // 2
        self._check_expert_weight(w1, "w1", (self.E, 2 * F, self.H))
        self._check_expert_weight(w2, "w2", (self.E, self.H, F))
        return F

    def mlp_backward_scratch_bytes(self, F: int) -> int:
        return int(A.lib().moe_mlp_backward_scratch_bytes(C.byref(self.h), int(F)))

    def alloc_mlp_backward_scratch(self, F: int) -> torch.Tensor:
        n = self.mlp_backward_scratch_bytes(F)
        _need(n > 0, "the FFN width must be a multiple of 8")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def grouped_mlp_backward(self, grad_out: torch.Tensor, perm: torch.Tensor, h: torch.Tensor, w1: torch.Tensor,
                             w2: torch.Tensor, *, grad_perm: Optional[torch.Tensor] = None,
                             grad_w1: Optional[torch.Tensor] = None, grad_w2: Optional[torch.Tensor] = None,
                             grad_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
                             want_rows: bool = True, want_weights: bool = True,
                             scratch: Optional[torch.Tensor] = None):
        """Gradients of grouped_mlp_keep from that of its output (as
        combine_backward gives it): (grad_perm [R,H], as dispatch_backward
        takes it, grad_w1, grad_w2), the last two of ``grad_dtype`` (bf16 or
        fp32) or of the type of the tensors given; with ``accumulate`` they are
        added to those.  None without ``want_rows`` / ``want_weights``.  The
        activations and h's gradient, operands of the three products, are
        rounded to bf16 once, whatever the type of the gradients."""
        F = self._check_mlp_pair(w1, w2)
        _check_rows(grad_out, "grad_out", (self.R, self.H), _BF16)
        _check_rows(perm, "perm", (self.R, self.H), _BF16)
        _check_rows(h, "h", (self.R, 2 * F), _BF16)
        if want_rows:
            if grad_perm is None:
                grad_perm = torch.empty((self.R, self.H), dtype=torch.bfloat16, device=self.device)
            _check_rows(grad_perm, "grad_perm", (self.R, self.H), _BF16)
        else:
            _need(grad_perm is None, "grad_perm needs want_rows")
        if want_weights:
            _need(not accumulate or (grad_w1 is not None and grad_w2 is not None),
                  "accumulate needs grad_w1 and grad_w2")
            if grad_w1 is None:
                grad_w1 = torch.empty(w1.shape, dtype=grad_dtype if grad_w2 is None else grad_w2.dtype,
                                      device=self.device)
            if grad_w2 is None:
                grad_w2 = torch.empty(w2.shape, dtype=grad_w1.dtype, device=self.device)
            _check_rows(grad_w1, "grad_w1", w1.shape, _ROW_DT)
            _check_rows(grad_w2, "grad_w2", w2.shape, (grad_w1.dtype,))
        else:
            _need(grad_w1 is None and grad_w2 is None and not accumulate,
                  "grad_w1, grad_w2 and accumulate need want_weights")
        if scratch is None:
            scratch = self.alloc_mlp_backward_scratch(F)
        _need(scratch.is_contiguous(), "scratch must be contiguous")
        need = self._scratch_need.get((F, "backward"))
        if need is None:
            need = self._scratch_need[F, "backward"] = self.mlp_backward_scratch_bytes(F)
        if need <= 0:
            raise ValueError(f"invalid FFN width {F}")
        if _nbytes(scratch) < need:
            raise ValueError(f"scratch holds fewer than the {need} bytes needed")
        _check_current_device((("the Dispatcher's workspace", self.ws), ("grad_out", grad_out), ("perm", perm),
                               ("h", h), ("w1", w1), ("w2", w2), ("grad_perm", grad_perm), ("grad_w1", grad_w1),
                               ("grad_w2", grad_w2), ("scratch", scratch)))
        A.check(A.lib().moe_grouped_mlp_backward(C.byref(self.h), F,
                                                 A.BF16 if grad_w1 is None else _ROW_DT[grad_w1.dtype],
                                                 1 if accumulate else 0, _ptr(grad_out), _ptr(perm), _ptr(h), _ptr(w1),
                                                 _ptr(w2), _ptr(scratch), _nbytes(scratch), _ptr(grad_perm),
                                                 _ptr(grad_w1), _ptr(grad_w2), _stream()), "moe_grouped_mlp_backward")
        return grad_perm, grad_w1, grad_w2

    def decode_layer_scratch_bytes(self, F: int) -> int:
        return int(A.lib().moe_decode_layer_scratch_bytes(C.byref(self.h), int(F)))

    def decode_layer_fp8(self, x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, w1_scales: torch.Tensor,
                         w2_scales: torch.Tensor, *, scratch: torch.Tensor, expert_out: torch.Tensor,
                         out: torch.Tensor, status: torch.Tensor, apply_probs: bool = True) -> torch.Tensor:
        """The rest of the layer after preprocess(), as one persistent kernel:
        quantise-on-dispatch, FC1 + SwiGLU, activation quantiser, FC2 into
        ``expert_out`` and the combine into ``out``, with fp8 weights.
        ``status`` (one int32 on the device): the call clears bits 0 and 1
        and keeps bit 2, the caller's abort request (every wait returns at
        once).  Afterwards bit 0 means a wait ran past its bound and bit 1 a
        workgroup on an XCD numbered 8 or more; with any bit set the outputs
        are unspecified."""
        _need(self.payload == A.BF16, "the decode layer takes bf16 token rows")
        self._check_x(x)
        F, wdtype = self._check_w1(w1, w1_scales)
        F2, wdtype2 = self._check_w2(w2, w2_scales)
        _need(wdtype == "fp8" and wdtype2 == "fp8" and F2 == F, "the decode layer takes fp8 w1 and w2 of one FFN width")
        self._dev(scratch, "scratch")
        need = self.decode_layer_scratch_bytes(F)
        _need(need > 0 and _nbytes(scratch) >= need,
              f"scratch holds fewer than the {need} bytes needed")
        self._check_expert_out(expert_out)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.T, self.H), "out must be bf16 [T,H]")
        self._dev(status, "status")
        _need(status.dtype == torch.int32 and status.numel() == 1, "status must be one int32")
        A.check(A.lib().moe_decode_layer_fp8(C.byref(self.h), F, _ptr(x), _ptr(w1), _ptr(w1_scales), _ptr(w2),
                                             _ptr(w2_scales), _ptr(scratch), _nbytes(scratch), _ptr(expert_out),
                                             1 if apply_probs else 0, _ptr(out), _ptr(status), _stream()),
                "moe_decode_layer_fp8")
        return out

    def decode_fused_scratch_bytes(self, F: int) -> int:
        return int(A.lib().moe_decode_fused_scratch_bytes(C.byref(self.h), int(F)))

    def decode_fused_fp8(self, x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, w1_scales: torch.Tensor,
                         w2_scales: torch.Tensor, *, scratch: torch.Tensor, expert_out: torch.Tensor,
                         out: torch.Tensor, apply_probs: bool = True) -> torch.Tensor:
        """The rest of the layer after preprocess(), with fp8 weights, in two
        launches: quantise-on-dispatch, then one persistent kernel for FC1 +
        SwiGLU, the activation blocks, FC2 into ``expert_out`` and the combine
        into ``out``."""
        _need(self.payload == A.BF16, "the decode layer takes bf16 token rows")
        self._check_x(x)
        F, wdtype = self._check_w1(w1, w1_scales)
        F2, wdtype2 = self._check_w2(w2, w2_scales)
        _need(wdtype == "fp8" and wdtype2 == "fp8" and F2 == F, "the decode layer takes fp8 w1 and w2 of one FFN width")
        self._dev(scratch, "scratch")
        need = self.decode_fused_scratch_bytes(F)
        _need(need > 0, "the fused decode layer needs H, F multiples of 128 and H <= 8192")
        _need(_nbytes(scratch) >= need, f"scratch holds fewer than the {need} bytes needed")
        self._check_expert_out(expert_out)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.T, self.H), "out must be bf16 [T,H]")
        A.check(A.lib().moe_decode_fused_fp8(C.byref(self.h), F, _ptr(x), _ptr(w1), _ptr(w1_scales), _ptr(w2),
                                             _ptr(w2_scales), _ptr(scratch), _nbytes(scratch),
                                             _ptr(expert_out), 1 if apply_probs else 0, _ptr(out), _stream()),
                "moe_decode_fused_fp8")
        return out

    def _check_layer(self, x, routing, probs, w1, w2, w1_scales, w2_scales, T_live, router, gate, perm, perm_scales,
                     scratch, expert_out, out):
        """Whatever the layer's steps behind the norm check that does not wait
        for the router's logits.  Returns the five buffers, those that the
        caller omits allocated."""
        _need(tuple(x.shape) == (self.T, self.H), f"x shape {tuple(x.shape)} != {(self.T, self.H)}")
        if router is not None:
            self._check_gate_options(**(gate or {}))
            if T_live is not None:
                self._dev(T_live, "T_live")
                _need(T_live.dtype == torch.int32 and T_live.numel() == 1, "T_live must be one int32")
        else:
            _need(routing is not None, "the layer needs routing or a router")
            self._check_routing(routing, probs, T_live)
            _check_aligned(routing=routing)
        F, wdtype = self._check_w1(w1, w1_scales)
        F2, wdtype2 = self._check_w2(w2, w2_scales)
        _need(F2 == F and wdtype2 == wdtype, "w1 and w2 must share the FFN width and dtype")
        if wdtype == "bf16":
            _need(self.H % 256 == 0 and F % 128 == 0, "bf16 weights need H % 256 == 0 and F % 128 == 0")
        elif wdtype == "int4":
            self._check_here()
        fp8 = self.payload == A.FP8E4M3_B128
        _need(not fp8 or wdtype == "fp8", "e4m3 rows need fp8 weights")
        if perm is None:
            perm = torch.empty((self.R, self.H), dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16,
                               device=self.device)
        if fp8 and perm_scales is None:
            perm_scales = torch.empty((self.R, self.H // 128), dtype=torch.float32, device=self.device)
        self._check_perm(perm, perm_scales)
        if scratch is None:
            scratch = self.alloc_mlp_scratch(F, wdtype)
        self._check_scratch(scratch, F, wdtype)
        if expert_out is None:
            expert_out = torch.empty((self.R, self.H), dtype=torch.bfloat16, device=self.device)
        self._check_expert_out(expert_out)
        if out is None:
            out = torch.empty((self.T, self.H), dtype=torch.bfloat16, device=self.device)
        self._dev(out, "out")
        _need(out.dtype == torch.bfloat16 and tuple(out.shape) == (self.T, self.H), "out must be bf16 [T,H]")
        _check_aligned(w1=w1, w2=w2, perm=perm, scratch=scratch, expert_out=expert_out, out=out)
        return perm, perm_scales, scratch, expert_out, out

    def layer(self, x, routing, probs, w1, w2, *, perm=None, perm_scales=None, scratch=None, expert_out=None,
              out=None, w1_scales=None, w2_scales=None, T_live=None, apply_probs=True, check_overflow=False,
              norm=None, router=None, gate=None, rms=None, residual=None):
        """dispatch -> grouped MLP -> combine on the current stream.  With
        ``norm`` = (weight, bias) or (weight, bias, eps), the layer reads
        layer_norm(x) in bf16 in place of x.  With ``rms`` = (weight,) or
        (weight, eps), it reads rms_norm(x + residual), and ``residual`` (if
        given) becomes x + residual in every row, those from T_live on among
        them; with a handle of fp8 payload the norm writes the codes that the
        dispatch takes, and bf16 rows for the router alone.  A call that is
        refused leaves ``residual`` as it was, unless it is refused for what
        the router raised or returned: the router reads the norm's rows, and
        the sum has been written with them.  With ``router``, a callable that takes the
        rows the layer reads and returns their logits [T,E], routing and probs
        (None then) are ``self.gate`` of those logits, with the keyword
        arguments ``gate`` (bias, score, normalize, scale).  With a
        handle of fp8 payload and bf16 tokens, dispatch quantises on the way
        (routing metadata, then moe_permute_quantize into e4m3 rows ``perm``
        with 1x128 scales ``perm_scales``).  With ``check_overflow``, a
        device-side assert on the overflow flag is enqueued after the combine
        (no host wait; capturable).  Buffers the caller omits are allocated
        per call."""
        _need(router is not None or gate is None, "gate needs a router")
        _need(norm is None or rms is None, "norm and rms exclude each other")
        _need(rms is not None or residual is None, "residual needs rms")
        _need(router is None or (routing is None and probs is None), "routing and probs come from the router's logits")
        x_scales = None
        if norm is not None:
            x, _, _ = layer_norm(x, *norm, out_dtype=torch.bfloat16)
        elif rms is not None:
            if residual is not None:
                perm, perm_scales, scratch, expert_out, out = self._check_layer(
                    x, routing, probs, w1, w2, w1_scales, w2_scales, T_live, router, gate, perm, perm_scales, scratch,
                    expert_out, out)
            fp8 = self.payload == A.FP8E4M3_B128
            rows = router is not None or not fp8
            normed = rms_norm(x, *rms, residual=residual, total=residual, want_rows=rows, quantize=fp8,
                              out_dtype=torch.bfloat16 if rows else None)
            x, x_scales = (normed.codes, normed.scales) if fp8 else (normed.out, None)
        if router is not None:
            routing, probs = self.gate(router(x if x_scales is None else normed.out), **(gate or {}))
        if self.payload == A.FP8E4M3_B128 and x.dtype == torch.bfloat16:
            _, flag = self.preprocess(routing, probs, T_live)
            perm, perm_scales = self.permute_quantize(x, out=perm, out_scales=perm_scales)
        else:
            perm, _, flag, _, perm_scales = self.dispatch(x, routing, probs, x_scales=x_scales, out=perm,
                                                          out_scales=perm_scales, T_live=T_live)
        y = self.grouped_mlp(perm, w1, w2, w1_scales=w1_scales, w2_scales=w2_scales, scratch=scratch,
                             out=expert_out, perm_scales=perm_scales)
        y = self.combine(y, apply_probs=apply_probs, out=out)
        if check_overflow:
            assert_no_overflow(flag)
        return y


class BufferRing:
    """Caller-owned ring of persistent device slots (dispatch outputs, FC2
    outputs): ``acquire`` hands the next slot to a producer on the current
    stream, which first waits on the device for the slot's last release;
    ``release`` marks the final consumer's use on its stream.  Reuse before
    release raises (MOE_EBUSY), as does a second release (MOE_ESTATE).  The
    storage is one torch allocation made here; the library only carves it."""

    def __init__(self, n_slots: int, shape, dtype: torch.dtype, device=None):
        self.device = torch.device(device if device is not None else "cuda")
        self.shape = tuple(shape)
        self.dtype = dtype
        n = 1
        for v in self.shape:
            n *= int(v)
        self.nbytes = n * torch.empty(0, dtype=dtype).element_size()
        self.slot_bytes = (self.nbytes + 255) // 256 * 256
        self.storage = torch.empty(n_slots * self.slot_bytes, dtype=torch.uint8, device=self.device)
        self.r = A.MoeRing()
        A.check(A.lib().moe_ring_init(C.byref(self.r), _ptr(self.storage), self.slot_bytes, int(n_slots)),
                "moe_ring_init")
        self.n_slots = n_slots

    def acquire(self, stream=None):
        """(slot index, tensor view of the slot) for a producer on ``stream``
        (default: the current stream)."""
        st = C.c_void_p((stream or torch.cuda.current_stream()).cuda_stream)
        ptr = C.c_void_p()
        idx = C.c_int32()
        A.check(A.lib().moe_ring_acquire(C.byref(self.r), st, C.byref(ptr), C.byref(idx)), "moe_ring_acquire")
        off = int(idx.value) * self.slot_bytes
        view = self.storage[off:off + self.nbytes].view(self.dtype).view(self.shape)
        return int(idx.value), view

    def release(self, slot: int, stream=None):
        st = C.c_void_p((stream or torch.cuda.current_stream()).cuda_stream)
        A.check(A.lib().moe_ring_release(C.byref(self.r), int(slot), st), "moe_ring_release")

    def close(self):
        A.check(A.lib().moe_ring_destroy(C.byref(self.r)), "moe_ring_destroy")
