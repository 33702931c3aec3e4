"""Operators of networks over serialised voxel rows: windowed attention, gated scan, layer norm with residual and dropout.

Thin marshalling of torch tensors into the calls of libssc, with autograd wrappers.  Work runs on the current stream of
the tensors' device; without the built library every call raises.
"""
from __future__ import annotations

import struct

import torch
from torch.autograd.function import once_differentiable

from .attention import _MAX_ROW_STRIDE, _attn_shape, _dense, _launch, _new, _packed, _ptr, _workspace
from .binding import DTYPE_CODE, SSCError, _need, lib

# the C structs of the calls' sizes (include/ssc.h), packed: a bytes object is passed as the pointer to them
_NORM_SHAPE = struct.Struct("=3qd3if")
_SCAN_SHAPE = struct.Struct("=3q5i")
_WINDOW = struct.Struct("=3i")

SCAN_FORMS = {"mix": 0, "sum": 1}


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, shape: tuple | None = None) -> int:
    """The row stride of a [n, channels] view whose rows are 16-byte vectors."""
    have = t.shape
    if len(have) != 2 or t.dtype != dtype or t.device != device or (shape is not None and have != shape):
        want = "[n, channels]" if shape is None else list(shape)
        raise ValueError(f"{name}: expected {dtype} {want} on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    rows, channels = have
    if t.is_contiguous() and t.data_ptr() % 16 == 0:  # the calls refuse rows that are not 16-byte vectors
        return channels if rows > 1 else 0
    row, one = t.stride()
    if rows <= 1:
        row = 0  # a single row's stride is never used and may be anything
    if channels > 1 and one != 1 or row * dtype.itemsize % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}: a row's elements must be contiguous and rows 16-byte aligned, got strides {t.stride()}")
    return row


def _dense_rows(t: torch.Tensor | None, most: int = 1 << 40) -> torch.Tensor | None:
    """t itself where the calls take its rows as they lie (at most `most` elements apart), else a contiguous copy."""
    if t is None or t.dim() != 2:
        return t
    taken = (t.stride(1) == 1 or t.shape[1] <= 1) and t.data_ptr() % 16 == 0 and (
        t.shape[0] <= 1 or t.stride(0) * t.element_size() % 16 == 0 and t.stride(0) <= most)
    return t if taken else t.clone(memory_format=torch.contiguous_format)


def _dtype_code(func: str, dtype: torch.dtype) -> int:
    if dtype not in DTYPE_CODE:
        raise SSCError(func, 2)
    return DTYPE_CODE[dtype]


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

def _need_rng(rng: torch.Tensor | None, p: float, layer: int, device: torch.device) -> None:
    if not 0 <= layer < 1 << 31:
        raise ValueError(f"dropout: layer must be in [0, 2^31), got {layer}")
    if p > 0 and rng is None:
        raise ValueError("dropout: rng is needed where p > 0")
    if rng is not None:
        _need(rng, "rng", torch.int64, (2,), device)


def dropout_fwd(x: torch.Tensor, p: float, rng: torch.Tensor | None = None, layer: int = 0,
                residual: torch.Tensor | None = None) -> torch.Tensor:
    """ssc_dropout: x (any shape, contiguous) with elements dropped with chance p and the others scaled, plus residual.

    rng: int64 [2] on the device, (seed, step); the same rng, layer and p drop the same elements of a tensor's shape."""
    code = _dtype_code("ssc_dropout", x.dtype)
    dev = x.device
    _need(x, "x", x.dtype, tuple(x.shape), dev)
    if residual is not None:
        _need(residual, "residual", x.dtype, tuple(x.shape), dev)
    _need_rng(rng, p, layer, dev)
    y = torch.empty_like(x)
    _launch("ssc_dropout", dev, x.numel(), code, p, layer, _ptr(x), _ptr(residual), _ptr(rng), _ptr(y))
    return y


def dropout_bwd(dy: torch.Tensor, p: float, rng: torch.Tensor | None = None, layer: int = 0) -> torch.Tensor:
    """The gradient of dropout_fwd's x: dy through the same choice (the residual's gradient is dy itself)."""
    return dropout_fwd(dy, p, rng, layer)


class DropoutFunction(torch.autograd.Function):
    """autograd wrapper: forward = ssc_dropout, backward = ssc_dropout of the output gradient."""

    @staticmethod
    def forward(ctx, x, p, rng, layer, residual):
        ctx.save_for_backward(rng)
        ctx.rest = (p, layer)
        return dropout_fwd(_packed(x), p, rng, layer, _packed(residual))

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (rng,) = ctx.saved_tensors
        p, layer = ctx.rest
        dx = dropout_bwd(_packed(dy), p, rng, layer) if ctx.needs_input_grad[0] else None
        return dx, None, None, None, dy if ctx.needs_input_grad[4] else None


def dropout(x: torch.Tensor, p: float, rng: torch.Tensor | None = None, layer: int = 0,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable dropout_fwd.  rng may change only after the backward pass has read it (autograd says so)."""
    return DropoutFunction.apply(x, p, rng, layer, residual)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def _norm_shape(x, x_name, weight, bias, eps, p=0.0, layer=0, residual_row=0):
    code = _dtype_code("ssc_layer_norm", x.dtype)
    dev = x.device
    row = _rows(x, x_name, x.dtype, dev)
    n, c = x.shape
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _need(t, name, x.dtype, (c,), dev)
    return _NORM_SHAPE.pack(n, row, residual_row, p, c, code, layer, eps), dev


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   eps: float = 1e-5) -> torch.Tensor:
    """ssc_layer_norm_fwd: y of x [n, C] (rows may be strided), contiguous."""
    sh, dev = _norm_shape(x, "x", weight, bias, eps)
    y = _new(x)
    _launch("ssc_layer_norm_fwd", dev, sh, _ptr(x), None, _ptr(weight), _ptr(bias), None, _ptr(y), None)
    return y


def add_layer_norm_fwd(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                       bias: torch.Tensor | None = None, eps: float = 1e-5, p: float = 0.0,
                       rng: torch.Tensor | None = None, layer: int = 0):
    """ssc_layer_norm_fwd with a residual: (y, s), s = residual + dropout(x) and y its norm, both contiguous.

    p, rng and layer as dropout_fwd's, whose choice for a contiguous x it is."""
    row = _rows(residual, "residual", x.dtype, x.device, x.shape)
    sh, dev = _norm_shape(x, "x", weight, bias, eps, p, layer, row)
    _need_rng(rng, p, layer, dev)
    y, s = _new(x), _new(x)
    _launch("ssc_layer_norm_fwd", dev, sh, _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), _ptr(rng), _ptr(y), _ptr(s))
    return y, s


def _norm_bwd(sh, dev, s, dy, ds, weight, bias, rng, dx, dresidual, need_weights):
    dw = torch.empty_like(weight) if need_weights and weight is not None else None
    db = torch.empty_like(bias) if need_weights and bias is not None else None
    ws, nbytes = None, 0
    if dw is not None or db is not None:
        nbytes = int(lib().ssc_layer_norm_workspace_bytes(sh))
        if nbytes == 0:
            raise SSCError("ssc_layer_norm_workspace_bytes", 2)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _launch("ssc_layer_norm_bwd", dev, sh, _ptr(s), _ptr(dy), _ptr(ds), _ptr(weight), _ptr(rng), _ptr(dx),
            _ptr(dresidual), _ptr(dw), _ptr(db), _ptr(ws), nbytes)
    return dw, db


def layer_norm_bwd(x: torch.Tensor, dy: torch.Tensor, weight: torch.Tensor | None = None,
                   bias: torch.Tensor | None = None, eps: float = 1e-5, need_dx: bool = True, need_weights: bool = True):
    """ssc_layer_norm_bwd: (dx, dweight, dbias); a gradient not asked for, or of a weight or bias not given, is None."""
    sh, dev = _norm_shape(x, "x", weight, bias, eps)
    _need(dy, "dy", x.dtype, tuple(x.shape), dev)
    dx = torch.empty_like(dy) if need_dx else None
    dw, db = _norm_bwd(sh, dev, x, dy, None, weight, bias, None, dx, None, need_weights)
    return dx, dw, db


def add_layer_norm_bwd(s: torch.Tensor, dy: torch.Tensor, ds: torch.Tensor | None, weight: torch.Tensor | None = None,
                       bias: torch.Tensor | None = None, eps: float = 1e-5, p: float = 0.0,
                       rng: torch.Tensor | None = None, layer: int = 0, need_dx: bool = True,
                       need_dresidual: bool = True, need_weights: bool = True):
    """ssc_layer_norm_bwd with a residual: (dx, dresidual, dweight, dbias) from the s of the forward call and the output
    gradients dy and ds (or None).  Without dropout dx and dresidual are one tensor."""
    sh, dev = _norm_shape(s, "s", weight, bias, eps, p, layer)
    _need(dy, "dy", s.dtype, tuple(s.shape), dev)
    if ds is not None:
        _need(ds, "ds", s.dtype, tuple(s.shape), dev)
    _need_rng(rng, p, layer, dev)
    one = p == 0
    dresidual = torch.empty_like(dy) if need_dresidual or (one and need_dx) else None
    dx = torch.empty_like(dy) if need_dx and not one else None
    dw, db = _norm_bwd(sh, dev, s, dy, ds, weight, bias, rng, dx, dresidual, need_weights)
    return (dresidual if need_dx else None) if one else dx, dresidual if need_dresidual else None, dw, db


class LayerNormFunction(torch.autograd.Function):
    """autograd wrapper: forward = ssc_layer_norm_fwd, backward = ssc_layer_norm_bwd."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x, weight, bias = _dense_rows(x), _packed(weight), _packed(bias)
        ctx.save_for_backward(x, weight, bias)
        ctx.eps = eps
        return layer_norm_fwd(x, weight, bias, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_bwd(x, _packed(dy), weight, bias, ctx.eps, need[0], need[1] or need[2])
        return dx, dw, db, None


class AddLayerNormFunction(torch.autograd.Function):
    """autograd wrapper of the form with a residual: outputs (y, s)."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, p, rng, layer):
        weight, bias = _packed(weight), _packed(bias)
        y, s = add_layer_norm_fwd(_dense_rows(x), _dense_rows(residual), weight, bias, eps, p, rng, layer)
        ctx.save_for_backward(s, weight, bias, rng)
        ctx.rest = (eps, p, layer)
        ctx.set_materialize_grads(False)
        return y, s

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds):
        s, weight, bias, rng = ctx.saved_tensors
        eps, p, layer = ctx.rest
        need = ctx.needs_input_grad
        if dy is None:  # y was not used: s alone carries a gradient
            if ds is None:
                return (None,) * 8
            dx = None if not need[0] else dropout_bwd(_packed(ds), p, rng, layer) if p > 0 else ds
            return dx, ds if need[1] else None, None, None, None, None, None, None
        dx, dr, dw, db = add_layer_norm_bwd(s, _packed(dy), _packed(ds), weight, bias, eps, p, rng, layer, need[0], need[1],
                                            need[2] or need[3])
        return dx, dr, dw, db, None, None, None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer_norm_fwd."""
    return LayerNormFunction.apply(x, weight, bias, eps)


def add_layer_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                   bias: torch.Tensor | None = None, eps: float = 1e-5, p: float = 0.0,
                   rng: torch.Tensor | None = None, layer: int = 0):
    """Differentiable add_layer_norm_fwd: (y, s).  rng may change only after the backward pass has read it."""
    return AddLayerNormFunction.apply(x, residual, weight, bias, eps, p, rng, layer)


# ---------------------------------------------------------------------------
# gated scan
# ---------------------------------------------------------------------------

_MAX_SCAN_ROW_STRIDE = 1 << 21  # SSC_MAX_SCAN_ROW_STRIDE


def _scan_shape(x, gate, offsets, h0, reverse, form):
    code = _dtype_code("ssc_gated_scan", x.dtype)
    if form not in SCAN_FORMS:
        raise ValueError(f"form must be one of {sorted(SCAN_FORMS)}, got {form!r}")
    dev = x.device
    x_row = _rows(x, "x", x.dtype, dev)
    gate_row = _rows(gate, "gate", x.dtype, dev, x.shape)
    n, c = x.shape
    batch = int(offsets.shape[0]) - 1
    _need(offsets, "offsets", torch.int32, (batch + 1,), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (batch, c), dev)
    return _SCAN_SHAPE.pack(n, x_row, gate_row, batch, c, code, SCAN_FORMS[form], 1 if reverse else 0), dev, (batch, c)


def _scan_bytes(func: str, sh: bytes) -> int:
    nbytes = int(getattr(lib(), func)(sh))
    if nbytes == 0:
        raise SSCError(func, 2)
    return nbytes


def gated_scan_fwd(x: torch.Tensor, gate: torch.Tensor, offsets: torch.Tensor, h0: torch.Tensor | None = None,
                   reverse: bool = False, form: str = "mix", need_carries: bool = False):
    """ssc_gated_scan_fwd: (y, last, carries) of x and gate [n, C] (rows may be strided) along each sample's rows.

    h = sigmoid(gate) h + (1 - sigmoid(gate)) x (form "mix") or + x ("sum"), from h0 [batch, C] fp32 (zeros without one),
    from a sample's last row to its first where reversed.  y [n, C]; last [batch, C] fp32, the final states; carries: what
    gated_scan_bwd takes over, where asked for.  One row a sample and h0 make a step of the recurrence."""
    sh, dev, state = _scan_shape(x, gate, offsets, h0, reverse, form)
    nbytes = _scan_bytes("ssc_gated_scan_workspace_bytes", sh)
    ws = _workspace(nbytes, nbytes == 256, dev)  # the smallest size: a single tile exchanges nothing
    y = _new(x)
    last = x.new_empty(state, dtype=torch.float32)
    carries = None
    if need_carries:
        carries = x.new_empty(_scan_bytes("ssc_gated_scan_carry_bytes", sh) // 4, dtype=torch.float32)
    _launch("ssc_gated_scan_fwd", dev, sh, _ptr(x), _ptr(gate), _ptr(offsets), _ptr(h0), _ptr(y), _ptr(last), _ptr(carries),
            _ptr(ws), nbytes)
    return y, last, carries


def gated_scan_bwd(x: torch.Tensor, gate: torch.Tensor, carries: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor,
                   h0: torch.Tensor | None = None, dlast: torch.Tensor | None = None, reverse: bool = False,
                   form: str = "mix"):
    """ssc_gated_scan_bwd: (dx, dgate, dh0) from the output gradients dy and dlast (or None); dh0 is None without h0."""
    sh, dev, state = _scan_shape(x, gate, offsets, h0, reverse, form)
    _need(dy, "dy", x.dtype, tuple(x.shape), dev)
    _need(carries, "carries", torch.float32, (_scan_bytes("ssc_gated_scan_carry_bytes", sh) // 4,), dev)
    if dlast is not None:
        _need(dlast, "dlast", torch.float32, state, dev)
    nbytes = _scan_bytes("ssc_gated_scan_workspace_bytes", sh)
    ws = _workspace(nbytes, nbytes == 256, dev)  # the smallest size: a single tile exchanges nothing
    dx, dgate = torch.empty_like(dy), torch.empty_like(dy)
    dh0 = torch.empty_like(h0) if h0 is not None else None
    _launch("ssc_gated_scan_bwd", dev, sh, _ptr(x), _ptr(gate), _ptr(carries), _ptr(dy), _ptr(offsets), _ptr(h0),
            _ptr(dlast), _ptr(dx), _ptr(dgate), _ptr(dh0), _ptr(ws), nbytes)
    return dx, dgate, dh0


class GatedScanFunction(torch.autograd.Function):
    """autograd wrapper: forward = ssc_gated_scan_fwd, backward = ssc_gated_scan_bwd; outputs (y, last)."""

    @staticmethod
    def forward(ctx, x, gate, offsets, h0, reverse, form):
        x, gate, h0 = _dense_rows(x, _MAX_SCAN_ROW_STRIDE), _dense_rows(gate, _MAX_SCAN_ROW_STRIDE), _packed(h0)
        y, last, carries = gated_scan_fwd(x, gate, offsets, h0, reverse, form, need_carries=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, gate, offsets, h0, carries)
        ctx.rest = (reverse, form)
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, gate, offsets, h0, carries = ctx.saved_tensors
        if dy is None and dlast is None:
            return (None,) * 6
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _packed(dy)
        dx, dgate, dh0 = gated_scan_bwd(x, gate, carries, dy, offsets, h0, _packed(dlast), *ctx.rest)
        need = ctx.needs_input_grad
        return dx if need[0] else None, dgate if need[1] else None, None, dh0 if need[3] else None, None, None


def gated_scan(x: torch.Tensor, gate: torch.Tensor, offsets: torch.Tensor, h0: torch.Tensor | None = None,
               reverse: bool = False, form: str = "mix"):
    """Differentiable gated_scan_fwd: (y, last)."""
    return GatedScanFunction.apply(x, gate, offsets, h0, reverse, form)


# ---------------------------------------------------------------------------
# windowed attention
# ---------------------------------------------------------------------------

_MAX_WINDOW = 1 << 28  # SSC_MAX_ATTN_ROWS


def _window(left: int | None, right: int | None, sinks: int) -> bytes:
    for v, name in ((left, "left"), (right, "right"), (sinks, "sinks")):
        if v is not None and (v < 0 or v > _MAX_WINDOW) or (v is None and name == "sinks"):
            raise ValueError(f"{name} must be in [0, 2^28]{'' if name == 'sinks' else ', or None for no bound'}, got {v}")
    return _WINDOW.pack(-1 if left is None else left, -1 if right is None else right, sinks)


def _window_workspace(sh: bytes, window: bytes, backward: int, dev: torch.device) -> torch.Tensor:
    nbytes = int(lib().ssc_window_attn_workspace_bytes(sh, window, backward))
    if nbytes == 0:
        raise SSCError("ssc_window_attn_workspace_bytes", 2)
    return _workspace(nbytes, nbytes == 256 and not backward, dev)  # the smallest size: nothing is kept there


def window_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                         kv_offsets: torch.Tensor, left: int | None, right: int | None, sinks: int = 0,
                         kv_mask: torch.Tensor | None = None, scale: float | None = None):
    """ssc_window_attn_fwd: cross_attention_fwd in which row i of a sample, at place t = i + keys - rows of its keys, sees
    the keys j <= t + right with j >= t - left or j < sinks (None: no bound) -> (out [nq, Hq, D], lse [Hq, nq])."""
    window = _window(left, right, sinks)
    sh, dev, _, rows = _attn_shape(q, k, v, q_offsets, kv_offsets, kv_mask, scale)
    ws = _window_workspace(sh, window, 0, dev)
    out = _new(q)
    lse = q.new_empty(rows, dtype=torch.float32)
    _launch("ssc_window_attn_fwd", dev, sh, window, _ptr(q), _ptr(k), _ptr(v), _ptr(q_offsets), _ptr(kv_offsets),
            _ptr(kv_mask), _ptr(out), _ptr(lse), _ptr(ws), ws.numel())
    return out, lse


def window_attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                         dout: torch.Tensor, q_offsets: torch.Tensor, kv_offsets: torch.Tensor, left: int | None,
                         right: int | None, sinks: int = 0, kv_mask: torch.Tensor | None = None,
                         scale: float | None = None, need_dq: bool = True, need_dk: bool = True, need_dv: bool = True):
    """ssc_window_attn_bwd: (dq, dk, dv) of window_attention_fwd; entries not asked for are None."""
    window = _window(left, right, sinks)
    sh, dev, dt, rows = _attn_shape(q, k, v, q_offsets, kv_offsets, kv_mask, scale)
    _need(out, "out", dt, tuple(q.shape), dev)
    _need(dout, "dout", dt, tuple(q.shape), dev)
    _need(lse, "lse", torch.float32, rows, dev)
    ws = _window_workspace(sh, window, 1, dev)
    dq = torch.empty_like(dout) if need_dq else None
    dk = _new(k) if need_dk else None
    dv = _new(v) if need_dv else None
    _launch("ssc_window_attn_bwd", dev, sh, window, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
            _ptr(q_offsets), _ptr(kv_offsets), _ptr(kv_mask), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel())
    return dq, dk, dv


class WindowAttentionFunction(torch.autograd.Function):
    """autograd wrapper: forward = ssc_window_attn_fwd, backward = ssc_window_attn_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, q_offsets, kv_offsets, left, right, sinks, kv_mask, scale):
        q, k, v = (_dense(t, _MAX_ROW_STRIDE) for t in (q, k, v))
        out, lse = window_attention_fwd(q, k, v, q_offsets, kv_offsets, left, right, sinks, kv_mask, scale)
        ctx.save_for_backward(q, k, v, out, lse, q_offsets, kv_offsets, kv_mask)
        ctx.rest = (left, right, sinks, scale)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, qo, ko, mask = ctx.saved_tensors
        left, right, sinks, scale = ctx.rest
        need = ctx.needs_input_grad
        dq, dk, dv = window_attention_bwd(q, k, v, out, lse, _packed(dout), qo, ko, left, right, sinks, mask, scale,
                                          need[0], need[1], need[2])
        return dq, dk, dv, None, None, None, None, None, None, None


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                     kv_offsets: torch.Tensor, left: int | None, right: int | None, sinks: int = 0,
                     kv_mask: torch.Tensor | None = None, scale: float | None = None) -> torch.Tensor:
    """Differentiable window_attention_fwd (its out)."""
    return WindowAttentionFunction.apply(q, k, v, q_offsets, kv_offsets, left, right, sinks, kv_mask, scale)
