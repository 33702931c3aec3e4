"""Attention over voxel rows: query/key norm with position rotation, and ragged cross attention.

Thin marshalling of torch tensors into the ssc_qk_norm_rope_* and ssc_cross_attn_* calls of libssc, with autograd
wrappers.  Work runs on the current stream of the tensors' device; without the built library every call raises.
"""
from __future__ import annotations

import dataclasses
import math
import struct

import torch
from torch.autograd.function import once_differentiable

from .binding import DTYPE_CODE, SSC_OK, SSCError, _need, lib

ROPE_LAYOUTS = {"interleaved": 0, "halves": 1}


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _launch(func: str, device: torch.device, *args) -> None:
    """Calls func with the arguments and the current stream of `device`, which is the current GPU during the call."""
    if device.type != "cuda":
        raise ValueError(f"expected tensors on a GPU, got {device}")
    index = device.index
    # the bare checks and handles: a device guard's context takes 0.5 us, a Stream object 2 us
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            code = getattr(lib(), func)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        code = getattr(lib(), func)(*args, torch._C._cuda_getCurrentRawStream(index))
    if code != SSC_OK:
        raise SSCError(func, code)


def _new(like: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of like's shape and type."""
    return torch.empty_like(like) if like.is_contiguous() else like.new_empty(like.shape)


# the C structs of the calls' sizes (include/ssc.h), packed: a bytes object is passed as the pointer to them
_NORM_ROPE_SHAPE = struct.Struct("=6q9if")
_ATTN_SHAPE = struct.Struct("=8q5if")


def _heads(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, n: int | None = None) -> tuple:
    """(rows, heads, head_dim, row stride, head stride) of a [n, heads, head_dim] view whose heads are 16-byte vectors."""
    shape = t.shape
    if len(shape) != 3 or t.dtype != dtype or t.device != device or (n is not None and shape[0] != n):
        raise ValueError(f"{name}: expected {dtype} [{'n' if n is None else n}, heads, head_dim] on {device}, "
                         f"got {t.dtype} {tuple(shape)} on {t.device}")
    rows, heads, dim = shape
    rs, hs, es = t.stride()
    if rows <= 1:
        rs = 0  # a single row's stride is never used and may be anything
    if heads <= 1:
        hs = 0
    size = dtype.itemsize
    if dim > 1 and es != 1 or rs * size % 16 or hs * size % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}: a head's elements must be contiguous and rows and heads 16-byte aligned, "
                         f"got strides {t.stride()}")
    return rows, heads, dim, rs, hs


_MAX_ROW_STRIDE = 1 << 23  # SSC_MAX_ATTN_ROW_STRIDE


def _taken(t: torch.Tensor, most_row: int) -> bool:
    e = t.element_size()
    return (t.stride(2) == 1 and t.data_ptr() % 16 == 0
            and (t.shape[0] <= 1 or t.stride(0) * e % 16 == 0 and t.stride(0) <= most_row)
            and (t.shape[1] <= 1 or t.stride(1) * e % 16 == 0))


def _dense(t: torch.Tensor, most_row: int = 1 << 40) -> torch.Tensor:
    """t itself where the calls take its strides and its address, else a contiguous copy."""
    return t if t.dim() != 3 or _taken(t, most_row) else t.clone(memory_format=torch.contiguous_format)


def _packed(t: torch.Tensor | None) -> torch.Tensor | None:
    """t contiguous and 16-byte aligned: a contiguous view may start anywhere in its buffer."""
    if t is None or t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


# ---------------------------------------------------------------------------
# norm of queries and keys with position rotation
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class RopeTable:
    """The pairs of a rotation: revolutions per unit of position, and the position column each pair follows."""
    turns: torch.Tensor  # [pairs] float64
    axis: torch.Tensor   # [pairs] int32


def rope_table(axis_pairs, theta: float = 10000.0, device="cuda") -> RopeTable:
    """Pairs of a rotation over several axes: axis a gets axis_pairs[a] pairs, pair j of them turning by
    theta ** (-j / axis_pairs[a]) radians per unit of that axis's position (x, y, z of a voxel; time, height, width)."""
    counts = [int(m) for m in axis_pairs]
    if any(m < 0 for m in counts) or theta <= 0:
        raise ValueError(f"rope_table: expected counts of pairs and a positive theta, got {axis_pairs}, {theta}")
    turns = [theta ** (-j / m) / (2 * math.pi) for m in counts for j in range(m)]
    axis = [a for a, m in enumerate(counts) for _ in range(m)]
    return RopeTable(torch.tensor(turns, dtype=torch.float64, device=device),
                     torch.tensor(axis, dtype=torch.int32, device=device))


def _rope_shape(q, k, positions, table, q_weight, k_weight, eps, norm, layout):
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("qk_norm_rope: neither queries nor keys")
    dev, dt, n = ref.device, ref.dtype, int(ref.shape[0])
    if dt not in DTYPE_CODE:
        raise SSCError("ssc_qk_norm_rope", 2)
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    _, hq, dq, qr, qh = _heads(q, "q", dt, dev, n) if q is not None else (0, 0, 0, 0, 0)
    _, hk, dk, kr, kh = _heads(k, "k", dt, dev, n) if k is not None else (0, 0, 0, 0, 0)
    if q is not None and k is not None and dq != dk:
        raise ValueError(f"queries and keys have head sizes {dq} and {dk}")
    dim = dq or dk
    pairs = axes = pos_row = 0
    if (table is None) != (positions is None):
        raise ValueError("positions and table come together")
    if table is not None:
        pairs = int(table.turns.numel())
        _need(table.turns, "table.turns", torch.float64, (pairs,), dev)
        _need(table.axis, "table.axis", torch.int32, (pairs,), dev)
        if positions.dtype != torch.int32 or positions.dim() != 2 or positions.shape[0] != n or positions.device != dev:
            raise ValueError(f"positions: expected int32 [{n}, axes] on {dev}, got {positions.dtype} "
                             f"{tuple(positions.shape)} on {positions.device}")
        axes, pos_row = int(positions.shape[1]), int(positions.stride(0))
        if axes > 1 and positions.stride(1) != 1:
            raise ValueError("positions: a row's columns must be contiguous")
    per_head = None
    for w, name, h in ((q_weight, "q_weight", hq), (k_weight, "k_weight", hk)):
        if w is None:
            continue
        each = w.dim() == 2
        _need(w, name, dt, (h, dim) if each else (dim,), dev)
        if per_head is not None and per_head != each:
            raise ValueError("q_weight and k_weight: both [heads, head_dim] or both [head_dim]")
        per_head = each
    sh = _NORM_ROPE_SHAPE.pack(n, qr, qh, kr, kh, pos_row, hq, hk, dim, DTYPE_CODE[dt], axes, pairs,
                               ROPE_LAYOUTS[layout], 1 if norm else 0, 1 if per_head else 0, eps)
    return sh, dev, dt, (n, hq, dim), (n, hk, dim)


def _table_ptrs(positions, table):
    if table is None:
        return None, None, None
    return _ptr(positions), _ptr(table.turns), _ptr(table.axis)


def qk_norm_rope_fwd(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                     table: RopeTable | None = None, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, eps: float = 1e-6, norm: bool = True,
                     layout: str = "interleaved"):
    """ssc_qk_norm_rope_fwd: q [n, Hq, D], k [n, Hk, D] (views of a packed projection are taken as they are; either may
    be None) -> (q_out, k_out) contiguous.  positions: int32 [n, axes], for example coords[:, 1:]."""
    sh, dev, *_ = _rope_shape(q, k, positions, table, q_weight, k_weight, eps, norm, layout)
    qo = _new(q) if q is not None else None
    ko = _new(k) if k is not None else None
    _launch("ssc_qk_norm_rope_fwd", dev, sh, _ptr(q), _ptr(k), *_table_ptrs(positions, table), _ptr(q_weight),
            _ptr(k_weight), _ptr(qo), _ptr(ko))
    return qo, ko


def qk_norm_rope_bwd(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None,
                     table: RopeTable | None, dq_out: torch.Tensor | None, dk_out: torch.Tensor | None,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     norm: bool = True, layout: str = "interleaved", need_weights: bool = True):
    """ssc_qk_norm_rope_bwd: (dq, dk, dq_weight, dk_weight) for the output gradients (either may be None: its inputs'
    gradients are then None); a weight's gradient is None where there is no weight."""
    sh, dev, dt, qs, ks = _rope_shape(q, k, positions, table, q_weight, k_weight, eps, norm, layout)
    if dq_out is not None:
        _need(dq_out, "dq_out", dt, qs, dev)
    if dk_out is not None:
        _need(dk_out, "dk_out", dt, ks, dev)
    dq = torch.empty_like(dq_out) if dq_out is not None else None
    dk = torch.empty_like(dk_out) if dk_out is not None else None
    dqw = torch.empty_like(q_weight) if need_weights and q_weight is not None and dq_out is not None else None
    dkw = torch.empty_like(k_weight) if need_weights and k_weight is not None and dk_out is not None else None
    ws = None
    if dqw is not None or dkw is not None:
        nbytes = int(lib().ssc_qk_norm_rope_workspace_bytes(sh))
        if nbytes == 0:
            raise SSCError("ssc_qk_norm_rope_workspace_bytes", 2)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _launch("ssc_qk_norm_rope_bwd", dev, sh, _ptr(q), _ptr(k), *_table_ptrs(positions, table), _ptr(q_weight),
            _ptr(k_weight), _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(ws),
            0 if ws is None else ws.numel())
    return dq, dk, dqw, dkw


class QKNormRopeFunction(torch.autograd.Function):
    """autograd wrapper: forward = ssc_qk_norm_rope_fwd, backward = ssc_qk_norm_rope_bwd."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, table, eps, norm, layout):
        q, k = (None if t is None else _dense(t) for t in (q, k))
        q_weight, k_weight = _packed(q_weight), _packed(k_weight)
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        ctx.rest = (table, eps, norm, layout)
        return qk_norm_rope_fwd(q, k, positions, table, q_weight, k_weight, eps, norm, layout)

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko):
        q, k, qw, kw, positions = ctx.saved_tensors
        table, eps, norm, layout = ctx.rest
        need = ctx.needs_input_grad
        dqo = _packed(dqo) if dqo is not None and q is not None and (need[0] or need[2]) else None
        dko = _packed(dko) if dko is not None and k is not None and (need[1] or need[3]) else None
        if dqo is None and dko is None:
            return (None,) * 9
        dq, dk, dqw, dkw = qk_norm_rope_bwd(q, k, positions, table, dqo, dko, qw, kw, eps, norm, layout,
                                            need_weights=need[2] or need[3])
        return dq, dk, dqw, dkw, None, None, None, None, None


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 table: RopeTable | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, norm: bool = True,
                 layout: str = "interleaved"):
    """Differentiable qk_norm_rope_fwd."""
    return QKNormRopeFunction.apply(q, k, q_weight, k_weight, positions, table, eps, norm, layout)


# ---------------------------------------------------------------------------
# cross attention
# ---------------------------------------------------------------------------

def row_offsets(coords: torch.Tensor, batch: int) -> torch.Tensor:
    """[batch + 1] int32 offsets of the samples' rows in coords [n, 4] (b, x, y, z), whose rows are grouped by sample."""
    b = coords[:, 0].contiguous()
    return torch.searchsorted(b, torch.arange(batch + 1, dtype=b.dtype, device=b.device)).to(torch.int32)


def _attn_shape(q, k, v, q_offsets, kv_offsets, kv_mask, scale):
    dev, dt = q.device, q.dtype
    if dt not in DTYPE_CODE:
        raise SSCError("ssc_cross_attn", 2)
    nq, hq, dim, qr, qh = _heads(q, "q", dt, dev)
    nk, hk, dim_k, kr, kh = _heads(k, "k", dt, dev)
    _, hv, dim_v, vr, vh = _heads(v, "v", dt, dev, nk)
    if dim_k != dim or dim_v != dim or hv != hk:
        raise ValueError(f"q, k, v: heads and head sizes {tuple(q.shape[1:])}, {tuple(k.shape[1:])}, {tuple(v.shape[1:])} "
                         "do not match")
    batch = int(q_offsets.shape[0]) - 1
    _need(q_offsets, "q_offsets", torch.int32, (batch + 1,), dev)
    _need(kv_offsets, "kv_offsets", torch.int32, (batch + 1,), dev)
    if kv_mask is not None:
        if kv_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"kv_mask: expected bool (True: attended), got {kv_mask.dtype}")
        _need(kv_mask, "kv_mask", kv_mask.dtype, (nk,), dev)
    if scale is None:
        scale = dim ** -0.5
    sh = _ATTN_SHAPE.pack(nq, nk, qr, qh, kr, kh, vr, vh, batch, hq, hk, dim, DTYPE_CODE[dt], scale)
    return sh, dev, dt, (hq, nq)


_unused: dict[int, torch.Tensor] = {}  # by device: stands for the workspace of calls that use none


def _attn_workspace(sh: bytes, backward: int, dev: torch.device) -> torch.Tensor:
    nbytes = int(lib().ssc_cross_attn_workspace_bytes(sh, backward))
    if nbytes == 0:
        raise SSCError("ssc_cross_attn_workspace_bytes", 2)
    if nbytes == 256 and not backward:  # the smallest size: nothing is kept there
        ws = _unused.get(dev.index)
        if ws is None:
            ws = _unused[dev.index] = torch.empty(256, dtype=torch.uint8, device=dev)
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def cross_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                        kv_offsets: torch.Tensor, kv_mask: torch.Tensor | None = None, scale: float | None = None):
    """ssc_cross_attn_fwd: q [nq, Hq, D] attends k, v [nk, Hk, D] sample by sample -> (out [nq, Hq, D], lse [Hq, nq]).

    Offsets are int32 [batch + 1] on the device, kv_mask [nk] bool (True: attended), scale 1 / sqrt(D) by default."""
    sh, dev, _, rows = _attn_shape(q, k, v, q_offsets, kv_offsets, kv_mask, scale)
    ws = _attn_workspace(sh, 0, dev)
    out = _new(q)
    lse = q.new_empty(rows, dtype=torch.float32)
    _launch("ssc_cross_attn_fwd", dev, sh, _ptr(q), _ptr(k), _ptr(v), _ptr(q_offsets), _ptr(kv_offsets),
            _ptr(kv_mask), _ptr(out), _ptr(lse), _ptr(ws), ws.numel())
    return out, lse


def cross_attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                        dout: torch.Tensor, q_offsets: torch.Tensor, kv_offsets: torch.Tensor,
                        kv_mask: torch.Tensor | None = None, scale: float | None = None, need_dq: bool = True,
                        need_dk: bool = True, need_dv: bool = True):
    """ssc_cross_attn_bwd: (dq, dk, dv) of cross_attention_fwd; entries not asked for are None."""
    sh, dev, dt, rows = _attn_shape(q, k, v, q_offsets, kv_offsets, kv_mask, scale)
    _need(out, "out", dt, tuple(q.shape), dev)
    _need(dout, "dout", dt, tuple(q.shape), dev)
    _need(lse, "lse", torch.float32, rows, dev)
    ws = _attn_workspace(sh, 1, dev)
    dq = torch.empty_like(dout) if need_dq else None
    dk = _new(k) if need_dk else None
    dv = _new(v) if need_dv else None
    _launch("ssc_cross_attn_bwd", dev, sh, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
            _ptr(q_offsets), _ptr(kv_offsets), _ptr(kv_mask), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel())
    return dq, dk, dv


class CrossAttentionFunction(torch.autograd.Function):
    """autograd wrapper: forward = ssc_cross_attn_fwd, backward = ssc_cross_attn_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, q_offsets, kv_offsets, kv_mask, scale):
        q, k, v = (_dense(t, _MAX_ROW_STRIDE) for t in (q, k, v))
        out, lse = cross_attention_fwd(q, k, v, q_offsets, kv_offsets, kv_mask, scale)
        ctx.save_for_backward(q, k, v, out, lse, q_offsets, kv_offsets, kv_mask)
        ctx.scale = scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, qo, ko, mask = ctx.saved_tensors
        nq, nk, nv = ctx.needs_input_grad[:3]
        dq, dk, dv = cross_attention_bwd(q, k, v, out, lse, _packed(dout), qo, ko, mask, ctx.scale, nq, nk, nv)
        return dq, dk, dv, None, None, None, None


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor, kv_offsets: torch.Tensor,
                    kv_mask: torch.Tensor | None = None, scale: float | None = None) -> torch.Tensor:
    """Differentiable cross_attention_fwd (its out)."""
    return CrossAttentionFunction.apply(q, k, v, q_offsets, kv_offsets, kv_mask, scale)
