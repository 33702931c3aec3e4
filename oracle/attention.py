"""Oracle of the voxel-attention operators in float64: query/key norm with position rotation, ragged cross attention.

Written from the operators' definitions, sample by sample and head by head; it shares no code with the GPU path.
Each function can also return the sums of absolute values that its result's rounding errors scale with, which the
tests turn into tolerances.
"""
from __future__ import annotations

import numpy as np


def rope_turns(axis_pairs, theta: float = 10000.0):
    """(turns [P], axis [P]): revolutions per unit of position of every pair, and the position column it follows."""
    turns, axis = [], []
    for a, m in enumerate(axis_pairs):
        for j in range(m):
            turns.append(theta ** (-j / m) / (2 * np.pi))
            axis.append(a)
    return np.array(turns, np.float64), np.array(axis, np.int64)


def _pair_elements(pairs: int, layout: str):
    j = np.arange(pairs)
    return (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + pairs)


def rotate(x, positions, turns, axis, layout: str, back: bool = False):
    """x [n, H, D] with every pair turned by 2 pi turns[j] positions[:, axis[j]] (back: by the negative angle)."""
    y = np.array(x, np.float64)
    a, b = _pair_elements(len(turns), layout)
    for j in range(len(turns)):
        t = positions[:, axis[j]].astype(np.float64) * turns[j]
        ang = 2 * np.pi * (t - np.rint(t)) * (-1.0 if back else 1.0)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        xa, xb = x[..., a[j]], x[..., b[j]]
        y[..., a[j]] = xa * c - xb * s
        y[..., b[j]] = xa * s + xb * c
    return y


def _pair_size(x, turns, layout: str):
    """|x| of the elements a rotated element is made of: |x_a| + |x_b| for a pair, |x| past the pairs."""
    y = np.abs(np.array(x, np.float64))
    a, b = _pair_elements(len(turns), layout)
    both = y[..., a] + y[..., b]
    y[..., a] = both
    y[..., b] = both
    return y


def norm_rope_fwd(x, weight, positions, turns, axis, eps: float, layout: str = "interleaved", norm: bool = True):
    """y [n, H, D], and the size its rounding errors scale with."""
    x = np.asarray(x, np.float64)
    u = x
    if norm:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            u = u * np.asarray(weight, np.float64)
    return rotate(u, positions, turns, axis, layout), _pair_size(u, turns, layout)


def norm_rope_bwd(x, weight, positions, turns, axis, dy, eps: float, layout: str = "interleaved", norm: bool = True):
    """(dx, dweight or None, size of dx's errors, size of dweight's errors)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    g, gs = rotate(dy, positions, turns, axis, layout, back=True), _pair_size(dy, turns, layout)
    if not norm:
        return g, None, gs, None
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xn = x * r
    dx = r * (g * w - xn * (g * w * xn).mean(-1, keepdims=True))
    dxs = r * (gs * np.abs(w) + np.abs(xn) * (gs * np.abs(w) * np.abs(xn)).mean(-1, keepdims=True))
    if weight is None:
        return dx, None, dxs, None
    over = (0, 1) if np.ndim(weight) == 1 else 0
    return dx, (g * xn).sum(over), dxs, (gs * np.abs(xn)).sum(over)


def _samples(q_offsets, kv_offsets):
    for b in range(len(q_offsets) - 1):
        yield slice(int(q_offsets[b]), int(q_offsets[b + 1])), np.arange(int(kv_offsets[b]), int(kv_offsets[b + 1]))


def cross_attention_fwd(q, k, v, q_offsets, kv_offsets, kv_mask=None, scale=None):
    """(out [nq, Hq, D], lse [Hq, nq], sizes): sizes = (sum P |v| [nq, Hq, D], largest scale * sum |q k| [Hq, nq])."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    (nq, hq, d), hk = q.shape, k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, size = np.zeros((nq, hq, d)), np.zeros((nq, hq, d))
    lse, top = np.full((hq, nq), -np.inf), np.zeros((hq, nq))
    for rows, keys in _samples(q_offsets, kv_offsets):
        if kv_mask is not None:
            keys = keys[np.asarray(kv_mask)[keys] != 0]
        if len(keys) == 0 or rows.stop <= rows.start:
            continue
        for h in range(hq):
            kh, vh = k[keys, h * hk // hq], v[keys, h * hk // hq]
            s = scale * (q[rows, h] @ kh.T)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            tot = e.sum(1, keepdims=True)
            out[rows, h] = (e / tot) @ vh
            size[rows, h] = (e / tot) @ np.abs(vh)
            lse[h, rows] = (m + np.log(tot))[:, 0]
            top[h, rows] = (abs(scale) * (np.abs(q[rows, h]) @ np.abs(kh).T)).max(1)
    return out, lse, (size, top)


def cross_attention_bwd(q, k, v, dout, q_offsets, kv_offsets, kv_mask=None, scale=None, err=None):
    """(dq, dk, dv, sizes or None).  err = (ep, es, eo): relative errors of a probability and of dS, and an absolute
    error [nq, Hq, D] of the forward result that delta = sum dout * out is formed from; sizes are then the bounds of the
    errors of (dq, dk, dv) that these cause."""
    q, k, v, dout = (np.asarray(t, np.float64) for t in (q, k, v, dout))
    (nq, hq, d), hk = q.shape, k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    grads = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    sizes = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for rows, keys in _samples(q_offsets, kv_offsets):
        if kv_mask is not None:
            keys = keys[np.asarray(kv_mask)[keys] != 0]
        if len(keys) == 0 or rows.stop <= rows.start:
            continue
        for h in range(hq):
            g = h * hk // hq
            qh, kh, vh, do = q[rows, h], k[keys, g], v[keys, g], dout[rows, h]
            s = scale * (qh @ kh.T)
            e = np.exp(s - s.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            o = p @ vh
            ds = p * (do @ vh.T - (do * o).sum(1, keepdims=True))
            grads[0][rows, h] = scale * (ds @ kh)
            grads[1][keys, g] += scale * (ds.T @ qh)
            grads[2][keys, g] += p.T @ do
            if err is not None:
                ep, es, eo = err
                mag = np.abs(do) @ np.abs(vh).T + (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
                eds = es * np.abs(ds) + p * (np.abs(do) * eo[rows, h]).sum(1, keepdims=True) + ep * p * mag
                sizes[0][rows, h] = abs(scale) * (eds @ np.abs(kh))
                sizes[1][keys, g] += abs(scale) * (eds.T @ np.abs(qh))
                sizes[2][keys, g] += (ep + es) * (p.T @ np.abs(do))
    return grads[0], grads[1], grads[2], (sizes if err is not None else None)
