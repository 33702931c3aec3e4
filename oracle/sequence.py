"""Oracle of the operators over serialised voxel rows in float64: layer norm, dropout, gated scan, windowed attention.

Written from the operators' definitions; it shares no code with the GPU path.  Next to a result each function can return
the bound on an fp32 evaluation's error before the result's own rounding, which the tests turn into tolerances.
"""
from __future__ import annotations

import numpy as np

F = 2.0 ** -24  # half a step of fp32


def philox(counter, key, rounds: int = 10):
    """Philox-4x32 on lists of words (Salmon, Moraes, Dror and Shaw 2011), in Python's own integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_threshold(p: float) -> int:
    return min(65535, int(np.floor(p * 65536 + 0.5)))


def dropout_factor(count: int, p: float, seed: int, step: int, layer: int):
    """[count] 0 or 65536 / (65536 - t) for each element."""
    t = dropout_threshold(p)
    if t == 0:
        return np.ones(count)
    m = 0xFFFFFFFF
    seed, step = seed % (1 << 64), step % (1 << 64)
    out = np.zeros((count + 7) // 8 * 8)
    for b in range((count + 7) // 8):
        words = philox([b, layer, step & m, step >> 32], [seed & m, seed >> 32])
        for i in range(8):
            if (words[i // 2] >> (16 * (i % 2))) & 0xFFFF >= t:
                out[8 * b + i] = 65536.0 / (65536 - t)
    return out[:count]


def _statistics(s, eps):
    """(differences, r, z, error of a difference, relative error of r) of rows s; es: error of s itself is 3 f |s|."""
    c = s.shape[1]
    mean = s.mean(1, keepdims=True)
    d = s - mean
    var = (d * d).mean(1, keepdims=True)
    r = 1.0 / np.sqrt(var + eps)
    # the mean: a sum of C terms in any order; the variance's first-order term in the mean's error is zero
    em = (c + 2) * F * np.abs(s).mean(1, keepdims=True)
    ed = em + 3 * F * np.abs(s) + F * np.abs(d)
    rel = 0.5 * ((c + 4) * F + 2 * (ed * np.abs(d)).mean(1, keepdims=True) * r * r + (ed * ed).mean(1, keepdims=True) * r * r) + 4 * F
    return d, r, d * r, ed, rel


def layer_norm_fwd(s, weight, bias, eps: float):
    """(y [n, C], error bound)."""
    s = np.asarray(s, np.float64)
    d, r, z, ed, rel = _statistics(s, eps)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    b = 0.0 if bias is None else np.asarray(bias, np.float64)
    y = z * w + b
    return y, np.abs(w) * (r * ed + np.abs(z) * (rel + 3 * F)) + F * (np.abs(z * w) + np.abs(y))


def layer_norm_bwd(s, dy, weight, eps: float, ds=None):
    """(dresidual, dweight, dbias, (their error bounds))."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    n, c = s.shape
    d, r, z, ed, rel = _statistics(s, eps)
    ez = r * ed + np.abs(z) * (rel + 2 * F)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    g = dy * w
    mg, mz = g.mean(1, keepdims=True), (g * z).mean(1, keepdims=True)
    inner = g - mg - z * mz
    dx = r * inner
    emg = (c + 3) * F * np.abs(g).mean(1, keepdims=True)
    emz = (c + 4) * F * np.abs(g * z).mean(1, keepdims=True) + (np.abs(g) * ez).mean(1, keepdims=True)
    mag = np.abs(g) + np.abs(mg) + np.abs(z * mz)
    err = r * (4 * F * mag + emg + np.abs(z) * emz + np.abs(mz) * ez) + (rel + 2 * F) * np.abs(dx)
    if ds is not None:
        dx = dx + np.asarray(ds, np.float64)
        err = err + F * np.abs(dx)
    dw, db = (dy * z).sum(0), dy.sum(0)
    edw = (np.abs(dy) * ez).sum(0) + (n + 4) * F * np.abs(dy * z).sum(0)
    return dx, dw, db, (err, edw, (n + 4) * F * np.abs(dy).sum(0))


def gated_scan_fwd(x, gate, offsets, h0=None, reverse: bool = False, form: str = "mix", ea: float = 0.0):
    """(y [n, C], last [batch, C], their error bounds), row by row.

    ea: bound on the relative error of the smaller side q of (a, 1 - a); the larger one, 1 - q, is then off by ea q + F."""
    x, gate = np.asarray(x, np.float64), np.asarray(gate, np.float64)
    n, c = x.shape
    batch = len(offsets) - 1
    y, ey = np.zeros((n, c)), np.zeros((n, c))
    last = np.zeros((batch, c)) if h0 is None else np.array(h0, np.float64)
    el = np.zeros((batch, c))
    for b in range(batch):
        rows = range(int(offsets[b]), int(offsets[b + 1]))
        h, e = last[b].copy(), np.zeros(c)
        for t in (reversed(rows) if reverse else rows):
            a, keep, da, dk = _sides(gate[t], ea)
            add, dadd = (keep * x[t], dk * np.abs(x[t])) if form == "mix" else (x[t], 0.0)
            e = a * e + da * (np.abs(h) + e) + dadd + 2 * F * (np.abs(add) + a * np.abs(h))
            h = a * h + add
            e = e + F * np.abs(h)
            y[t], ey[t] = h, e
        last[b], el[b] = h, e
    return y, last, (ey, el)


def _sides(g, ea):
    """(a, 1 - a, error of a, error of 1 - a) of gate logits."""
    a, keep = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    q = np.minimum(a, keep)
    small, large = ea * q, ea * q + F
    return a, keep, np.where(a <= keep, small, large), np.where(a <= keep, large, small)


def gated_scan_bwd(x, gate, dy, offsets, h0=None, dlast=None, reverse: bool = False, form: str = "mix", ea: float = 0.0):
    """(dx, dgate, dh0, (their error bounds)), row by row; bounds as gated_scan_fwd's."""
    x, gate, dy = (np.asarray(t, np.float64) for t in (x, gate, dy))
    n, c = x.shape
    batch = len(offsets) - 1
    first = np.zeros((batch, c)) if h0 is None else np.asarray(h0, np.float64)
    y, _, (ey, _) = gated_scan_fwd(x, gate, offsets, h0, reverse, form, ea)
    dx, dg, ex, eg = (np.zeros((n, c)) for _ in range(4))
    dh0 = np.zeros((batch, c)) if dlast is None else np.array(dlast, np.float64)
    eh = np.zeros((batch, c))
    for b in range(batch):
        rows = list(range(int(offsets[b]), int(offsets[b + 1])))
        if reverse:
            rows.reverse()
        d, e = dh0[b].copy(), np.zeros(c)  # what the row behind hands over
        for i in range(len(rows) - 1, -1, -1):
            t = rows[i]
            a, keep, da, dk = _sides(gate[t], ea)
            D = dy[t] + d
            eD = e + F * np.abs(D)
            prev, ep = (y[rows[i - 1]], ey[rows[i - 1]]) if i else (first[b], 0.0)
            if form == "mix":
                dx[t], ex[t] = keep * D, keep * eD + dk * (np.abs(D) + eD) + 2 * F * np.abs(keep * D)
                u, eu = prev - x[t], ep + 2 * F * np.abs(prev - x[t])
            else:
                dx[t], ex[t] = D, eD
                u, eu = prev, ep
            dg[t] = a * keep * D * u
            rel = 2 * ea + 8 * F
            eg[t] = a * keep * (eD * (np.abs(u) + eu) + np.abs(D) * eu) * (1 + rel) + rel * np.abs(dg[t])
            d = a * D
            e = a * eD + da * (np.abs(D) + eD) + 2 * F * np.abs(d)
        dh0[b], eh[b] = d, e
    return dx, dg, dh0, (ex, eg, eh)


def _windows(nq, nk, q_offsets, kv_offsets, left, right, sinks, kv_mask):
    """For each sample: its rows, its keys and the truth [rows, keys] of what a row sees."""
    for b in range(len(q_offsets) - 1):
        rows = np.arange(int(q_offsets[b]), int(q_offsets[b + 1]))
        keys = np.arange(int(kv_offsets[b]), int(kv_offsets[b + 1]))
        t = np.arange(len(rows))[:, None] + len(keys) - len(rows)
        j = np.arange(len(keys))[None, :]
        see = np.ones((len(rows), len(keys)), bool)
        if right is not None:
            see &= j <= t + right
        if left is not None:
            see &= (j >= t - left) | (j < sinks)
        if kv_mask is not None:
            see &= np.asarray(kv_mask)[keys][None, :] != 0
        yield rows, keys, see


def _attend(qh, kh, see, scale):
    """(P, lse, largest |scale| sum |q k| of a row) with P zero where nothing is seen."""
    s = np.where(see, scale * (qh @ kh.T), -np.inf)
    m = s.max(1, keepdims=True, initial=-np.inf)
    e = np.where(see, np.exp(s - np.where(np.isinf(m), 0.0, m)), 0.0)
    tot = e.sum(1, keepdims=True)
    some = tot[:, 0] > 0
    lse = np.full(len(qh), -np.inf)
    lse[some] = (m + np.log(np.where(tot > 0, tot, 1.0)))[some, 0]
    top = np.where(see, abs(scale) * (np.abs(qh) @ np.abs(kh).T), 0.0).max(1, initial=0.0)
    return e / np.where(tot > 0, tot, 1.0), lse, top


def _clean(t, kv_mask):
    t = np.array(t, np.float64)
    if kv_mask is not None:
        t[np.asarray(kv_mask) == 0] = 0.0  # a masked row is never used
    return t


def window_attention_fwd(q, k, v, q_offsets, kv_offsets, left, right, sinks=0, kv_mask=None, scale=None):
    """(out [nq, Hq, D], lse [Hq, nq], sizes): sizes as cross_attention_fwd's of the attention oracle."""
    q, k, v = np.asarray(q, np.float64), _clean(k, kv_mask), _clean(v, kv_mask)
    (nq, hq, d), (nk, hk) = q.shape, k.shape[:2]
    scale = d ** -0.5 if scale is None else scale
    out, size = np.zeros((nq, hq, d)), np.zeros((nq, hq, d))
    lse, top = np.full((hq, nq), -np.inf), np.zeros((hq, nq))
    for rows, keys, see in _windows(nq, nk, q_offsets, kv_offsets, left, right, sinks, kv_mask):
        for h in range(hq if len(rows) and len(keys) else 0):
            vh = v[keys, h * hk // hq]
            p, lse[h, rows], top[h, rows] = _attend(q[rows, h], k[keys, h * hk // hq], see, scale)
            out[rows, h] = p @ vh
            size[rows, h] = p @ np.abs(vh)
    return out, lse, (size, top)


def window_attention_bwd(q, k, v, dout, q_offsets, kv_offsets, left, right, sinks=0, kv_mask=None, scale=None, err=None):
    """(dq, dk, dv, sizes or None); err and sizes as cross_attention_bwd's of the attention oracle."""
    q, dout, k, v = np.asarray(q, np.float64), np.asarray(dout, np.float64), _clean(k, kv_mask), _clean(v, kv_mask)
    (nq, hq, d), (nk, hk) = q.shape, k.shape[:2]
    scale = d ** -0.5 if scale is None else scale
    grads, sizes = ([np.zeros_like(t) for t in (q, k, v)] for _ in range(2))
    for rows, keys, see in _windows(nq, nk, q_offsets, kv_offsets, left, right, sinks, kv_mask):
        for h in range(hq if len(rows) and len(keys) else 0):
            g = h * hk // hq
            qh, kh, vh, do = q[rows, h], k[keys, g], v[keys, g], dout[rows, h]
            p, _, _ = _attend(qh, kh, see, scale)
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
