"""Pins of the oracle of the operators over serialised rows: published values, hand values, torch float64, differences."""
import numpy as np
import pytest
import torch

from oracle import sequence as S


def test_philox_known_answers():
    """The generator's published test vectors (ten rounds)."""
    assert S.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert S.philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert S.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_factor():
    f = S.dropout_factor(4003, 0.25, 7, 9, 1)
    assert set(np.unique(f)) == {0.0, 4 / 3}
    kept = (f > 0).mean()
    assert abs(kept - 0.75) < 5 * np.sqrt(0.75 * 0.25 / 4003)          # five standard deviations of a fair choice
    assert np.array_equal(S.dropout_factor(100, 0.25, 7, 9, 1), f[:100])  # an element's choice is its own
    for other in ((8, 9, 1), (7, 10, 1), (7, 9, 2), (7 + (1 << 40), 9, 1), (7, 9 + (1 << 40), 1)):
        assert not np.array_equal(S.dropout_factor(4003, 0.25, *other), f)
    assert (S.dropout_factor(9, 0.0, 1, 1, 0) == 1).all() and (S.dropout_factor(9, 2.0 ** -18, 1, 1, 0) == 1).all()
    assert S.dropout_threshold(0.9999999) == 65535 and S.dropout_threshold(0.5) == 32768


def test_layer_norm_hand():
    y, _ = S.layer_norm_fwd([[1.0, 3.0]], [2.0, 2.0], [0.5, 0.0], 0.0)
    assert np.allclose(y, [[-1.5, 2.0]])


@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_against_torch(affine):
    g = np.random.default_rng(1)
    x, dy, ds = (g.standard_normal((7, 12)) for _ in range(3))
    w, b = (g.standard_normal(12), g.standard_normal(12)) if affine else (None, None)
    tx = torch.tensor(x, requires_grad=True)
    tw, tb = (torch.tensor(t, requires_grad=True) if affine else None for t in (w, b))
    ty = torch.nn.functional.layer_norm(tx, (12,), tw, tb, 1e-5)
    ((ty * torch.tensor(dy)).sum() + (tx * torch.tensor(ds)).sum()).backward()
    y, _ = S.layer_norm_fwd(x, w, b, 1e-5)
    dx, dw, db, _ = S.layer_norm_bwd(x, dy, w, 1e-5, ds)
    assert np.allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dx, tx.grad.numpy(), rtol=1e-11, atol=1e-12)
    if affine:
        assert np.allclose(dw, tw.grad.numpy(), rtol=1e-12) and np.allclose(db, tb.grad.numpy(), rtol=1e-12)


def test_layer_norm_gradient_is_the_difference():
    g = np.random.default_rng(2)
    x, dy, w, dirn = g.standard_normal((3, 8)), g.standard_normal((3, 8)), g.standard_normal(8), g.standard_normal((3, 8))
    h = 1e-5
    up, down = (S.layer_norm_fwd(x + s * h * dirn, w, None, 1e-5)[0] for s in (1, -1))
    dx = S.layer_norm_bwd(x, dy, w, 1e-5)[0]
    assert abs(((up - down) * dy).sum() / (2 * h) - (dx * dirn).sum()) < 1e-8 * np.abs(dx).sum()


def _scan_torch(x, gate, offsets, h0, reverse, form):
    ys, last = [None] * len(x), []
    for b in range(len(offsets) - 1):
        h = h0[b]
        rows = range(offsets[b], offsets[b + 1])
        for t in (reversed(rows) if reverse else rows):
            a = torch.sigmoid(gate[t])
            h = a * h + ((1 - a) * x[t] if form == "mix" else x[t])
            ys[t] = h
        last.append(h)
    return torch.stack(ys), torch.stack(last)


def test_scan_hand():
    y, last, _ = S.gated_scan_fwd([[2.0], [4.0]], [[0.0], [0.0]], [0, 2], [[8.0]])
    assert np.allclose(y, [[5.0], [4.5]]) and np.allclose(last, [[4.5]])
    y, last, _ = S.gated_scan_fwd([[2.0], [4.0]], [[0.0], [0.0]], [0, 2], None, True, "sum")
    assert np.allclose(y, [[4.0], [4.0]]) and np.allclose(last, [[4.0]])


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("form", ["mix", "sum"])
def test_scan_against_torch(reverse, form):
    g = np.random.default_rng(3)
    off = [0, 4, 4, 9]
    x, gate, dy = (g.standard_normal((9, 3)) for _ in range(3))
    h0, dl = (g.standard_normal((3, 3)) for _ in range(2))
    tx, tg, th = (torch.tensor(t, requires_grad=True) for t in (x, gate, h0))
    ty, tl = _scan_torch(tx, tg, off, th, reverse, form)
    ((ty * torch.tensor(dy)).sum() + (tl * torch.tensor(dl)).sum()).backward()
    y, last, _ = S.gated_scan_fwd(x, gate, off, h0, reverse, form)
    dx, dg, dh, _ = S.gated_scan_bwd(x, gate, dy, off, h0, dl, reverse, form)
    for a, b in ((y, ty), (last, tl), (dx, tx.grad), (dg, tg.grad), (dh, th.grad)):
        assert np.allclose(a, b.detach().numpy(), rtol=1e-12, atol=1e-13)


def test_scan_gradient_is_the_difference():
    g = np.random.default_rng(4)
    off = [0, 6]
    x, gate, dy, dirn = (g.standard_normal((6, 4)) for _ in range(4))
    h = 1e-5
    up, down = (S.gated_scan_fwd(x, gate + s * h * dirn, off)[0] for s in (1, -1))
    dg = S.gated_scan_bwd(x, gate, dy, off)[1]
    assert abs(((up - down) * dy).sum() / (2 * h) - (dg * dirn).sum()) < 1e-8 * np.abs(dg).sum()


WINDOWS = [(0, 0, 0), (2, 0, 0), (1, 2, 1), (None, 0, 0), (0, None, 2), (None, None, 0), (3, 1, 4)]


@pytest.mark.parametrize("window", WINDOWS, ids=str)
@pytest.mark.parametrize("masked", [False, True])
def test_window_attention_against_torch(window, masked):
    """Against softmax over a dense truth table, built entry by entry, and its autograd; more rows than keys in one sample."""
    left, right, sinks = window
    g = np.random.default_rng(5)
    qo, ko = [0, 5, 5, 9, 13], [0, 5, 8, 15, 17]
    q, do = g.standard_normal((13, 4, 8)), g.standard_normal((13, 4, 8))
    k, v = g.standard_normal((17, 2, 8)), g.standard_normal((17, 2, 8))
    mask = np.ones(17, bool)
    if masked:
        mask[[1, 2, 9, 16]] = False
    see = np.zeros((13, 17), bool)
    for b in range(4):
        for i in range(qo[b + 1] - qo[b]):
            t = i + (ko[b + 1] - ko[b]) - (qo[b + 1] - qo[b])
            for j in range(ko[b + 1] - ko[b]):
                see[qo[b] + i, ko[b] + j] = (right is None or j <= t + right) and (left is None or j >= t - left or j < sinks) \
                    and mask[ko[b] + j]
    tq, tk, tv = (torch.tensor(t, requires_grad=True) for t in (q, k, v))
    s = torch.einsum("ihd,jhd->hij", tq, tk.repeat_interleave(2, 1)) * 8 ** -0.5
    s = s.masked_fill(~torch.tensor(see), float("-inf"))
    some = torch.tensor(see.any(1))
    p = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], s, torch.zeros_like(s)), -1), torch.zeros_like(s))
    to = torch.einsum("hij,jhd->ihd", p, tv.repeat_interleave(2, 1))
    (to * torch.tensor(do)).sum().backward()
    args = (qo, ko, left, right, sinks, mask if masked else None)
    out, lse, _ = S.window_attention_fwd(q, k, v, *args)
    assert np.allclose(out, to.detach().numpy(), atol=1e-13)
    assert np.array_equal(np.isinf(lse), np.broadcast_to(~see.any(1), (4, 13)))
    want = torch.logsumexp(s, -1).detach().numpy()
    assert np.allclose(lse[:, see.any(1)], want[:, see.any(1)])
    dq, dk, dv, _ = S.window_attention_bwd(q, k, v, do, *args)
    for a, b in ((dq, tq), (dk, tk), (dv, tv)):
        assert np.allclose(a, b.grad.numpy(), atol=1e-12)


def test_unbounded_window_is_cross_attention():
    from oracle import attention as A
    g = np.random.default_rng(6)
    q, k, v, do = (g.standard_normal((n, h, 8)) for n, h in ((7, 2), (9, 1), (9, 1), (7, 2)))
    off = ([0, 3, 7], [0, 4, 9])
    for a, b in zip(S.window_attention_fwd(q, k, v, *off, None, None)[:2], A.cross_attention_fwd(q, k, v, *off)[:2]):
        assert np.allclose(a, b)
    for a, b in zip(S.window_attention_bwd(q, k, v, do, *off, None, None)[:3], A.cross_attention_bwd(q, k, v, do, *off)[:3]):
        assert np.allclose(a, b)
