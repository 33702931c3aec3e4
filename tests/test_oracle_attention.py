"""The voxel-attention oracle against hand values, torch's float64 autograd on dense masked forms, and differences."""
import numpy as np
import pytest
import torch

from oracle import attention as A


def _ragged(seed, q_lens, kv_lens, hq, hk, d):
    rng = np.random.default_rng(seed)
    q, k, v, do = (rng.standard_normal((n, h, d)) for n, h in
                   ((sum(q_lens), hq), (sum(kv_lens), hk), (sum(kv_lens), hk), (sum(q_lens), hq)))
    off = [np.concatenate([[0], np.cumsum(x)]) for x in (q_lens, kv_lens)]
    return q, k, v, do, off[0], off[1]


def test_rotation_hand_values():
    # a quarter turn per unit: (1, 0) -> (0, 1) at position 1, (-1, 0) at 2; the dimension past the pairs stays
    x = np.array([[[1.0, 0.0, 5.0]], [[1.0, 0.0, 6.0]]])
    y = A.rotate(x, np.array([[1], [2]]), np.array([0.25]), np.array([0]), "interleaved")
    assert np.allclose(y, [[[0, 1, 5]], [[-1, 0, 6]]], atol=1e-15)
    x = np.array([[[1.0, 2.0, 0.0, 0.0]]])
    y = A.rotate(x, np.array([[1, 3]]), np.array([0.25, 0.25]), np.array([0, 1]), "halves")
    assert np.allclose(y, [[[0, 0, 1, -2]]], atol=1e-14)
    # whole turns at a far position
    assert np.allclose(A.rotate(x, np.array([[2**31 - 4, -2**31]]), np.array([0.25, 0.25]), np.array([0, 1]), "halves"), x)


def test_norm_hand_values():
    y, _ = A.norm_rope_fwd(np.array([[[3.0, 4.0]]]), np.array([1.0, 2.0]), None, [], [], 0.0)
    assert np.allclose(y, [[[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]])


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("weight", ["none", "shared", "head"])
def test_norm_rope_gradients_are_differences(layout, weight):
    rng = np.random.default_rng(3)
    n, h, d = 3, 2, 8
    x, dy = rng.standard_normal((2, n, h, d))
    w = {"none": None, "shared": rng.standard_normal(d), "head": rng.standard_normal((h, d))}[weight]
    pos = rng.integers(-50, 50, (n, 2))
    turns, axis = A.rope_turns((2, 1))
    dx, dw, _, _ = A.norm_rope_bwd(x, w, pos, turns, axis, dy, 1e-3, layout)

    def loss(x, w):
        return (A.norm_rope_fwd(x, w, pos, turns, axis, 1e-3, layout)[0] * dy).sum()

    step = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dx[i]) < 1e-8
    for i in np.ndindex(w.shape) if w is not None else ():
        e = np.zeros_like(w)
        e[i] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[i]) < 1e-8


def test_attention_hand_values():
    # two keys with equal scores average the values; a third, masked, holds NaN
    q = np.ones((1, 1, 2))
    k = np.array([[[1.0, 0]], [[0, 1.0]], [[np.nan, np.inf]]])
    v = np.array([[[2.0, 0]], [[4.0, 6]], [[np.nan, np.nan]]])
    out, lse, _ = A.cross_attention_fwd(q, k, v, [0, 1], [0, 3], [1, 1, 0], scale=2.0)
    assert np.allclose(out, [[[3, 3]]]) and np.allclose(lse, 2 + np.log(2))


def test_empty_samples_give_zeros():
    q, k, v, do, qo, ko = _ragged(1, [2, 3, 0, 1], [4, 0, 2, 3], 2, 1, 4)
    mask = np.array([1, 1, 0, 1, 1, 1, 0, 0, 0])
    out, lse, _ = A.cross_attention_fwd(q, k, v, qo, ko, mask)
    assert (out[2:] == 0).all() and (lse[:, 2:] == -np.inf).all() and np.isfinite(lse[:, :2]).all()
    dq, dk, dv, _ = A.cross_attention_bwd(q, k, v, do, qo, ko, mask)
    assert (dq[2:] == 0).all() and (dk[[2, 4, 5, 6, 7, 8]] == 0).all() and (dv[[2, 4, 5, 6, 7, 8]] == 0).all()
    assert (dk[0] != 0).all()


@pytest.mark.parametrize("hq,hk", [(2, 2), (6, 2), (4, 1)])
def test_attention_matches_dense_autograd(hq, hk):
    """One dense [rows, keys] score matrix with the samples and the mask as a -inf pattern, torch float64 autograd."""
    q, k, v, do, qo, ko = _ragged(2, [5, 1, 7], [3, 9, 4], hq, hk, 6)
    mask = np.random.default_rng(5).random(16) < 0.7
    mask[0] = True
    scale = 0.3
    tq, tk, tv = (torch.tensor(t, requires_grad=True) for t in (q, k, v))
    qs = np.repeat(np.arange(3), np.diff(qo))
    ks = np.repeat(np.arange(3), np.diff(ko))
    keep = torch.tensor((qs[:, None] == ks[None]) & mask[None])
    kk, vv = (t.repeat_interleave(hq // hk, dim=1) for t in (tk, tv))
    s = (tq.transpose(0, 1) @ kk.permute(1, 2, 0)) * scale
    s = s.masked_fill(~keep, float("-inf"))
    o = (torch.softmax(s, -1) @ vv.transpose(0, 1)).transpose(0, 1)
    o.backward(torch.tensor(do))
    out, lse, _ = A.cross_attention_fwd(q, k, v, qo, ko, mask, scale)
    assert np.allclose(out, o.detach().numpy(), atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(s, -1).detach().numpy(), atol=1e-13)
    for got, ref in zip(A.cross_attention_bwd(q, k, v, do, qo, ko, mask, scale), (tq, tk, tv)):
        assert np.allclose(got, ref.grad.numpy(), atol=1e-12)


def test_attention_gradients_are_differences():
    q, k, v, do, qo, ko = _ragged(4, [2, 1], [3, 2], 2, 1, 4)
    grads = A.cross_attention_bwd(q, k, v, do, qo, ko)[:3]
    step = 1e-6
    for which, g in enumerate(grads):
        for i in np.ndindex(g.shape):
            t = [np.array(x) for x in (q, k, v)]
            t[which][i] += step
            up = (A.cross_attention_fwd(*t, qo, ko)[0] * do).sum()
            t[which][i] -= 2 * step
            down = (A.cross_attention_fwd(*t, qo, ko)[0] * do).sum()
            assert abs((up - down) / (2 * step) - g[i]) < 1e-8
