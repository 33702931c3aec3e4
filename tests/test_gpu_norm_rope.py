"""GPU parity of ssc_qk_norm_rope_fwd / _bwd against the float64 oracle.

Tolerances are elementwise bounds.  With u half a step of the type and f = 2^-24: r's sum of D squares, its root and
division are off by (D + 8) f, an angle of up to half a turn by pi f (the reduced turns' rounding) and the sine and
cosine by 4 f, each product and sum by f, so a result is off by u of itself and (D + 32) f of the sizes it is formed
from (|u_a| + |u_b| of a pair); a weight gradient's sum over n rows and heads adds n f of its terms' sizes.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F = 2.0 ** -24


@pytest.fixture(scope="module")
def ssc():
    import sparse_submanifold_convolution_amd as m
    m.lib()
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, tol, what):
    bad = ~(np.abs(_f64(got) - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst |err|/tol "
                           f"{np.nanmax(np.abs(_f64(got) - ref) / np.maximum(tol, 1e-300)):.3g} at {np.argwhere(bad)[0]}")


def _check(ssc, seed, n, hq, hk, d, dt, pairs, layout, weight, norm=True, span=100, packed=False, eps=1e-5, theta=10000.0):
    g = torch.Generator().manual_seed(seed)
    q, dqo = (torch.randn(n, hq, d, generator=g).to(DT[dt]) for _ in range(2))
    k, dko = (torch.randn(n, hk, d, generator=g).to(DT[dt]) for _ in range(2))
    pos = torch.randint(-span, span, (n, 1 + len(pairs)), generator=g, dtype=torch.int64).to(torch.int32)
    ws = [None, None]
    if weight != "none":
        ws = [(1 + 0.3 * torch.randn((h, d) if weight == "head" else (d,), generator=g)).to(DT[dt]) for h in (hq, hk)]
    table = ssc.rope_table(pairs, theta, DEV) if pairs else None
    gq, gk = q.to(DEV), k.to(DEV)
    if packed:
        both = torch.cat([gq, gk, gk], dim=1)
        gq, gk = both[:, :hq], both[:, hq:hq + hk]
    gpos = pos.to(DEV)[:, 1:] if pairs else None  # as a coordinate tensor's columns past the sample number
    kw = dict(q_weight=None if ws[0] is None else ws[0].to(DEV), k_weight=None if ws[1] is None else ws[1].to(DEV),
              eps=eps, norm=norm, layout=layout)
    got = ssc.qk_norm_rope_fwd(gq, gk, gpos, table, **kw)
    grads = ssc.qk_norm_rope_bwd(gq, gk, gpos, table, dqo.to(DEV), dko.to(DEV), **kw)
    turns, axis = A.rope_turns(pairs, theta)
    u = torch.finfo(DT[dt]).eps / 2
    tiny = 2.0 ** -25 if dt == "f16" else 1e-30
    f = (d + 32) * F
    for x, w, dy, y, dx, dw, name in ((q, ws[0], dqo, got[0], grads[0], grads[2], "q"),
                                      (k, ws[1], dko, got[1], grads[1], grads[3], "k")):
        w = None if w is None else _f64(w)
        args = (_f64(x), w, pos[:, 1:].numpy(), turns, axis)
        ref, size = A.norm_rope_fwd(*args, eps, layout, norm)
        _within(y, ref, u * np.abs(ref) + f * size + tiny, name)
        rdx, rdw, sdx, sdw = A.norm_rope_bwd(*args, _f64(dy), eps, layout, norm)
        _within(dx, rdx, u * np.abs(rdx) + f * sdx + tiny, "d" + name)
        if w is None:
            assert dw is None
        else:
            _within(dw, rdw, u * np.abs(rdw) + (f + x.shape[0] * x.shape[1] * F) * sdw + tiny, "weight of " + name)


CASES = [  # n, heads_q, heads_kv, head_dim, pairs per axis, layout, weight
    (1, 1, 1, 8, (4,), "interleaved", "shared"),
    (1, 16, 4, 64, (10, 10, 10), "interleaved", "head"),
    (7, 3, 1, 40, (6, 7, 7), "interleaved", "shared"),
    (333, 6, 2, 64, (10, 11, 11), "halves", "head"),
    (1000, 4, 4, 96, (16, 16, 16), "halves", "shared"),
    (2050, 2, 2, 32, (5, 5, 5), "interleaved", "none"),
    (130, 5, 3, 128, (13, 20, 30), "interleaved", "head"),
    (90, 2, 1, 256, (32, 64), "halves", "head"),
    (65, 2, 2, 72, (32,), "halves", "shared"),
    (4097, 9, 3, 80, (0, 20, 20), "interleaved", "head"),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"n{c[0]}-h{c[1]}.{c[2]}-d{c[3]}-{c[5]}-{c[6]}" for c in CASES])
def test_parity(ssc, case, dt):
    n, hq, hk, d, pairs, layout, weight = case
    print(f"[norm_rope] {dt} {case}", flush=True)
    _check(ssc, 1, n, hq, hk, d, dt, pairs, layout, weight)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_far_positions_keep_their_phase(ssc, dt):
    _check(ssc, 2, 300, 2, 2, 64, dt, (10, 11, 11), "interleaved", "head", span=2 ** 31 - 1)


@pytest.mark.parametrize("norm,pairs,weight", [(False, (16, 16), "none"), (True, (), "head"), (False, (), "none")])
def test_rotation_or_norm_alone(ssc, norm, pairs, weight):
    _check(ssc, 3, 200, 4, 2, 64, "bf16", pairs, "halves", weight, norm=norm)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_packed_projection(ssc, dt):
    _check(ssc, 4, 500, 4, 2, 64, dt, (10, 10, 10), "interleaved", "head", packed=True)


def test_zero_rows_and_epsilon(ssc):
    """A row of zeros normalises to zeros; its gradient is g w / sqrt(eps)."""
    q = torch.zeros(3, 1, 64, device=DEV)
    dy = torch.ones(3, 1, 64, device=DEV)
    y, _ = ssc.qk_norm_rope_fwd(q, None, eps=2.0 ** -20)
    assert not y.any()
    dq, dk, dw, _ = ssc.qk_norm_rope_bwd(q, None, None, None, dy, None, eps=2.0 ** -20)
    assert (dq == 1024).all() and dk is None and dw is None


def test_empty_and_one_sided(ssc):
    table = ssc.rope_table((16, 16), device=DEV)
    w = torch.ones(64, device=DEV)
    q, pos = torch.empty(0, 2, 64, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    y, none = ssc.qk_norm_rope_fwd(q, None, pos, table, q_weight=w)
    assert y.shape == q.shape and none is None
    dq, _, dw, _ = ssc.qk_norm_rope_bwd(q, None, pos, table, q, None, q_weight=w)
    assert dq.shape == q.shape and not dw.any()
    k = torch.randn(5, 3, 64, device=DEV)
    pos = torch.arange(10, dtype=torch.int32, device=DEV).view(5, 2)
    both = ssc.qk_norm_rope_fwd(k, k, pos, table, q_weight=w, k_weight=w)
    alone = ssc.qk_norm_rope_fwd(None, k, pos, table, k_weight=w)[1]
    assert torch.equal(both[0], alone) and torch.equal(both[1], alone)


def test_autograd_matches_the_calls(ssc):
    g = torch.Generator(device=DEV).manual_seed(5)
    qkv = torch.randn(40, 6, 32, device=DEV, generator=g, requires_grad=True)
    w = [torch.randn(2, 32, device=DEV, generator=g).requires_grad_() for _ in range(2)]
    pos = torch.randint(0, 64, (40, 4), device=DEV, generator=g, dtype=torch.int32)
    table = ssc.rope_table((5, 5, 5), device=DEV)
    q, k = ssc.qk_norm_rope(qkv[:, :2], qkv[:, 2:4], pos[:, 1:], table, *w)
    (q.sum() + (k * k).sum()).backward()
    ref = ssc.qk_norm_rope_bwd(qkv[:, :2].detach(), qkv[:, 2:4].detach(), pos[:, 1:], table, torch.ones_like(q),
                               2 * k.detach(), w[0].detach(), w[1].detach())
    assert torch.equal(qkv.grad[:, :2], ref[0]) and torch.equal(qkv.grad[:, 2:4], ref[1]) and not qkv.grad[:, 4:].any()
    assert torch.equal(w[0].grad, ref[2]) and torch.equal(w[1].grad, ref[3])


def test_graph_replays(ssc):
    g = torch.Generator(device=DEV).manual_seed(6)
    q, dq = (torch.randn(3000, 4, 64, device=DEV, generator=g).half() for _ in range(2))
    w = torch.randn(4, 64, device=DEV, generator=g).half()
    pos = torch.randint(0, 64, (3000, 3), device=DEV, generator=g, dtype=torch.int32)
    table = ssc.rope_table((10, 11, 11), device=DEV)

    def both():
        return (*ssc.qk_norm_rope_fwd(q, q, pos, table, w, w), *ssc.qk_norm_rope_bwd(q, q, pos, table, dq, dq, w, w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for i in range(4):
        q.mul_(-1.25)
        pos.add_(i)
        graph.replay()
        torch.cuda.synchronize()
        eager = both()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)
