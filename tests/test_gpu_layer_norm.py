"""GPU parity of ssc_layer_norm_fwd / _bwd and ssc_dropout against the float64 oracle.

A tolerance is the oracle's bound on the fp32 evaluation's error (sums of C or n terms in any order, f = 2^-24 each) plus
the result's own rounding: u = half a step of the type (bf16 2^-8, fp16 2^-11, fp32 2^-24) relative to the value, and half
of fp16's smallest step (2^-25).
"""
import numpy as np
import pytest
import torch

from oracle import sequence as S

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


def _rng(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device=DEV)


def _within(got, ref, err, what):
    u = torch.finfo(got.dtype).eps / 2
    tol = u * np.abs(ref) + (1 + u) * err + (2.0 ** -25 if got.dtype == torch.float16 else 1e-36)
    got = _f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - ref) / tol):.3g}"


def _inputs(seed, n, c, dt, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x, res, dy, ds = ((offset + torch.randn(n, c, generator=g)).to(DT[dt]) for _ in range(4))
    w, b = ((1 + 0.3 * torch.randn(c, generator=g)).to(DT[dt]) for _ in range(2))
    return x, res, dy, ds, w, b


def _check(ssc, n, c, dt, affine=True, residual=False, p=0.0, offset=0.0, eps=1e-5):
    x, res, dy, ds, w, b = _inputs(n + c, n, c, dt, offset)
    if not affine:
        w = b = None
    gx, gres, gdy, gds, gw, gb = (None if t is None else t.to(DEV) for t in (x, res, dy, ds, w, b))
    nw, nb = (None if t is None else _f64(t) for t in (w, b))
    if not residual:
        y = ssc.layer_norm_fwd(gx, gw, gb, eps)
        dx, dw, db = ssc.layer_norm_bwd(gx, gdy, gw, gb, eps)
        s, up, factor = _f64(x), None, 1.0
    else:
        drop = dict(p=p, rng=_rng(n, 5 << 33), layer=2)
        y, gs = ssc.add_layer_norm_fwd(gx, gres, gw, gb, eps, **drop)
        dx, dr, dw, db = ssc.add_layer_norm_bwd(gs, gdy, gds, gw, gb, eps, **drop)
        factor = S.dropout_factor(n * c, p, n, 5 << 33, 2).reshape(n, c)
        s = factor * _f64(x) + _f64(res)
        _within(gs, s, F * (2 * np.abs(factor * _f64(x)) + np.abs(s)), "s")
        up = _f64(ds)
    ry, ey = S.layer_norm_fwd(s, nw, nb, eps)
    if residual:  # s itself is formed in fp32: the oracle's bound has 3 f |s| for it, of the terms rather than of their sum
        r = 1.0 / np.sqrt(s.var(1, keepdims=True) + eps)
        es = 3 * F * (np.abs(factor * _f64(x)) + np.abs(_f64(res)))
        ey = ey + r * (1.0 if nw is None else np.abs(nw)) * (es + es.mean(1, keepdims=True) * (1 + np.abs(ry)))
    _within(y, ry, ey, "y")
    back = _f64(gs) if residual else s
    rdx, rdw, rdb, (edx, edw, edb) = S.layer_norm_bwd(back, _f64(dy), nw, eps, up)
    if residual:
        _within(dr, rdx, edx, "dresidual")
        assert (dx is dr) == (p == 0)
    _within(dx, factor * rdx, factor * edx + 2 * F * np.abs(factor * rdx), "dx")
    if affine:
        _within(dw, rdw, edw, "dweight")
        _within(db, rdb, edb, "dbias")
    else:
        assert dw is None and db is None


# every form of a row: parts of a wave, whole waves with one, two and four vectors a lane, workgroups with two, four, eight
WIDTHS = {"f32": [4, 20, 40, 64, 100, 256, 260, 512, 1000, 1028, 2048, 2052, 4096, 4100, 8192],
          "f16": [8, 24, 40, 64, 200, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192],
          "bf16": [8, 32, 72, 128, 256, 488, 768, 1024, 1536, 2040, 2504, 4096, 6000, 8192]}
CASES = [(dt, c) for dt in WIDTHS for c in WIDTHS[dt]]


@pytest.mark.parametrize("dt,c", CASES)
def test_plain(ssc, dt, c):
    print(f"[norm] {dt} C={c}", flush=True)
    _check(ssc, 37, c, dt)


@pytest.mark.parametrize("dt,c", CASES)
def test_residual(ssc, dt, c):
    print(f"[norm+residual] {dt} C={c}", flush=True)
    _check(ssc, 5, c, dt, residual=True, affine=c % 16 == 0)


@pytest.mark.parametrize("dt,c", CASES)
def test_residual_and_dropout(ssc, dt, c):
    print(f"[norm+residual+dropout] {dt} C={c}", flush=True)
    _check(ssc, 3, c, dt, residual=True, p=0.3)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 5000])
def test_rows(ssc, dt, n):
    """One row, a wave's worth and one past it, and more rows than the backward grid has groups."""
    _check(ssc, n, 40, dt)
    _check(ssc, n, 8, dt, affine=False)


def test_more_rows_than_the_grid(ssc):
    _check(ssc, 2048 * 4 + 5, 512, "bf16")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_rows_far_from_zero(ssc, dt):
    _check(ssc, 50, 128, dt, offset=100.0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_constant_rows(ssc, dt):
    """No variance: y is the bias, and the gradient stays finite through eps."""
    x = torch.full((3, 64), 1.5, dtype=DT[dt], device=DEV)
    b = torch.arange(64, device=DEV).to(DT[dt])
    assert torch.equal(ssc.layer_norm_fwd(x, None, b), b.expand(3, 64))
    dx, _, db = ssc.layer_norm_bwd(x, torch.ones_like(x), None, b)
    assert torch.isfinite(dx).all() and (db == 3).all()


def test_no_rows(ssc):
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    assert ssc.layer_norm_fwd(x, w, w).shape == (0, 64)
    dx, dw, db = ssc.layer_norm_bwd(x, x, w, w)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    y, s = ssc.add_layer_norm_fwd(x, x, w, w, p=0.5, rng=_rng(1, 1))
    assert y.shape == s.shape == (0, 64)
    assert ssc.dropout_fwd(x, 0.5, _rng(1, 1)).shape == (0, 64)


def test_strided_rows(ssc):
    """Rows of a packed projection, and one row broadcast to all."""
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(20, 3 * 64, generator=g).to(torch.bfloat16).to(DEV)
    x, r = wide[:, 64:128], wide[:, 128:]
    assert torch.equal(ssc.layer_norm_fwd(x), ssc.layer_norm_fwd(x.contiguous()))
    for a, b in zip(ssc.add_layer_norm_fwd(x, r), ssc.add_layer_norm_fwd(x.contiguous(), r.contiguous())):
        assert torch.equal(a, b)
    dy = torch.randn(20, 64, generator=g).to(torch.bfloat16).to(DEV)
    assert torch.equal(ssc.layer_norm_bwd(x, dy)[0], ssc.layer_norm_bwd(x.contiguous(), dy)[0])
    one = wide[:1, :64].expand(20, 64)
    assert torch.equal(ssc.layer_norm_fwd(one), ssc.layer_norm_fwd(one.contiguous()))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (3, 5, 7), (1000, 33), (257, 64)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(ssc, dt, shape, residual):
    g = torch.Generator().manual_seed(len(shape))
    x, r = (torch.randn(*shape, generator=g).to(DT[dt]) for _ in range(2))
    seed, step, p = (1 << 62) + 12345, (7 << 32) + 3, 0.37
    y = ssc.dropout_fwd(x.to(DEV), p, _rng(seed, step), 9, r.to(DEV) if residual else None)
    f = S.dropout_factor(x.numel(), p, seed, step, 9).reshape(shape)
    ref = f * _f64(x) + (_f64(r) if residual else 0)
    _within(y, ref, 3 * F * (np.abs(f * _f64(x)) + np.abs(ref)), "y")
    if not residual:
        assert np.array_equal(_f64(y) != 0, (f * _f64(x)) != 0)
        assert torch.equal(ssc.dropout_bwd(x.to(DEV), p, _rng(seed, step), 9), y)


def test_dropout_edges(ssc):
    x = torch.randn(1000, 8, device=DEV)
    assert torch.equal(ssc.dropout_fwd(x, 0.0), x)
    assert torch.equal(ssc.dropout_fwd(x, 2.0 ** -18, _rng(1, 1)), x)         # rounds to nothing dropped
    y = ssc.dropout_fwd(x, 0.999999, _rng(-5, -1))                           # held below one; negative words are words
    f = S.dropout_factor(8000, 0.999999, -5, -1, 0).reshape(1000, 8)
    assert np.array_equal(_f64(y) != 0, f != 0)
    # what a dropped element holds does not matter
    x[:] = float("nan")
    y = ssc.dropout_fwd(x, 0.5, _rng(3, 4))
    f = S.dropout_factor(8000, 0.5, 3, 4, 0).reshape(1000, 8)
    assert np.array_equal(np.isnan(_f64(y)), f != 0) and (_f64(y)[f == 0] == 0).all()
    y, s = ssc.add_layer_norm_fwd(x, torch.ones_like(x), p=0.5, rng=_rng(3, 4))
    assert np.array_equal(np.isnan(_f64(s)), f != 0)


def test_dropout_follows_its_rng_in_a_graph(ssc):
    """A captured call reads seed and step when it is replayed."""
    x = torch.randn(4096, 40, device=DEV)
    res, w = torch.randn_like(x), torch.randn(40, device=DEV)
    rng = _rng(11, 0)
    ssc.add_layer_norm_bwd(*ssc.add_layer_norm_fwd(x, res, w, w, p=0.2, rng=rng)[::-1], None, w, w, p=0.2, rng=rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = ssc.dropout_fwd(x, 0.2, rng, 1)
        y, s = ssc.add_layer_norm_fwd(x, res, w, w, p=0.2, rng=rng)
        grads = ssc.add_layer_norm_bwd(s, y, d, w, w, p=0.2, rng=rng)
    for step in range(4):
        rng.copy_(_rng(11, step))
        graph.replay()
        torch.cuda.synchronize()
        ed = ssc.dropout_fwd(x, 0.2, _rng(11, step), 1)
        ey, es = ssc.add_layer_norm_fwd(x, res, w, w, p=0.2, rng=_rng(11, step))
        eg = ssc.add_layer_norm_bwd(es, ey, ed, w, w, p=0.2, rng=_rng(11, step))
        for a, b in zip((d, y, s, *grads), (ed, ey, es, *eg)):
            assert torch.equal(a, b), step


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_results_repeat(ssc, dt):
    x, res, dy, ds, w, b = (t.to(DEV) for t in _inputs(4, 9001, 136, dt))
    first = ssc.add_layer_norm_bwd(x, dy, ds, w, b, p=0.1, rng=_rng(1, 2))
    for _ in range(3):
        for a, c in zip(first, ssc.add_layer_norm_bwd(x, dy, ds, w, b, p=0.1, rng=_rng(1, 2))):
            assert torch.equal(a, c)


def test_wrappers(ssc):
    """The differentiable calls give the raw calls' gradients, whatever part of the outputs is used."""
    x, res, dy, ds, w, b = (t.to(DEV) for t in _inputs(5, 33, 72, "f32"))
    rng = _rng(6, 7)
    leaves = [t.clone().requires_grad_() for t in (x, res, w, b)]

    def grads(loss):
        return torch.autograd.grad(loss, leaves, allow_unused=True)

    y, s = ssc.add_layer_norm(*leaves, 1e-5, 0.25, rng, 3)
    got = grads((y * dy).sum() + (s * ds).sum())
    want = ssc.add_layer_norm_bwd(s.detach(), dy, ds, w, b, 1e-5, 0.25, rng, 3)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    y, s = ssc.add_layer_norm(*leaves, 1e-5, 0.25, rng, 3)
    want = ssc.add_layer_norm_bwd(s.detach(), dy, None, w, b, 1e-5, 0.25, rng, 3)
    assert all(torch.equal(a, c) for a, c in zip(grads((y * dy).sum()), want))
    for p in (0.0, 0.25):
        y, s = ssc.add_layer_norm(*leaves, 1e-5, p, rng, 3)
        got = grads((s * ds).sum())
        assert torch.equal(got[0], ssc.dropout_bwd(ds, p, rng, 3)) and torch.equal(got[1], ds) and got[2] is None
    y, s = ssc.add_layer_norm(*leaves)
    got = grads((y * dy).sum() + (s * ds).sum())
    assert torch.equal(got[0], got[1])
    got = grads((ssc.layer_norm(leaves[0], leaves[2], leaves[3]) * dy).sum())
    want = ssc.layer_norm_bwd(x, dy, w, b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[1]) and torch.equal(got[3], want[2])
    got = grads((ssc.dropout(leaves[0], 0.25, rng, 3, leaves[1]) * dy).sum())
    assert torch.equal(got[0], ssc.dropout_bwd(dy, 0.25, rng, 3)) and torch.equal(got[1], dy)
    # views that start anywhere in their buffers
    odd = torch.randn(33 * 72 + 1, device=DEV)[1:].view(33, 72).requires_grad_()
    (ssc.dropout(odd, 0.25, rng) * dy).sum().backward()
    (ssc.layer_norm(odd, odd[0].detach()) * dy).sum().backward()
    # rng may not change between the passes
    y = ssc.dropout(leaves[0], 0.25, rng)
    rng.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_another_stream(ssc):
    x = torch.randn(2000, 256, device=DEV)
    want = ssc.layer_norm_fwd(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ssc.layer_norm_fwd(x)
    side.synchronize()
    assert torch.equal(got, want)
