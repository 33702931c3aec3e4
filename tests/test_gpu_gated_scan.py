"""GPU parity of ssc_gated_scan_fwd / _bwd against the float64 oracle.

Tolerances: the oracle carries a bound on an fp32 evaluation's error along the rows (every product and sum off by
f = 2^-24, the decay by what its exponential and reciprocal are off), plus the result's rounding, u = half a step of the
type, and half of fp16's smallest step.  The smaller side q of (a, 1 - a) is off by a relative ea: the exponent's rounding
(|g| log2(e) up to |g| 2^-23.4 in e), 2^-22 of the exponential, 2^-22 of the reciprocal or division and two roundings:
ea = 2^-20 for |g| <= 8, and (8 + |g|) 2^-24 more than that for larger gates.  A tile joins the same maps in another order, whose products are off by
one f each: the bound's 2 f a row is doubled for them (a factor of 2 on the whole).
"""
import numpy as np
import pytest
import torch

from oracle import sequence as S

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ssc():
    import sparse_submanifold_convolution_amd as m
    m.lib()
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, err, what):
    u = torch.finfo(got.dtype).eps / 2
    tol = u * np.abs(ref) + 2 * (1 + u) * err + (2.0 ** -25 if got.dtype == torch.float16 else 1e-30)
    got = _f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - ref) / tol):.3g}, {np.argwhere(bad)[0]}"


def _case(seed, lens, c, dt, state=True, lead=0, tail=0):
    g = torch.Generator().manual_seed(seed)
    n = lead + sum(lens) + tail
    x, dy = (torch.randn(n, c, generator=g).to(DT[dt]) for _ in range(2))
    gate = (torch.randn(n, c, generator=g) + torch.linspace(-1, 6, c)).to(DT[dt])
    off = torch.tensor(lead + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    h0, dl = (torch.randn(len(lens), c, generator=g) if state else None for _ in range(2))
    return x, gate, dy, off, h0, dl


def _check(ssc, case, reverse=False, form="mix"):
    x, gate, dy, off, h0, dl = case
    # rows of no sample, which may hold anything, take no part and so are left out of the largest gate
    most = float(gate[off[0]:off[-1]].float().abs().max()) if off[-1] > off[0] else 0.0
    ea = 2.0 ** -20 + (8 + most) * 2.0 ** -24
    gx, gg, gdy, goff, gh0, gdl = (None if t is None else t.to(DEV) for t in case)
    y, last, carries = ssc.gated_scan_fwd(gx, gg, goff, gh0, reverse, form, need_carries=True)
    dx, dg, dh = ssc.gated_scan_bwd(gx, gg, carries, gdy, goff, gh0, gdl, reverse, form)
    nx, ng, ndy = _f64(x), _f64(gate), _f64(dy)
    nh0, ndl = (None if t is None else _f64(t) for t in (h0, dl))
    o = off.tolist()
    ry, rl, (ey, el) = S.gated_scan_fwd(nx, ng, o, nh0, reverse, form, ea)
    rx, rg, rh, (ex, eg, eh) = S.gated_scan_bwd(nx, ng, ndy, o, nh0, ndl, reverse, form, ea)
    _within(y, ry, ey, "y")
    _within(last, rl, el, "last")
    _within(dx, rx, ex, "dx")
    _within(dg, rg, eg, "dgate")
    if h0 is not None:
        _within(dh, rh, eh, "dh0")
    y2, last2, none = ssc.gated_scan_fwd(gx, gg, goff, gh0, reverse, form)
    assert torch.equal(y, y2) and torch.equal(last, last2) and none is None
    return y, last, dx, dg, dh


LENS = [[1], [2], [7], [8], [9], [127], [128], [129], [1000], [1] * 40, [0, 5, 0, 0, 300, 1, 0], [513, 700, 129], [2600]]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("reverse", [False, True])
def test_lengths(ssc, dt, lens, reverse):
    print(f"[scan] {dt} {lens} reverse {reverse}", flush=True)
    _check(ssc, _case(1, lens, 40, dt), reverse)
    _check(ssc, _case(2, lens, 136, dt, state=False), reverse, "sum")


@pytest.mark.parametrize("dt,c", [(d, c) for d in ("f32", "f16", "bf16") for c in (4, 8, 12, 32, 64, 72, 128, 200, 1024) if d == "f32" or c % 8 == 0])
def test_widths(ssc, dt, c):
    print(f"[scan] {dt} C={c}", flush=True)
    _check(ssc, _case(3, [300, 0, 41], c, dt), False, "mix")
    _check(ssc, _case(4, [600], c, dt), True, "sum")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_long(ssc, dt):
    """Many tiles and few channels."""
    print(f"[scan] long {dt}", flush=True)
    _check(ssc, _case(5, [9000, 31, 3500], 8, dt))
    _check(ssc, _case(6, [12000], 8, dt), True)


@pytest.mark.parametrize("reverse", [False, True])
def test_rows_of_no_sample(ssc, reverse):
    """Rows before the first and behind the last offset: zeros, whatever they hold."""
    x, gate, dy, off, h0, dl = _case(7, [50, 90], 64, "bf16", lead=20, tail=30)
    for t in (x, gate, dy):
        t[:20] = float("nan")
        t[-30:] = float("inf")
    y, last, dx, dg, dh = _check(ssc, (x, gate, dy, off, h0, dl), reverse)
    for t in (y, dx, dg):
        assert (t[:20] == 0).all() and (t[-30:] == 0).all()


@pytest.mark.parametrize("reverse", [False, True])
def test_samples_do_not_touch(ssc, reverse):
    """A sample of infinities and NaN leaves the others' results as they were, bit for bit."""
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(8, [200, 37, 300], 64, "f32"))
    outs = []
    for spoil in (False, True):
        if spoil:
            x[200:237], dy[210:230], gate[205] = float("nan"), float("inf"), float("nan")
            h0[1], dl[1] = float("inf"), float("nan")
        y, last, carries = ssc.gated_scan_fwd(x, gate, off, h0, reverse, need_carries=True)
        outs.append((y, last, *ssc.gated_scan_bwd(x, gate, carries, dy, off, h0, dl, reverse)))
    for a, b in zip(*outs):
        rows = [0, 2] if a.shape[0] == 3 else list(range(200)) + list(range(237, 537))
        assert torch.equal(a[rows], b[rows])
    assert torch.isnan(outs[1][0][200 if reverse else 236]).all()


def test_gates_at_the_ends(ssc):
    """Infinite gates keep or replace the state exactly; a NaN stays one."""
    x = torch.randn(6, 8, device=DEV)
    off = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    h0 = torch.randn(1, 8, device=DEV)
    gate = torch.full((6, 8), float("inf"), device=DEV)
    y, last, c = ssc.gated_scan_fwd(x, gate, off, h0, need_carries=True)
    assert torch.equal(y, h0.expand(6, 8)) and torch.equal(last, h0)
    dx, dg, dh = ssc.gated_scan_bwd(x, gate, c, torch.ones_like(x), off, h0)
    assert (dx == 0).all() and (dg == 0).all() and (dh == 6).all()
    y, last, c = ssc.gated_scan_fwd(x, -gate, off, h0, need_carries=True)
    assert torch.equal(y, x)
    dx, dg, dh = ssc.gated_scan_bwd(x, -gate, c, torch.ones_like(x), off, h0)
    assert (dx == 1).all() and (dg == 0).all() and (dh == 0).all()
    gate[2, 3] = float("nan")
    y, _, _ = ssc.gated_scan_fwd(x, gate, off, h0)
    assert torch.isnan(y[2:, 3]).all() and not torch.isnan(y[:2]).any() and not torch.isnan(y[:, :3]).any()


@pytest.mark.parametrize("form", ["mix", "sum"])
@pytest.mark.parametrize("reverse", [False, True])
def test_a_nan_gate_of_the_first_row(ssc, form, reverse):
    """With and without an initial state: a NaN decay times any state is NaN, in that channel and from that row on."""
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(16, [300, 20], 64, "f32"))
    first = 299 if reverse else 0
    gate[first, 5] = float("nan")
    for h in (None, h0):
        y, last, c = ssc.gated_scan_fwd(x, gate, off, h, reverse, form, need_carries=True)
        assert torch.isnan(y[:300, 5]).all() and torch.isnan(last[0, 5]) and torch.isnan(y).sum() == 300
        dx, dg, _ = ssc.gated_scan_bwd(x, gate, c, dy, off, h, None, reverse, form)
        # the gradient of a later row does not know of it, but every decay's gradient holds a state
        assert torch.isnan(dg[:300, 5]).all() and torch.isnan(dg).sum() == 300
        assert torch.isnan(dx).sum() == (1 if form == "mix" else 0)


def test_two_calls_at_once(ssc):
    """Calls on two streams, each with its own exchange between tiles."""
    cases = [[t.to(DEV) for t in _case(17 + i, [9000, 4000], 256, "bf16")] for i in range(2)]

    def run(case):
        x, gate, dy, off, h0, dl = case
        y, last, c = ssc.gated_scan_fwd(x, gate, off, h0, need_carries=True)
        return (y, last, *ssc.gated_scan_bwd(x, gate, c, dy, off, h0, dl))

    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_strided_and_packed(ssc):
    g = torch.Generator().manual_seed(9)
    both = torch.randn(700, 3 * 64, generator=g).to(torch.float16).to(DEV)
    off = torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)
    x, gate, dy = both[:, :64], both[:, 64:128], both[:, 128:].contiguous()
    a = ssc.gated_scan_fwd(x, gate, off, need_carries=True)
    b = ssc.gated_scan_fwd(x.contiguous(), gate.contiguous(), off, need_carries=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    ga = ssc.gated_scan_bwd(x, gate, a[2], dy, off)
    gb = ssc.gated_scan_bwd(x.contiguous(), gate.contiguous(), b[2], dy, off)
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1]) and ga[2] is None
    one = gate[:1].expand(700, 64)  # one gate for all rows
    assert torch.equal(ssc.gated_scan_fwd(x, one, off)[0], ssc.gated_scan_fwd(x, one.contiguous(), off)[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_steps_give_the_whole(ssc, dt):
    """Row by row from the last states, as while serving: the states stay fp32, so the whole call's results come out up to
    the order of its products."""
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(10, [20, 20, 20], 64, dt))
    y, last, _ = ssc.gated_scan_fwd(x, gate, off, h0)
    each = torch.arange(4, dtype=torch.int32, device=DEV)
    h, rows = h0, torch.tensor([0, 20, 40], device=DEV)
    for t in range(20):
        yt, h, _ = ssc.gated_scan_fwd(x[rows + t], gate[rows + t], each, h)
    assert torch.allclose(h, last, rtol=1e-5, atol=1e-6)
    assert torch.allclose(yt.float(), y[rows + 19].float(), rtol=2 * torch.finfo(DT[dt]).eps, atol=1e-6)


def test_no_rows(ssc):
    x = torch.empty(0, 64, device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    h0, dl = torch.randn(3, 64, device=DEV), torch.randn(3, 64, device=DEV)
    y, last, c = ssc.gated_scan_fwd(x, x, off, h0, need_carries=True)
    assert y.shape == (0, 64) and torch.equal(last, h0)
    assert (ssc.gated_scan_fwd(x, x, off)[1] == 0).all()
    dx, dg, dh = ssc.gated_scan_bwd(x, x, c, x, off, h0, dl)
    assert torch.equal(dh, dl) and dx.shape == dg.shape == (0, 64)


def test_offsets_are_taken_into_the_rows(ssc):
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(11, [100, 100], 64, "f32"))
    wild = torch.tensor([-7, 100, 999], dtype=torch.int32, device=DEV)
    for reverse in (False, True):
        outs = []
        for o in (off, wild):
            y, last, c = ssc.gated_scan_fwd(x, gate, o, h0, reverse, need_carries=True)
            outs.append((y, last, *ssc.gated_scan_bwd(x, gate, c, dy, o, h0, dl, reverse)))
        assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("reverse", [False, True])
def test_graph(ssc, reverse):
    """Captured passes over several tiles, replayed on changing inputs; two graphs take turns."""
    case = [t.to(DEV) for t in _case(12, [3000, 0, 1300], 256, "bf16")]
    x, gate, dy, off, h0, dl = case

    def step():
        y, last, c = ssc.gated_scan_fwd(x, gate, off, h0, reverse, need_carries=True)
        return (y, last, *ssc.gated_scan_bwd(x, gate, c, dy, off, h0, dl, reverse))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(4):
        x.copy_(torch.randn(x.shape, device=DEV))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs[i % 2], step()):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_results_repeat(ssc, dt):
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(13, [20000, 7000], 256, dt))
    outs = []
    for _ in range(4):
        y, last, c = ssc.gated_scan_fwd(x, gate, off, h0, need_carries=True)
        outs.append((y, last, c, *ssc.gated_scan_bwd(x, gate, c, dy, off, h0, dl)))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


def test_wrapper(ssc):
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(14, [33, 0, 200], 72, "f32"))
    leaves = [t.clone().requires_grad_() for t in (x, gate, h0)]
    _, _, c = ssc.gated_scan_fwd(x, gate, off, h0, True, "sum", need_carries=True)

    def grads(pick):
        y, last = ssc.gated_scan(leaves[0], leaves[1], off, leaves[2], True, "sum")
        return torch.autograd.grad(pick(y, last), leaves)

    got = grads(lambda y, last: (y * dy).sum() + (last * dl).sum())
    assert all(torch.equal(a, b) for a, b in zip(got, ssc.gated_scan_bwd(x, gate, c, dy, off, h0, dl, True, "sum")))
    got = grads(lambda y, last: (y * dy).sum())
    assert all(torch.equal(a, b) for a, b in zip(got, ssc.gated_scan_bwd(x, gate, c, dy, off, h0, None, True, "sum")))
    got = grads(lambda y, last: (last * dl).sum())
    assert all(torch.equal(a, b) for a, b in
               zip(got, ssc.gated_scan_bwd(x, gate, c, torch.zeros_like(dy), off, h0, dl, True, "sum")))
    # views that start anywhere, transposed ones, and a gradient that is a broadcast
    odd = torch.randn(233 * 72 + 1, device=DEV)[1:].view(233, 72).requires_grad_()
    ssc.gated_scan(odd, odd.t().contiguous().t(), off)[0].sum().backward()
    assert torch.isfinite(odd.grad).all()


def test_gradient_is_the_difference(ssc):
    """A directional difference of a loss of order one in fp32: the fourth-order difference with steps of 2^-5 along a
    direction of unit size is off by the step's fourth power and the fp32 loss's rounding over the step, both below one part
    in a hundred of the slope along the gradient itself."""
    x, gate, dy, off, h0, dl = (t.to(DEV) for t in _case(15, [90, 60], 64, "f32"))
    leaves = [t.clone().requires_grad_() for t in (x, gate, h0)]

    def loss(a, b, c):
        y, last = ssc.gated_scan(a, b, off, c)
        return (y.double() * dy.double()).mean() + (last.double() ** 2).mean()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in grads)).item()
    vals = {}
    for s in (-2, -1, 1, 2):
        with torch.no_grad():
            vals[s] = loss(*[t + (s * 2.0 ** -5 * g / norm) for t, g in zip((x, gate, h0), grads)]).item()
    slope = (8 * (vals[1] - vals[-1]) - (vals[2] - vals[-2])) / (12 * 2.0 ** -5)
    assert abs(slope - norm) <= 0.01 * norm
