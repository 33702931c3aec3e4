"""GPU parity of ssc_window_attn_fwd / _bwd against the float64 oracle.

Tolerances are the elementwise bounds of the cross attention tests, whose arithmetic these kernels share.  With u half a
step of the type (bf16 2^-8, fp16 2^-11, fp32 2^-24), f = 2^-24 and, per row, T = max_j scale sum_d |q k_j| over the keys it
sees: a score is off by at most (D + 4) f T, its exponent's rounding by 2 f T more, the exponential itself by 2^-22, so a
probability (and the sum it is divided by) by a relative ep = 2 (D + 8) f T + 2^-21; the sums of n terms add n f;
probabilities and dS are rounded to the type for the second product (u each; none for fp32); the result is rounded once.
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


def _offsets(lens, lead=0):
    return torch.tensor(lead + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def _inputs(seed, q_lens, kv_lens, hq, hk, d, dt, masked=False):
    g = torch.Generator().manual_seed(seed)
    nq, nk = sum(q_lens), sum(kv_lens)
    q, do = (torch.randn(nq, hq, d, generator=g).to(DT[dt]) for _ in range(2))
    k, v = (torch.randn(nk, hk, d, generator=g).to(DT[dt]) for _ in range(2))
    mask = torch.rand(nk, generator=g) < 0.7 if masked else None
    if masked:
        k[~mask], v[~mask] = float("nan"), float("inf")
    return q, k, v, do, _offsets(q_lens), _offsets(kv_lens), mask


def _within(got, ref, tol, what):
    got = _f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst |err|/tol "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} at {np.argwhere(bad)[0]}")


def _check(ssc, case, window, views=None, scale=None):
    q, k, v, do, qo, ko, m = case
    dt = {v: k for k, v in DT.items()}[q.dtype]
    u, d = torch.finfo(q.dtype).eps / 2, q.shape[2]
    up = 0.0 if dt == "f32" else u
    gq, gk, gv, gdo, gqo, gko, gm = (None if t is None else t.to(DEV) for t in case)
    if views:
        gq, gk, gv = views(gq, gk, gv)
    where = (gqo, gko, *window, gm, scale)
    out, lse = ssc.window_attention_fwd(gq, gk, gv, *where)
    args = (_f64(q), _f64(k), _f64(v))
    nwhere = (qo.tolist(), ko.tolist(), *window, None if m is None else m.numpy(), scale)
    ref, rlse, (size, top) = S.window_attention_fwd(*args, *nwhere)
    n = int((ko[1:] - ko[:-1]).max())
    t = top.T[:, :, None]
    ep, es = 2 * (d + 8) * F * t + 2.0 ** -21, n * F
    eo = u * np.abs(ref) + (up + 2 * ep + 2 * es + 8 * F) * size
    tiny = 2.0 ** -25 if dt == "f16" else 1e-30  # half of fp16's smallest step
    _within(out, ref, eo + tiny, "out")
    glse = _f64(lse)
    assert np.array_equal(np.isinf(glse), np.isinf(rlse)) and not np.isnan(glse).any()
    fin = np.isfinite(rlse)
    tol = ep[:, :, 0].T + es + 8 * F * (1 + np.abs(np.where(fin, rlse, 0)) + top)
    assert (np.abs(glse[fin] - rlse[fin]) <= tol[fin]).all()
    grads = ssc.window_attention_bwd(gq, gk, gv, out, lse, gdo, *where)
    nb = max(n, int((qo[1:] - qo[:-1]).max()) * (q.shape[1] // k.shape[1]))
    p_err = (3 * ep.max() if ep.size else 0) + (nb + d + 16) * F * 2 + 8 * F * (np.abs(rlse[fin]).max() if fin.any() else 0)
    *want, sizes = S.window_attention_bwd(*args, _f64(do), *nwhere, err=(p_err, up, eo))
    for got, r, e, what in zip(grads, want, sizes, ("dq", "dk", "dv")):
        _within(got, r, u * np.abs(r) + e + tiny, what)
    return (out, lse, *grads)


CASES = [  # q_lens, kv_lens, heads_q, heads_kv, head_dim, (left, right, sinks), masked
    ([1], [1], 1, 1, 8, (0, 0, 0), False),
    ([1], [257], 8, 2, 64, (100, 0, 4), False),                    # one new row
    ([1, 1, 3], [4097, 63, 64], 4, 4, 64, (1000, 0, 2), False),
    ([5], [9000], 2, 1, 64, (4000, 0, 70), True),                  # few rows over many keys: splits
    ([300], [300], 2, 2, 64, (0, 0, 0), False),                    # a row sees itself alone
    ([300], [300], 2, 2, 64, (0, 0, 1), False),
    ([700], [700], 4, 2, 64, (64, 64, 0), False),
    ([700], [700], 4, 2, 64, (63, 65, 3), True),
    ([129, 0, 640, 1], [129, 5, 640, 1], 6, 2, 40, (100, 0, 1), True),
    ([513], [513], 2, 2, 32, (7, 3, 33), False),
    ([200], [200], 1, 1, 96, (None, 0, 0), False),                 # causal
    ([333], [333], 2, 1, 128, (None, 0, 5), True),
    ([260], [260], 2, 2, 72, (0, None, 0), False),
    ([260], [260], 2, 1, 80, (None, None, 3), True),               # no bounds
    ([400], [400], 2, 2, 128, (50, 20, 150), False),               # sinks of more than a tile
    ([100, 90], [30, 200], 2, 1, 64, (10, 10, 2), False),          # rows before the first key: nothing seen
    ([250], [250], 3, 1, 64, (1 << 28, 0, 1 << 28), False),        # bounds past every row
    ([2000], [2000], 2, 1, 32, (200, 0, 4), False),                # sinks' gradients split
    ([64, 7, 300], [64, 7, 300], 8, 8, 16, (5, 5, 16), True),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"q{sum(c[0])}-k{sum(c[1])}-h{c[2]}.{c[3]}-d{c[4]}-w{c[5]}{'m' if c[6] else ''}")
def test_parity(ssc, case, dt):
    ql, kl, hq, hk, d, window, masked = case
    print(f"[window] {dt} q{ql} k{kl} heads {hq}/{hk} d{d} {window} mask {masked}", flush=True)
    _check(ssc, _inputs(1, ql, kl, hq, hk, d, dt, masked), window)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("batch", [62, 63, 64, 200, 4500])
def test_many_samples(ssc, dt, batch):
    """Samples past what one look at the offsets holds, some empty, and sinks that take fewer rows than there are or more."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 7, batch).tolist()
    keys = rng.integers(0, 9, batch).tolist()
    lens[batch // 2], keys[batch // 2] = 150, 150
    for ql, kl, window in ((lens, lens, (1, 1, 1)), (lens, keys, (0, 2, 3)), ([1] * batch, keys, (3, 0, 40))):
        print(f"[window] {dt} {batch} samples {window}", flush=True)
        case = _inputs(14, ql, kl, 2, 1, 32, dt)
        _check(ssc, case, window)
        q, k, v, do, qo, ko, _ = (None if t is None else t.to(DEV) for t in case)
        a, al = ssc.window_attention_fwd(q, k, v, qo, ko, None, None)
        b, bl = ssc.cross_attention_fwd(q, k, v, qo, ko)
        assert torch.equal(a, b) and torch.equal(al, bl)
        for x, y in zip(ssc.window_attention_bwd(q, k, v, a, al, do, qo, ko, None, None),
                        ssc.cross_attention_bwd(q, k, v, b, bl, do, qo, ko)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("left", [0, 1, 31, 32, 33, 63, 64, 127, 128, 129])
def test_edges_of_tiles(ssc, dt, left):
    """Windows that end on, before and behind the borders of tiles and waves."""
    for right, sinks in ((0, 0), (left, 1), (128 - left, 64)):
        if right >= 0:
            _check(ssc, _inputs(2, [385], [385], 1, 1, 32, dt), (left, right, sinks))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 7, 16, 32, 33])
def test_new_rows_of_a_longer_sequence(ssc, dt, rows):
    """The last rows' results are those of the whole sequence's call: the same keys in other tiles."""
    q, k, v, do, off, _, _ = _inputs(3, [600], [600], 4, 2, 64, dt)
    new = torch.tensor([0, rows], dtype=torch.int32)
    got = _check(ssc, (q[-rows:], k, v, do[-rows:], new, off, None), (200, 0, 3))
    whole = _check(ssc, (q, k, v, do, off, off, None), (200, 0, 3))
    for a, b in ((got[0], whole[0][-rows:]), (got[1], whole[1][:, -rows:])):
        assert torch.allclose(a.float(), b.float(), rtol=4 * torch.finfo(a.dtype).eps, atol=4 * torch.finfo(a.dtype).eps)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_unseen_keys_are_never_used(ssc, dt):
    """Rows that left the window of every new row may hold anything, as do rows of no sample."""
    q, k, v, do, _, _, _ = _inputs(4, [9], [900], 2, 1, 64, dt)
    qo, ko = torch.tensor([0, 4, 9], dtype=torch.int32), torch.tensor([50, 500, 850], dtype=torch.int32)
    clean = _check(ssc, (q, k, v, do, qo, ko, None), (100, 0, 3))
    k, v = k.clone(), v.clone()
    for lo, hi in ((0, 50), (53, 500 - 4 - 100), (503, 850 - 5 - 100), (850, 900)):
        k[lo:hi], v[lo:hi] = float("nan"), float("inf")
    args = [t.to(DEV) for t in (q, k, v)]
    where = (qo.to(DEV), ko.to(DEV), 100, 0, 3)
    out, lse = ssc.window_attention_fwd(*args, *where)
    grads = ssc.window_attention_bwd(*args, out, lse, do.to(DEV), *where)
    for a, b in zip((out, lse, grads[0]), clean):
        assert torch.equal(a, b)
    seen = torch.zeros(900, dtype=torch.bool)
    for lo, hi in ((50, 53), (396, 500), (500, 503), (745, 850)):
        seen[lo:hi] = True
    for a, b in zip(grads[1:], clean[3:]):
        assert torch.equal(a[seen.to(DEV)], b[seen.to(DEV)]) and torch.isfinite(a.float()).all()


def test_a_window_over_everything_is_cross_attention(ssc):
    q, k, v, do, qo, ko, m = (None if t is None else t.to(DEV) for t in _inputs(5, [200, 77], [300, 91], 4, 2, 64, "bf16", True))
    a, al = ssc.window_attention_fwd(q, k, v, qo, ko, None, None, 0, m)
    b, bl = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
    assert torch.equal(a, b) and torch.equal(al, bl)
    for x, y in zip(ssc.window_attention_bwd(q, k, v, a, al, do, qo, ko, None, None, 0, m),
                    ssc.cross_attention_bwd(q, k, v, b, bl, do, qo, ko, m)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_packed_and_strided_views(ssc, dt):
    case = _inputs(6, [130, 20], [130, 77], 4, 2, 64, dt, True)

    def views(q, k, v):
        qs = q.transpose(0, 1).contiguous().transpose(0, 1)
        packed = torch.full((k.shape[0], 7, 64), float("nan"), dtype=k.dtype, device=DEV)
        packed[:, 1:3], packed[:, 4:6] = k, v
        return qs, packed[:, 1:3], packed[:, 4:6]

    _check(ssc, case, (30, 9, 2), views=views)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_scales(ssc, scale):
    _check(ssc, _inputs(7, [150], [150], 2, 1, 32, "f32"), (20, 10, 2), scale=scale)


def test_parts_of_the_gradient(ssc):
    q, k, v, do, qo, ko, _ = (None if t is None else t.to(DEV) for t in _inputs(8, [200], [200], 2, 1, 128, "bf16"))
    out, lse = ssc.window_attention_fwd(q, k, v, qo, ko, 30, 30, 4)
    whole = ssc.window_attention_bwd(q, k, v, out, lse, do, qo, ko, 30, 30, 4)
    for i in range(3):
        need = [j == i for j in range(3)]
        part = ssc.window_attention_bwd(q, k, v, out, lse, do, qo, ko, 30, 30, 4, None, None, *need)
        assert torch.equal(part[i], whole[i]) and all(part[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_samples_do_not_touch(ssc, dt):
    """A sample's results do not change with another's values, nor with a NaN or an infinity among them."""
    q, k, v, do, qo, ko, _ = (None if t is None else t.to(DEV) for t in _inputs(9, [130, 60, 200], [130, 60, 200], 2, 1, 64, dt))
    outs = []
    for spoil in (False, True):
        if spoil:
            q[130:190] *= 50
            do[140] = float("inf")
            k[150], v[160] = float("nan"), float("inf")
        out, lse = ssc.window_attention_fwd(q, k, v, qo, ko, 40, 0, 2)
        outs.append((out, lse.t(), *ssc.window_attention_bwd(q, k, v, out, lse, do, qo, ko, 40, 0, 2)))
    rows = list(range(130)) + list(range(190, 390))
    for a, b in zip(*outs):
        assert torch.equal(a[rows], b[rows])


def test_no_rows(ssc):
    q, k = torch.empty(0, 2, 64, device=DEV), torch.randn(5, 2, 64, device=DEV)
    qo, ko = torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    out, lse = ssc.window_attention_fwd(q, k, k, qo, ko, 3, 3, 2)
    assert out.shape == (0, 2, 64)
    _, dk, dv = ssc.window_attention_bwd(q, k, k, out, lse, out, qo, ko, 3, 3, 2)
    assert (dk == 0).all() and (dv == 0).all()
    out, lse = ssc.window_attention_fwd(k, q, q, ko, qo, 3, 3, 2)
    assert (out == 0).all() and torch.isinf(lse).all()
    assert (ssc.window_attention_bwd(k, q, q, out, lse, k, ko, qo, 3, 3, 2)[0] == 0).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_graph(ssc, dt):
    """Captured passes with splits and sinks, replayed on changing inputs; two graphs take turns."""
    q, k, v, do, qo, ko, _ = (None if t is None else t.to(DEV) for t in _inputs(10, [900, 300], [900, 300], 2, 1, 64, dt))

    def step():
        out, lse = ssc.window_attention_fwd(q, k, v, qo, ko, 100, 100, 4)
        return (out, lse, *ssc.window_attention_bwd(q, k, v, out, lse, do, qo, ko, 100, 100, 4))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(4):
        q.copy_(torch.randn(q.shape, device=DEV))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs[i % 2], step()):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_results_repeat(ssc, dt):
    q, k, v, do, qo, ko, _ = (None if t is None else t.to(DEV) for t in _inputs(11, [3000], [3000], 4, 2, 64, dt))
    outs = []
    for _ in range(4):
        out, lse = ssc.window_attention_fwd(q, k, v, qo, ko, 200, 200, 4)
        outs.append((out, lse, *ssc.window_attention_bwd(q, k, v, out, lse, do, qo, ko, 200, 200, 4)))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


def test_wrapper(ssc):
    q, k, v, do, qo, ko, m = (t.to(DEV) for t in _inputs(12, [90], [120], 4, 2, 64, "bf16", True))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    ssc.window_attention(*leaves, qo, ko, 20, 5, 3, m).backward(do)
    out, lse = ssc.window_attention_fwd(q, k, v, qo, ko, 20, 5, 3, m)
    for t, want in zip(leaves, ssc.window_attention_bwd(q, k, v, out, lse, do, qo, ko, 20, 5, 3, m)):
        assert torch.equal(t.grad, want)
    odd = torch.randn(90 * 2 * 64 + 1, device=DEV)[1:].view(90, 2, 64).requires_grad_()
    ssc.window_attention(odd, odd, odd, qo, qo, 20, 5).sum().backward()
    assert torch.isfinite(odd.grad).all()


def test_gradient_is_the_difference(ssc):
    """As the voxel block's test: the fourth-order difference of a loss of order one along the gradient, steps of 2^-5."""
    q, k, v, do, qo, ko, _ = (None if t is None else t.to(DEV) for t in _inputs(13, [150], [150], 2, 1, 32, "f32"))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]

    def loss(*t):
        return (ssc.window_attention(*t, qo, ko, 20, 10, 2).double() * do.double()).mean()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in grads)).item()
    vals = {}
    for s in (-2, -1, 1, 2):
        with torch.no_grad():
            vals[s] = loss(*[t + (s * 2.0 ** -5 * g / norm) for t, g in zip((q, k, v), grads)]).item()
    slope = (8 * (vals[1] - vals[-1]) - (vals[2] - vals[-2])) / (12 * 2.0 ** -5)
    assert abs(slope - norm) <= 0.01 * norm
