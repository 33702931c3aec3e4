"""GPU parity of ssc_cross_attn_fwd / ssc_cross_attn_bwd against the float64 oracle.

Tolerances are elementwise bounds derived from the kernels' arithmetic.  With u half a step of the type (bf16 2^-8,
fp16 2^-11, fp32 2^-24), f = 2^-24 and, per row, T = max_j scale sum_d |q k_j|:
  a score is off by at most (D + 4) f T, its exponent's rounding by 2 f T more, the exponential itself by 2^-22, so a
  probability (and the sum it is divided by) by a relative ep = 2 (D + 8) f T + 2^-21; the sums of n terms add n f;
  probabilities and dS are rounded to the type for the second product (u each; none for fp32, whose values stay fp32);
  the result is rounded once (u).  Sums of absolute values come from the oracle.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F = 2.0 ** -24


def _u(dt):
    return torch.finfo(DT[dt]).eps / 2


@pytest.fixture(scope="module")
def ssc():
    import sparse_submanifold_convolution_amd as m
    m.lib()
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(seed, q_lens, kv_lens, hq, hk, d, dt, mask=None, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    nq, nk = sum(q_lens), sum(kv_lens)
    q = (amp * torch.randn(nq, hq, d, generator=g)).to(DT[dt])
    k, v = (torch.randn(nk, hk, d, generator=g).to(DT[dt]) for _ in range(2))
    do = torch.randn(nq, hq, d, generator=g).to(DT[dt])
    m = None
    if mask == "random":
        m = torch.rand(nk, generator=g) < 0.7
    elif mask == "none left":
        m = torch.zeros(nk, dtype=torch.bool)
    off = [torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32) for x in (q_lens, kv_lens)]
    return q, k, v, do, off[0], off[1], m


def _to(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _bounds(dt, d, n, top):
    """(relative error of a probability, of the sums over n) for rows whose largest sum of |q k| is `top`."""
    return 2 * (d + 8) * F * top + 2.0 ** -21, n * F


def _within(got, ref, tol, what):
    got = _f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst |err|/tol "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} at {np.argwhere(bad)[0]}")


def _check(ssc, case, bwd=True, scale=None, views=None):
    """Runs one case on the GPU and holds it to the oracle.  views: maps (q, k, v) on the device to strided views."""
    q, k, v, do, qo, ko, m = case
    dt = {v: k for k, v in DT.items()}[q.dtype]
    u, d = _u(dt), q.shape[2]
    up = 0.0 if dt == "f32" else u
    gq, gk, gv, gdo, gqo, gko, gm = _to(q, k, v, do, qo, ko, m)
    if views:
        gq, gk, gv = views(gq, gk, gv)
    out, lse = ssc.cross_attention_fwd(gq, gk, gv, gqo, gko, gm, scale)
    args = (_f64(q), _f64(k), _f64(v))
    where = (qo.numpy(), ko.numpy(), None if m is None else m.numpy(), scale)
    ref, rlse, (size, top) = A.cross_attention_fwd(*args, *where)
    n = int((ko[1:] - ko[:-1]).max()) if len(k) else 0
    ep, es = _bounds(dt, d, n, top.T[:, :, None])
    eo = u * np.abs(ref) + (up + 2 * ep + 2 * es + 8 * F) * size
    _within(out, ref, eo + 1e-30 + (2.0 ** -25 if dt == "f16" else 0), "out")
    glse = _f64(lse)
    assert np.array_equal(np.isinf(glse), np.isinf(rlse)) and not np.isnan(glse).any()
    fin = np.isfinite(rlse)
    tol = (ep[:, :, 0].T + es + 8 * F * (1 + np.abs(np.where(fin, rlse, 0)) + top))
    assert (np.abs(glse[fin] - rlse[fin]) <= tol[fin]).all()
    if not bwd:
        return out, lse
    dq, dk, dv = ssc.cross_attention_bwd(gq, gk, gv, out, lse, gdo, gqo, gko, gm, scale)
    nb = max(n, int((qo[1:] - qo[:-1]).max()) * (q.shape[1] // k.shape[1]) if len(q) else 0)
    p_err = (3 * ep.max() if ep.size else 0) + (nb + d + 16) * F * 2 + 8 * F * (np.abs(rlse[fin]).max() if fin.any() else 0)
    rq, rk, rv, (sq, sk, sv) = A.cross_attention_bwd(*args, _f64(do), *where, err=(p_err, up, eo))
    tiny = 2.0 ** -25 if dt == "f16" else 1e-30  # half of fp16's smallest step
    _within(dq, rq, u * np.abs(rq) + sq + tiny, "dq")
    _within(dk, rk, u * np.abs(rk) + sk + tiny, "dk")
    _within(dv, rv, u * np.abs(rv) + sv + tiny, "dv")
    return out, lse, dq, dk, dv


CASES = [  # q_lens, kv_lens, heads_q, heads_kv, head_dim, mask
    ([1], [1], 1, 1, 8, None),                               # one row, one key
    ([1], [257], 8, 2, 64, None),                            # one token, grouped heads
    ([1, 1, 1], [4097, 63, 64], 4, 4, 64, None),             # one token a sample: key splits
    ([33], [65], 2, 2, 32, None),                            # one past a block on both sides
    ([128, 129], [64, 128], 2, 1, 64, None),                 # whole tiles and one past
    ([5, 0, 300, 1], [0, 9, 130, 77], 6, 2, 40, "random"),   # empty on either side, ragged, mask
    ([64, 7], [100, 33], 3, 3, 72, "none left"),             # every key masked
    ([70, 200], [513, 31], 4, 2, 96, "random"),
    ([190], [333], 2, 2, 128, None),
    ([17, 40], [5000, 6001], 4, 4, 80, "random"),            # few rows, long keys: both splits
    ([4000, 3001], [70, 129], 2, 2, 64, None),               # many rows, few keys: dK and dV splits
    ([700], [700], 5, 5, 48, None),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"q{sum(c[0])}-k{sum(c[1])}-h{c[2]}.{c[3]}-d{c[4]}" for c in CASES])
def test_parity(ssc, case, dt):
    ql, kl, hq, hk, d, mask = case
    print(f"[attention] {dt} q{ql} k{kl} heads {hq}/{hk} d{d} mask {mask}", flush=True)
    _check(ssc, _inputs(1, ql, kl, hq, hk, d, dt, mask))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_smallest_head(ssc, dt):
    d = 4 if dt == "f32" else 8
    _check(ssc, _inputs(2, [50], [90], 3, 1, d, dt))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_packed_and_strided_views(ssc, dt):
    """q as head-major storage, k and v as slices of one packed projection with room between rows."""
    case = _inputs(3, [130, 20], [200, 77], 4, 2, 64, dt, "random")

    def views(q, k, v):
        qs = q.transpose(0, 1).contiguous().transpose(0, 1)
        packed = torch.full((k.shape[0], 7, 64), float("nan"), dtype=k.dtype, device=DEV)
        packed[:, 1:3], packed[:, 4:6] = k, v
        return qs, packed[:, 1:3], packed[:, 4:6]

    a = _check(ssc, case, views=views)
    b = _check(ssc, case)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("scale", [0.0, -0.4, 3.0])
def test_scales(ssc, scale):
    _check(ssc, _inputs(4, [40, 3], [100, 70], 2, 2, 32, "bf16", "random", amp=0.5), scale=scale)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ql,kl", [([3], [3000]), ([300], [300])])
def test_large_scores(ssc, dt, ql, kl):
    """Scores in the hundreds: the running maximum carries the row, most probabilities vanish."""
    _check(ssc, _inputs(5, ql, kl, 2, 2, 64, dt, amp=30.0))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_masked_rows_are_never_used(ssc, dt, junk):
    q, k, v, do, qo, ko, m = _inputs(6, [60, 40], [150, 90], 4, 2, 64, dt, "random")
    clean = _check(ssc, (q, k, v, do, qo, ko, m))
    k, v = k.clone(), v.clone()
    value = torch.finfo(DT[dt]).min if junk == "lowest" else junk
    k[~m], v[~m] = value, value
    args = _to(q, k, v)
    gdo, gqo, gko, gm = _to(do, qo, ko, m)
    out, lse = ssc.cross_attention_fwd(*args, gqo, gko, gm)
    grads = ssc.cross_attention_bwd(*args, out, lse, gdo, gqo, gko, gm)
    for x, y in zip(clean, (out, lse, *grads)):
        assert torch.equal(x, y)


def test_nan_and_inf_stay_in_their_rows(ssc):
    """A NaN query spoils its own row, an infinite attended key the rows of its sample, nothing else."""
    q, k, v, do, qo, ko, _ = _inputs(7, [70, 70], [100, 100], 2, 2, 64, "bf16")
    clean = ssc.cross_attention_fwd(*_to(q, k, v, qo, ko))[0]
    q[5, 0] = float("nan")
    v[150, 1, 3] = float("inf")
    out = ssc.cross_attention_fwd(*_to(q, k, v, qo, ko))[0]
    assert torch.isnan(out[5, 0]).all() and torch.isinf(out[70:, 1, 3]).all()
    touched = torch.zeros(140, 2, 64, dtype=torch.bool, device=DEV)
    touched[5, 0] = True
    touched[70:, 1, 3] = True
    assert torch.equal(out[~touched], clean[~touched])


def test_rows_outside_the_samples(ssc):
    """Offsets that leave rows before and after the samples: zeros, lse -inf, zero gradients, nothing else changed."""
    q, k, v, do, _, _, _ = _inputs(8, [200], [300], 2, 2, 64, "f16")
    qo, ko = torch.tensor([10, 60, 150], dtype=torch.int32), torch.tensor([7, 107, 250], dtype=torch.int32)
    out, lse, dq, dk, dv = _check(ssc, (q, k, v, do, qo, ko, None))
    for t, lo, hi in ((out, 10, 150), (dq, 10, 150), (dk, 7, 250), (dv, 7, 250)):
        assert not t[:lo].any() and not t[hi:].any()
    assert (lse[:, :10] == -float("inf")).all() and (lse[:, 150:] == -float("inf")).all()


def test_many_samples(ssc):
    """More samples than one wave scans at once, with empty ones among them."""
    rng = np.random.default_rng(9)
    ql, kl = rng.integers(0, 9, 150).tolist(), rng.integers(0, 40, 150).tolist()
    _check(ssc, _inputs(9, ql, kl, 2, 1, 32, "bf16", "random"))


def test_empty_tensors(ssc):
    q, k, v, do, qo, ko, _ = _inputs(10, [0, 0], [5, 4], 2, 2, 32, "bf16")
    out, lse = ssc.cross_attention_fwd(*_to(q, k, v, qo, ko))
    assert out.shape == (0, 2, 32) and lse.shape == (2, 0)
    dq, dk, dv = ssc.cross_attention_bwd(*_to(q, k, v), out, lse, *_to(do, qo, ko))
    assert not dk.any() and not dv.any()
    q, k, v, do, qo, ko, _ = _inputs(10, [5, 4], [0, 0], 2, 2, 32, "bf16")
    out, lse = ssc.cross_attention_fwd(*_to(q, k, v, qo, ko))
    assert not out.any() and (lse == -float("inf")).all()
    dq, dk, dv = ssc.cross_attention_bwd(*_to(q, k, v), out, lse, *_to(do, qo, ko))
    assert not dq.any() and dk.shape == (0, 2, 32)


def test_each_gradient_alone(ssc):
    case = _inputs(11, [90, 30], [100, 200], 4, 2, 64, "bf16", "random")
    *_, dq, dk, dv = _check(ssc, case)
    q, k, v, do, qo, ko, m = _to(*case)
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
    for i, ref in enumerate((dq, dk, dv)):
        need = [j == i for j in range(3)]
        got = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m, None, *need)
        assert [g is not None for g in got] == need and torch.equal(got[i], ref)


@pytest.mark.parametrize("dt,amp", [("f16", 2.0 ** -14), ("f16", 2.0 ** 6), ("bf16", 2.0 ** -40)])
def test_small_and_large_output_gradients(ssc, dt, amp):
    """Gradients scale with dout by a power of two: bit for bit where the result's own rounding does not change."""
    q, k, v, do, qo, ko, _ = _inputs(12, [40], [3000], 2, 2, 64, dt)
    q, k, v, do, qo, ko = _to(q, k, v, do, qo, ko)
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko)
    small = (do.float() * amp).to(do.dtype)
    back = (small.float() / amp).to(do.dtype)
    a = ssc.cross_attention_bwd(q, k, v, out, lse, back, qo, ko)
    b = ssc.cross_attention_bwd(q, k, v, out, lse, small, qo, ko)
    # fp16's results may be subnormal: each is off by half of its smallest step, the first one's times amp
    for x, y in zip(a, b):
        tol = (2.0 ** -25 * (1 + amp) if dt == "f16" else 0) + x.double().abs() * amp * torch.finfo(x.dtype).eps
        assert ((x.double() * amp - y.double()).abs() <= tol).all()


def test_gradient_matches_differences(ssc):
    """fp32 forward differences along random directions against the kernels' gradients."""
    q, k, v, do, qo, ko, m = _to(*_inputs(13, [50, 20], [60, 33], 4, 2, 32, "f32", "random"))
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
    grads = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m)
    h = 2.0 ** -7
    g = torch.Generator(device=DEV).manual_seed(1)
    for i, grad in enumerate(grads):
        direction = torch.randn(grad.shape, generator=g, device=DEV)
        direction /= direction.norm()
        vals = []
        for s in (-2, -1, 1, 2):
            t = [q, k, v]
            t[i] = t[i] + s * h * direction
            vals.append((ssc.cross_attention_fwd(*t, qo, ko, m)[0].double() * do.double()).sum().item())
        diff = (8 * (vals[2] - vals[1]) - (vals[3] - vals[0])) / (12 * h)
        exact = (grad.double() * direction.double()).sum().item()
        # fourth-order difference: h^4 times fifth derivatives of order one, and the fp32 results' rounding
        # (about 2^-21 of sum |out dout|, as if all aligned, over h)
        slack = 64 * h ** 4 + 2.0 ** -21 * (out.double() * do.double()).abs().sum().item() ** 0.5 * 8 / h
        assert abs(diff - exact) <= slack, (i, diff, exact, slack)


def test_autograd_and_broadcast_inputs(ssc):
    """Gradients through the autograd wrapper: a key head shared by expand, and an expanded output gradient."""
    q, k, v, do, qo, ko, _ = _to(*_inputs(14, [40], [50], 4, 1, 32, "f32"))
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    out = ssc.cross_attention(q, k.expand(-1, 4, -1), v.expand(-1, 4, -1), qo, ko)
    out.sum().backward()
    got = [t.grad.clone() for t in (q, k, v)]
    one = torch.ones_like(out)
    o, lse = ssc.cross_attention_fwd(q.detach(), k.detach(), v.detach(), qo, ko)
    ref = ssc.cross_attention_bwd(q.detach(), k.detach(), v.detach(), o, lse, one, qo, ko)
    for a, b in zip(got, ref):
        assert (a - b).abs().max() <= 64 * F * 50 * b.abs().max()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_repeats_bit_for_bit_also_on_another_stream(ssc, dt):
    case = _to(*_inputs(15, [500, 7], [900, 1200], 4, 2, 64, dt, "random"))
    q, k, v, do, qo, ko, m = case

    def both():
        out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
        return (out, lse, *ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m))

    first = both()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        second = both()
    stream.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_graph_replays(ssc):
    """Forward and backward captured once; replays follow the inputs' new values and match the eager calls."""
    q, k, v, do, qo, ko, m = _to(*_inputs(16, [5, 90], [700, 300], 4, 2, 64, "f16", "random"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
        ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
        grads = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m)
    for i in range(4):
        q.copy_(torch.randn(q.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)))
        do.mul_(0.5)
        m.logical_xor_(torch.arange(m.numel(), device=DEV) % (i + 3) == 0)
        graph.replay()
        torch.cuda.synchronize()
        eo, el = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
        eager = (eo, el, *ssc.cross_attention_bwd(q, k, v, eo, el, do, qo, ko, m))
        torch.cuda.synchronize()
        for a, b in zip((out, lse, *grads), eager):
            assert torch.equal(a, b)


def test_key_rows_past_32_bit_offsets(ssc):
    """Keys and values whose last rows start beyond 2^32 elements of their buffer."""
    nk, row = 2200, 1 << 21
    buf = torch.empty(nk * row, dtype=torch.bfloat16, device=DEV)  # 9.2 GB, untouched but for the rows' heads
    q, k, v, do, qo, ko, _ = _inputs(17, [9], [nk], 2, 1, 32, "bf16")

    def views(gq, gk, gv):
        kk, vv = (buf.as_strided((nk, 1, 32), (row, 32, 1), o) for o in (0, 64))
        kk.copy_(gk)
        vv.copy_(gv)
        return gq, kk, vv

    _check(ssc, (q, k, v, do, qo, ko, None), views=views)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_broadcast_rows(ssc, dt):
    """Rows of stride 0: one query row for all, one key row for all, past a tile's end as well."""
    q, k, v, do, qo, ko, _ = _to(*_inputs(18, [50, 20], [70, 33], 2, 2, 64, dt))
    for name in ("q", "k", "v"):
        t = {"q": q, "k": k, "v": v}
        t[name] = t[name][:1].expand(t[name].shape)
        assert t[name].stride(0) == 0
        results = []
        for u in (t, {n: x.contiguous() for n, x in t.items()}):
            out, lse = ssc.cross_attention_fwd(u["q"], u["k"], u["v"], qo, ko)
            results.append((out, lse, *ssc.cross_attention_bwd(u["q"], u["k"], u["v"], out, lse, do, qo, ko)))
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_offsets_outside_the_rows_are_clamped(ssc):
    q, k, v, do, _, _, _ = _to(*_inputs(19, [40], [60], 2, 2, 32, "bf16"))

    def run(qo, ko):
        qo, ko = (torch.tensor(o, dtype=torch.int32, device=DEV) for o in (qo, ko))
        out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko)
        return (out, lse, *ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko))

    for a, b in zip(run([-5, 30, 1 << 30], [-(1 << 31), 25, 100]), run([0, 30, 40], [0, 25, 60])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_sum_of_value_gradients(ssc, dt, d):
    """A row's probabilities sum to one: the value gradients of a sample sum to the sum of its output gradients."""
    q, k, v, do, qo, ko, _ = _to(*_inputs(20, [300], [200], 1, 1, d, dt))
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko)
    _, _, dv = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko)
    got, ref = dv.double().sum(0), do.double().sum(0)
    # each of the n entries is off by u of itself, and by u and some fp32 steps of sum P |dout|; the sums of those are
    # at most the sum of |dout| each
    u = _u(dt)
    tol = (2 * u + 2 ** -14) * do.double().abs().sum(0) + (200 * 2.0 ** -25 if dt == "f16" else 0)
    assert ((got - ref).abs() <= tol).all()
