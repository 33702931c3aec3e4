"""The calls over serialised rows reject bad arguments on the host: no call here reaches the GPU."""
import ast
import ctypes
import inspect

import pytest
import torch

import sparse_submanifold_convolution_amd as ssc
from sparse_submanifold_convolution_amd import sequence as seq
from test_attention_abi import BAD_ATTN, _attn

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)  # aligned and not, never dereferenced
MUCH = 1 << 60


@pytest.fixture(scope="module")
def L():
    return ssc.lib()


def _struct(fields):
    kind = {"q": ctypes.c_int64, "i": ctypes.c_int32, "d": ctypes.c_double, "f": ctypes.c_float}
    return type("Shape", (ctypes.Structure,), {"_fields_": [(n, kind[k]) for n, k in fields]})


_Norm = _struct([("n", "q"), ("xr", "q"), ("rr", "q"), ("p", "d"), ("c", "i"), ("dt", "i"), ("layer", "i"), ("eps", "f")])
_Scan = _struct([("n", "q"), ("xr", "q"), ("gr", "q"), ("batch", "i"), ("c", "i"), ("dt", "i"), ("form", "i"), ("reverse", "i")])
_Win = _struct([("left", "i"), ("right", "i"), ("sinks", "i")])


def _norm(**kw):
    return ctypes.byref(_Norm(**{**dict(n=10, xr=64, rr=64, p=0.0, c=64, dt=2, layer=0, eps=1e-5), **kw}))


def _scan(**kw):
    return ctypes.byref(_Scan(**{**dict(n=10, xr=64, gr=128, batch=2, c=64, dt=2, form=0, reverse=0), **kw}))


def _win(left=10, right=10, sinks=2):
    return ctypes.byref(_Win(left, right, sinks))


def _calls(call, good, count, skip_null=(), skip_odd=()):
    """Every pointer of a call, NULL or misaligned: the indexes that are taken all the same."""
    for i in range(count):
        for v, skip in ((None, skip_null), (ODD, skip_odd)):
            args = [FAKE] * count
            args[i] = v
            if i not in skip:
                assert call(*good(args)) == 1, (i, v)


BAD_NORM = [(dict(n=-1), 1), (dict(n=(1 << 28) + 1), 1), (dict(c=0), 1), (dict(c=12), 2), (dict(c=6, dt=0), 2), (dict(c=8200), 2),
            (dict(dt=3), 2), (dict(p=1.0), 1), (dict(p=-0.1), 1), (dict(p=float("nan")), 1), (dict(layer=-1), 1),
            (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1), (dict(eps=float("nan")), 1), (dict(xr=-64), 1), (dict(xr=4), 1),
            (dict(rr=1 << 41), 1), (dict(n=1 << 26, c=512, xr=512, rr=512), 2), (dict(n=(1 << 24) + 1, c=2048, xr=2048, rr=2048, p=0.5), 2)]


@pytest.mark.parametrize("change,code", BAD_NORM, ids=[str(c[0]) for c in BAD_NORM])
def test_norm_refuses_shapes(L, change, code):
    sh = _norm(**change)
    assert L.ssc_layer_norm_fwd(sh, *[FAKE] * 7, None) == code
    assert L.ssc_layer_norm_bwd(sh, *[FAKE] * 10, MUCH, None) == code
    assert L.ssc_layer_norm_workspace_bytes(sh) == 0


def test_norm_refuses_pointers(L):
    f, b = L.ssc_layer_norm_fwd, L.ssc_layer_norm_bwd
    assert f(None, *[FAKE] * 7, None) == 1 and b(None, *[FAKE] * 10, MUCH, None) == 1
    assert L.ssc_layer_norm_workspace_bytes(None) == 0 and L.ssc_layer_norm_workspace_bytes(_norm()) > 0
    # x, residual, weight, bias, rng, y, s: weight and bias may be NULL, rng too without dropout
    _calls(f, lambda a: (_norm(), *a, None), 7, skip_null=(2, 3, 4), skip_odd=(4,))
    _calls(f, lambda a: (_norm(p=0.5), *a, None), 7, skip_null=(2, 3))
    assert f(_norm(), FAKE, None, None, None, None, FAKE, FAKE, None) == 1  # a sum without a residual
    assert f(_norm(p=0.5), FAKE, None, None, None, FAKE, FAKE, None, None) == 1  # dropout without one
    assert f(_norm(n=0), *[None] * 7, None) == 0
    # s, dy, ds, weight, rng, dx, dresidual, dweight, dbias, workspace
    _calls(b, lambda a: (_norm(), *a, MUCH, None), 10, skip_null=(2, 3, 4, 5, 6, 7, 8), skip_odd=(4,))
    _calls(b, lambda a: (_norm(p=0.5), *a, MUCH, None), 10, skip_null=(2, 3, 5, 6, 7, 8))
    assert b(_norm(), *[FAKE] * 10, 64, None) == 3
    assert b(_norm(), *[FAKE] * 5, None, None, None, None, None, 0, None) == 0  # no gradient asked for
    assert b(_norm(n=0), *[FAKE] * 7, None, None, None, 0, None) == 0


def test_dropout_refuses(L):
    f = L.ssc_dropout
    good = dict(n=100, dt=0, p=0.5, layer=0)
    for change, code in ((dict(n=-1), 1), (dict(dt=3), 2), (dict(p=1.0), 1), (dict(p=-1e-9), 1), (dict(p=float("nan")), 1),
                         (dict(layer=-1), 1), (dict(n=(1 << 35) + 1), 2)):
        a = {**good, **change}
        assert f(a["n"], a["dt"], a["p"], a["layer"], *[FAKE] * 4, None) == code, change
    _calls(f, lambda a: (100, 0, 0.5, 0, *a, None), 4, skip_null=(1,))
    assert f(0, 0, 0.5, 0, *[None] * 4, None) == 0


BAD_SCAN = [(dict(n=-1), 1), (dict(n=(1 << 28) + 1), 1), (dict(c=0), 1), (dict(c=12), 2), (dict(c=6, dt=0), 2), (dict(c=8200), 2),
            (dict(dt=-1), 2), (dict(batch=0), 1), (dict(batch=65537), 1), (dict(form=2), 2), (dict(form=-1), 2), (dict(xr=-8), 1),
            (dict(gr=12), 1), (dict(gr=1 << 41), 1), (dict(n=1 << 28, c=8192), 2)]


@pytest.mark.parametrize("change,code", BAD_SCAN, ids=[str(c[0]) for c in BAD_SCAN])
def test_scan_refuses_shapes(L, change, code):
    sh = _scan(**change)
    assert L.ssc_gated_scan_fwd(sh, *[FAKE] * 8, MUCH, None) == code
    assert L.ssc_gated_scan_bwd(sh, *[FAKE] * 11, MUCH, None) == code
    assert L.ssc_gated_scan_workspace_bytes(sh) == 0 and L.ssc_gated_scan_carry_bytes(sh) == 0


def test_scan_refuses_pointers(L):
    f, b = L.ssc_gated_scan_fwd, L.ssc_gated_scan_bwd
    assert f(None, *[FAKE] * 8, MUCH, None) == 1 and b(None, *[FAKE] * 11, MUCH, None) == 1
    # x, gate, offsets, h0, y, last, carries, workspace
    _calls(f, lambda a: (_scan(), *a, MUCH, None), 8, skip_null=(3, 6))
    # x, gate, carries, dy, offsets, h0, dlast, dx, dgate, dh0, workspace
    _calls(b, lambda a: (_scan(), *a, MUCH, None), 11, skip_null=(5, 6, 9))
    assert f(_scan(), *[FAKE] * 8, 8, None) == 3 and b(_scan(), *[FAKE] * 11, 8, None) == 3
    assert L.ssc_gated_scan_carry_bytes(_scan(n=0)) > 0


@pytest.mark.parametrize("change,code", BAD_ATTN, ids=[str(c[0]) for c in BAD_ATTN])
def test_window_refuses_shapes(L, change, code):
    sh = _attn(**change)
    assert L.ssc_window_attn_fwd(sh, _win(), *[FAKE] * 9, MUCH, None) == code
    assert L.ssc_window_attn_bwd(sh, _win(), *[FAKE] * 13, MUCH, None) == code
    assert L.ssc_window_attn_workspace_bytes(sh, _win(), 0) == 0 == L.ssc_window_attn_workspace_bytes(sh, _win(), 1)


@pytest.mark.parametrize("window", [(-2, 0, 0), (0, -2, 0), (0, 0, -1), ((1 << 28) + 1, 0, 0), (0, (1 << 28) + 1, 0), (0, 0, (1 << 28) + 1)])
def test_window_refuses_bounds(L, window):
    assert L.ssc_window_attn_fwd(_attn(), _win(*window), *[FAKE] * 9, MUCH, None) == 1
    assert L.ssc_window_attn_bwd(_attn(), _win(*window), *[FAKE] * 13, MUCH, None) == 1
    assert L.ssc_window_attn_workspace_bytes(_attn(), _win(*window), 0) == 0


def test_window_refuses_pointers(L):
    f, b = L.ssc_window_attn_fwd, L.ssc_window_attn_bwd
    assert f(None, _win(), *[FAKE] * 9, MUCH, None) == 1 and f(_attn(), None, *[FAKE] * 9, MUCH, None) == 1
    _calls(f, lambda a: (_attn(), _win(), *a, MUCH, None), 9, skip_null=(5,), skip_odd=(5,))  # the mask: bytes, may be NULL
    _calls(b, lambda a: (_attn(), _win(), *a, MUCH, None), 13, skip_null=(8, 9, 10, 11), skip_odd=(8,))
    assert f(_attn(), _win(), *[FAKE] * 9, 8, None) == 3 and b(_attn(), _win(), *[FAKE] * 13, 8, None) == 3
    assert f(_attn(nq=0), _win(), *[None] * 9, 0, None) == 0
    assert b(_attn(), _win(), *[FAKE] * 9, None, None, None, FAKE, 0, None) == 0
    # the sinks' gradients over many rows are split, and their partial sums need room
    rows = dict(nq=100000, nk=100000)
    assert L.ssc_window_attn_workspace_bytes(_attn(**rows), _win(), 1) > L.ssc_window_attn_workspace_bytes(_attn(**rows), _win(sinks=0), 1)


def test_window_refuses_launches_past_the_grid(L):
    """The sinks' launch has 2^28 / 32 + 2 x 8194 tiles of one wave and a join of four: past 2^32 threads with two heads and
    every key a sink, while the other passes fit seven."""
    shape = dict(nq=8, nk=1 << 28, batch=8192, d=64)
    for sinks, most in ((0, 7), (1 << 28, 1)):
        assert L.ssc_window_attn_workspace_bytes(_attn(**shape, hq=most, hk=most), _win(sinks=sinks), 1) > 0
        assert L.ssc_window_attn_workspace_bytes(_attn(**shape, hq=most + 1, hk=most + 1), _win(sinks=sinks), 1) == 0


def test_python_checks():
    x = torch.zeros(6, 64)
    off = torch.tensor([0, 6], dtype=torch.int32)
    rng = torch.zeros(2, dtype=torch.int64)
    w = torch.ones(64)
    bad = [
        lambda: ssc.layer_norm_fwd(x[0]), lambda: ssc.layer_norm_fwd(x[:, ::2]), lambda: ssc.layer_norm_fwd(x[:, 1:5]),
        lambda: ssc.layer_norm_fwd(x, w.half()), lambda: ssc.layer_norm_fwd(x, w[:32]), lambda: ssc.layer_norm_fwd(x, None, w[None]),
        lambda: ssc.add_layer_norm_fwd(x, x[:5]), lambda: ssc.add_layer_norm_fwd(x, x.half()), lambda: ssc.add_layer_norm_fwd(x, x, p=0.1),
        lambda: ssc.add_layer_norm_fwd(x, x, p=0.1, rng=rng.int()), lambda: ssc.add_layer_norm_fwd(x, x, p=0.1, rng=rng, layer=-1),
        lambda: ssc.layer_norm_bwd(x, x[:5]), lambda: ssc.add_layer_norm_bwd(x, x, x.t()), lambda: ssc.add_layer_norm_bwd(x, x, None, p=0.5),
        lambda: ssc.dropout_fwd(x, 0.5), lambda: ssc.dropout_fwd(x.t(), 0.5, rng), lambda: ssc.dropout_fwd(x, 0.5, rng[:1]),
        lambda: ssc.dropout_fwd(x, 0.5, rng, 1 << 31), lambda: ssc.dropout_fwd(x, 0.5, rng, 0, x[:5]),
        lambda: ssc.gated_scan_fwd(x, x[:5], off), lambda: ssc.gated_scan_fwd(x, x.half(), off), lambda: ssc.gated_scan_fwd(x, x, off.long()),
        lambda: ssc.gated_scan_fwd(x, x, off, form="max"), lambda: ssc.gated_scan_fwd(x, x, off, torch.zeros(2, 64)),
        lambda: ssc.gated_scan_fwd(x, x, off, torch.zeros(1, 64).half()), lambda: ssc.gated_scan_bwd(x, x, w, x, off),
        lambda: ssc.gated_scan_bwd(x, x, w, x[:5], off)]
    q = torch.zeros(6, 2, 64)
    for kw in (dict(left=-1), dict(right=-1), dict(sinks=-1), dict(sinks=None), dict(left=(1 << 28) + 1), dict(kv_mask=torch.zeros(5, dtype=torch.bool)),
               dict(q_offsets=off.long()), dict(k=q[:, :, :32]), dict(v=q[:5])):
        args = {**dict(q=q, k=q, v=q, q_offsets=off, kv_offsets=off, left=3, right=3), **kw}
        bad.append(lambda args=args: ssc.window_attention_fwd(**args))
    # sound arguments that are not on a GPU
    bad += [lambda: ssc.layer_norm_fwd(x), lambda: ssc.add_layer_norm_fwd(x, x), lambda: ssc.dropout_fwd(x, 0.0),
            lambda: ssc.gated_scan_fwd(x, x, off), lambda: ssc.window_attention_fwd(q, q, q, off, off, 3, 3)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was taken")
    for call in (lambda: ssc.layer_norm_fwd(x.double()), lambda: ssc.dropout_fwd(x.double(), 0.0),
                 lambda: ssc.gated_scan_fwd(x.double(), x.double(), off), lambda: ssc.gated_scan_fwd(x[:, :6].contiguous(), x[:, :6].contiguous(), off)):
        with pytest.raises((ssc.SSCError, ValueError)):
            call()


def test_every_launch_is_made_on_its_tensors_device():
    tree = ast.parse(inspect.getsource(seq))
    calls = [n for n in ast.walk(tree) if isinstance(n, ast.Call) and getattr(n.func, "id", "") == "_launch"]
    assert len(calls) >= 8 and all(ast.unparse(c.args[1]) == "dev" for c in calls)
    named = [n.attr for n in ast.walk(tree) if isinstance(n, ast.Attribute) and n.attr.startswith("ssc_")]
    assert named and all(n.endswith("_workspace_bytes") for n in named)


def _double(x):
    return x.detach() * 2


def _norm_call(mp):
    mp.setattr(seq, "layer_norm_fwd", lambda x, *r: _double(x))
    mp.setattr(seq, "layer_norm_bwd", lambda x, dy, *r: (_double(dy), None, None))
    x = torch.randn(3, 8, requires_grad=True)
    return x, ssc.layer_norm(x)


def _add_call(mp):
    mp.setattr(seq, "add_layer_norm_fwd", lambda x, r, *rest: (_double(x), _double(r)))
    mp.setattr(seq, "add_layer_norm_bwd", lambda s, dy, *rest: (_double(dy), _double(dy), None, None))
    x = torch.randn(3, 8, requires_grad=True)
    return x, ssc.add_layer_norm(x, x)[0]


def _drop_call(mp):
    mp.setattr(seq, "dropout_fwd", lambda x, *r: _double(x))
    x = torch.randn(3, 8, requires_grad=True)
    return x, ssc.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64))


def _scan_call(mp):
    mp.setattr(seq, "gated_scan_fwd", lambda x, g, *r, **kw: (_double(x), torch.zeros(1, 8), torch.zeros(8)))
    mp.setattr(seq, "gated_scan_bwd", lambda x, g, c, dy, *r: (_double(dy), _double(dy), None))
    x = torch.randn(3, 8, requires_grad=True)
    return x, ssc.gated_scan(x, x, torch.tensor([0, 3], dtype=torch.int32))[0]


def _window_call(mp):
    mp.setattr(seq, "window_attention_fwd", lambda q, *r: (_double(q), torch.zeros(2, 3)))
    mp.setattr(seq, "window_attention_bwd", lambda q, k, v, *r: tuple(_double(t) for t in (q, k, v)))
    x = torch.randn(3, 2, 8, requires_grad=True)
    off = torch.tensor([0, 3], dtype=torch.int32)
    return x, ssc.window_attention(x, x, x, off, off, 1, 1)


WRAPPERS = {"LayerNormFunction": _norm_call, "AddLayerNormFunction": _add_call, "DropoutFunction": _drop_call,
            "GatedScanFunction": _scan_call, "WindowAttentionFunction": _window_call}


@pytest.mark.parametrize("call", WRAPPERS.values(), ids=WRAPPERS.keys())
def test_second_derivatives_are_refused(call, monkeypatch):
    x, y = call(monkeypatch)
    (first,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    assert torch.isfinite(first).all()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((y * y).sum() + first.square().sum()).backward()


def test_every_wrapper_is_covered():
    found = {n for n, c in vars(seq).items()
             if isinstance(c, type) and issubclass(c, torch.autograd.Function) and c.__module__ == seq.__name__}
    assert found == set(WRAPPERS)
