"""The attention calls reject bad arguments on the host: no call here reaches the GPU."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import sparse_submanifold_convolution_amd as ssc
    return ssc.lib()


class _RopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("n", "qr", "qh", "kr", "kh", "pr")] + \
               [(n, ctypes.c_int32) for n in ("hq", "hk", "d", "dt", "axes", "pairs", "layout", "norm", "per_head")] + \
               [("eps", ctypes.c_float)]


def _rope(**kw):
    base = dict(n=10, qr=256, qh=64, kr=256, kh=64, pr=4, hq=4, hk=4, d=64, dt=2, axes=3, pairs=30, layout=0, norm=1,
                per_head=1, eps=1e-6)
    base.update(kw)
    return ctypes.byref(_RopeShape(**base))


BAD_ROPE = [(dict(n=-1), 1), (dict(n=(1 << 28) + 1), 1), (dict(hq=-1), 1), (dict(hk=1025), 2), (dict(d=0), 1),
            (dict(d=12), 2), (dict(d=264), 2), (dict(d=6, dt=0, pairs=0), 2), (dict(dt=3), 2), (dict(pairs=33), 1),
            (dict(pairs=-1), 1), (dict(axes=0), 1), (dict(axes=9), 1), (dict(pr=-1), 1), (dict(layout=2), 2),
            (dict(layout=1, pairs=20), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(qr=-8), 1),
            (dict(qh=4), 1), (dict(kr=1 << 41), 1)]


@pytest.mark.parametrize("change,code", BAD_ROPE, ids=[str(c[0]) for c in BAD_ROPE])
def test_norm_rope_refuses_shapes_on_host(L, change, code):
    sh = _rope(**change)
    assert L.ssc_qk_norm_rope_fwd(sh, *[FAKE] * 9, None) == code
    assert L.ssc_qk_norm_rope_bwd(sh, *[FAKE] * 14, 1 << 30, None) == code
    assert L.ssc_qk_norm_rope_workspace_bytes(sh) == 0


def test_norm_rope_refuses_pointers_on_host(L):
    f, b, odd = L.ssc_qk_norm_rope_fwd, L.ssc_qk_norm_rope_bwd, ctypes.c_void_p(0x10004)
    assert f(None, *[FAKE] * 9, None) == 1
    for i in range(9):
        for v in (odd, None):
            if v is None and i in (5, 6) or v is odd and i == 2:
                continue                                   # weights may be NULL; positions need 4 bytes only
            args = [FAKE] * 9
            args[i] = v
            assert f(_rope(), *args, None) == 1, (i, v)
    assert f(_rope(), FAKE, FAKE, ctypes.c_void_p(0x10002), *[FAKE] * 6, None) == 1
    assert f(_rope(norm=0), *[FAKE] * 9, None) == 1        # weights without a norm
    assert f(_rope(n=0), *[None] * 9, None) == 0           # nothing to do
    for i in (0, 1, 3, 4, 7, 8):
        args = [FAKE] * 14
        args[i] = None
        assert b(_rope(), *args, 1 << 30, None) == 1, i
    assert b(_rope(), *[FAKE] * 14, 64, None) == 3         # workspace
    assert b(_rope(), *[FAKE] * 13, None, 1 << 30, None) == 1
    args = [FAKE] * 14
    args[5] = None
    assert b(_rope(), *args, 1 << 30, None) == 1           # a weight's gradient without the weight
    assert L.ssc_qk_norm_rope_workspace_bytes(None) == 0 and L.ssc_qk_norm_rope_workspace_bytes(_rope()) > 0


class _AttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("nq", "nk", "qr", "qh", "kr", "kh", "vr", "vh")] + \
               [(n, ctypes.c_int32) for n in ("batch", "hq", "hk", "d", "dt")] + [("scale", ctypes.c_float)]


def _attn(**kw):
    base = dict(nq=100, nk=50, qr=256, qh=64, kr=128, kh=64, vr=128, vh=64, batch=2, hq=4, hk=2, d=64, dt=2, scale=0.125)
    base.update(kw)
    return ctypes.byref(_AttnShape(**base))


BAD_ATTN = [(dict(nq=-1), 1), (dict(nk=(1 << 28) + 1), 1), (dict(batch=0), 1), (dict(batch=65537), 1), (dict(hq=0), 1),
            (dict(hq=5), 2), (dict(hq=2048, hk=1024), 2), (dict(d=136), 2), (dict(d=12), 2), (dict(d=6, dt=0), 2),
            (dict(d=0), 1), (dict(dt=-1), 2), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
            (dict(qr=-64), 1), (dict(vh=12), 1), (dict(kh=1 << 41), 1), (dict(nq=1 << 28, hq=16, hk=1), 2)]


@pytest.mark.parametrize("change,code", BAD_ATTN, ids=[str(c[0]) for c in BAD_ATTN])
def test_attention_refuses_shapes_on_host(L, change, code):
    sh = _attn(**change)
    assert L.ssc_cross_attn_fwd(sh, *[FAKE] * 9, 1 << 40, None) == code
    assert L.ssc_cross_attn_bwd(sh, *[FAKE] * 13, 1 << 40, None) == code
    assert L.ssc_cross_attn_workspace_bytes(sh, 0) == 0 and L.ssc_cross_attn_workspace_bytes(sh, 1) == 0


def test_attention_refuses_pointers_on_host(L):
    f, b, odd = L.ssc_cross_attn_fwd, L.ssc_cross_attn_bwd, ctypes.c_void_p(0x10004)
    assert f(None, *[FAKE] * 9, 1 << 40, None) == 1
    for i in range(9):
        for v in (odd, None):
            if i == 5:
                continue                                   # the mask: bytes, may be NULL
            args = [FAKE] * 9
            args[i] = v
            assert f(_attn(), *args, 1 << 40, None) == 1, (i, v)
    assert f(_attn(), *[FAKE] * 9, 8, None) == 3
    assert f(_attn(nq=0), *[None] * 9, 0, None) == 0       # nothing to do
    for i in range(13):
        args = [FAKE] * 13
        if i == 8:
            continue
        args[i] = odd
        assert b(_attn(), *args, 1 << 40, None) == 1, i
    assert b(_attn(), *[FAKE] * 13, 8, None) == 3
    assert b(_attn(), *[FAKE] * 9, None, None, None, FAKE, 0, None) == 0   # no gradient asked for
    # few rows over long keys take key splits, whose partial sums need room
    assert L.ssc_cross_attn_workspace_bytes(_attn(nq=2, nk=100000), 0) > L.ssc_cross_attn_workspace_bytes(_attn(), 0) > 0


def test_attention_python_checks():
    import torch

    import sparse_submanifold_convolution_amd as ssc
    q, k = torch.zeros(4, 2, 64), torch.zeros(6, 2, 64)
    off = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0, 6], dtype=torch.int32)
    bad = [dict(q=torch.zeros(4, 64)), dict(k=torch.zeros(6, 2, 32)), dict(v=torch.zeros(5, 2, 64)),
           dict(k=torch.zeros(6, 2, 64, dtype=torch.float16)), dict(q=torch.zeros(4, 2, 128)[..., ::2]),
           dict(q=torch.zeros(4, 2, 65)[..., 1:]), dict(q_offsets=torch.tensor([0, 4])), dict(kv_offsets=off[0][:1]),
           dict(kv_mask=torch.zeros(6)), dict(kv_mask=torch.zeros(5, dtype=torch.bool))]
    for change in bad:
        args = dict(q=q, k=k, v=k, q_offsets=off[0], kv_offsets=off[1])
        args.update(change)
        with pytest.raises(ValueError):
            ssc.cross_attention_fwd(**args)
    with pytest.raises(ssc.SSCError):
        ssc.cross_attention_fwd(q.double(), k.double(), k.double(), *off)
    table = ssc.rope_table((8, 8), device="cpu")
    pos = torch.zeros(4, 2, dtype=torch.int32)
    for kw in (dict(positions=pos), dict(table=table), dict(positions=pos.long(), table=table),
               dict(positions=pos[:3], table=table), dict(positions=pos, table=table, layout="pairs"),
               dict(q_weight=torch.ones(3, 64)), dict(q_weight=torch.ones(64).half()),
               dict(q_weight=torch.ones(64), k_weight=torch.ones(2, 64))):
        with pytest.raises(ValueError):
            ssc.qk_norm_rope_fwd(q, q, **kw)
    with pytest.raises(ValueError):
        ssc.qk_norm_rope_fwd(None, None)
    with pytest.raises(ValueError):
        ssc.rope_table((4, -1), device="cpu")


def test_norm_rope_refuses_a_launch_past_the_grid(L):
    # 2^28 rows of 2,048 heads: more workgroups than a launch takes
    assert L.ssc_qk_norm_rope_workspace_bytes(_rope(n=1 << 28, hq=1024, hk=1024)) == 0


def test_attention_refuses_tensors_off_the_gpu():
    import torch

    import sparse_submanifold_convolution_amd as ssc
    q = torch.zeros(4, 2, 64)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        ssc.cross_attention_fwd(q, q, q, off, off)
    with pytest.raises(ValueError):
        ssc.qk_norm_rope_fwd(q, q)
