"""The operators over serialised rows where offsets pass 32 bits: long caches, wide strides, many elements, another GPU's stream.

Each result is held to the same call on a copy of the rows at hand, whose samples do not depend on the others.
"""
import numpy as np
import pytest
import torch

from oracle import sequence as S

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ssc():
    import sparse_submanifold_convolution_amd as m
    m.lib()
    return m


def _off(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows", [3, 300])
def test_window_at_the_end_of_a_long_cache(ssc, rows):
    """40M keys of 128 bytes: the last ones lie past 2^32 bytes, and past 2^31 elements."""
    n = 40_000_000
    print(f"[window] {rows} rows at the end of {n} keys", flush=True)
    k = torch.empty(n, 1, 64, dtype=torch.bfloat16, device=DEV)
    k[:8] = torch.randn(8, 1, 64, device=DEV).to(k.dtype)
    k[-2000:] = torch.randn(2000, 1, 64, device=DEV).to(k.dtype)
    q, do = (torch.randn(rows, 2, 64, device=DEV).to(k.dtype) for _ in range(2))
    args = (_off(0, rows), _off(0, n), 500, 0, 8)
    out, lse = ssc.window_attention_fwd(q, k, k, *args)
    near = torch.cat([k[:8], k[-2000:]])
    nargs = (_off(0, rows), _off(0, 2008), 500, 0, 8)
    nout, nlse = ssc.window_attention_fwd(q, near, near, *nargs)
    assert torch.equal(out, nout) and torch.equal(lse, nlse)
    dq, dk, dv = ssc.window_attention_bwd(q, k, k, out, lse, do, *args)
    ndq, ndk, ndv = ssc.window_attention_bwd(q, near, near, nout, nlse, do, *nargs)
    assert torch.equal(dq, ndq)
    tol = 2 * torch.finfo(k.dtype).eps
    for a, b in ((dk, ndk), (dv, ndv)):   # keys lie in other tiles: sums in another order
        assert torch.allclose(a[-2000:].float(), b[-2000:].float(), rtol=tol, atol=tol)
        assert torch.allclose(a[:8].float(), b[:8].float(), rtol=tol, atol=tol)
        assert (a[8:-2000].abs().amax() == 0)


@pytest.mark.parametrize("reverse", [False, True])
def test_scan_of_strided_rows_past_32_bits(ssc, reverse):
    n, c = 3_000_000, 256
    print(f"[scan] {n} rows {3 * c} apart, reverse {reverse}", flush=True)
    both = torch.zeros(n, 3 * c, dtype=torch.bfloat16, device=DEV)
    both[-5000:] = torch.randn(5000, 3 * c, device=DEV).to(both.dtype)
    x, gate = both[:, c:2 * c], both[:, 2 * c:]
    off = _off(0, n - 5000, n - 1200, n)
    y, last, car = ssc.gated_scan_fwd(x, gate, off, None, reverse, need_carries=True)
    dy = torch.zeros(n, c, dtype=x.dtype, device=DEV)
    dy[-5000:] = torch.randn(5000, c, device=DEV).to(x.dtype)
    dx, dg, _ = ssc.gated_scan_bwd(x, gate, car, dy, off, reverse=reverse)
    ox, og, od, oo = x[-5000:].contiguous(), gate[-5000:].contiguous(), dy[-5000:].contiguous(), _off(0, 3800, 5000)
    ny, nlast, ncar = ssc.gated_scan_fwd(ox, og, oo, None, reverse, need_carries=True)
    ndx, ndg, _ = ssc.gated_scan_bwd(ox, og, ncar, od, oo, reverse=reverse)
    # rows lie in other tiles, whose maps join in another order
    tol = 2 * torch.finfo(x.dtype).eps
    for a, b in ((y[-5000:], ny), (dx[-5000:], ndx), (dg[-5000:], ndg)):
        assert torch.allclose(a.float(), b.float(), rtol=tol, atol=1e-3)
    assert torch.allclose(last[1:], nlast, rtol=1e-4, atol=1e-4)
    assert (y[:-5000] == 0).all() and (last[0] == 0).all()


def test_norm_of_rows_past_32_bits(ssc):
    n, c = 3_000_000, 256
    print(f"[norm] {n} rows {3 * c} apart", flush=True)
    both = torch.zeros(n, 3 * c, dtype=torch.bfloat16, device=DEV)
    both[-64:] = torch.randn(64, 3 * c, device=DEV).to(both.dtype)
    x, r = both[:, c:2 * c], both[:, 2 * c:]
    w = torch.randn(c, device=DEV).to(x.dtype)
    y = ssc.layer_norm_fwd(x, w)
    assert torch.equal(y[-64:], ssc.layer_norm_fwd(x[-64:].contiguous(), w))
    y, s = ssc.add_layer_norm_fwd(x, r, w)
    ny, ns = ssc.add_layer_norm_fwd(x[-64:].contiguous(), r[-64:].contiguous(), w)
    assert torch.equal(y[-64:], ny) and torch.equal(s[-64:], ns)
    dx, _, _ = ssc.layer_norm_bwd(x, s, w)
    assert torch.equal(dx[-64:], ssc.layer_norm_bwd(x[-64:].contiguous(), s[-64:].contiguous(), w)[0])


def test_dropout_of_many_elements(ssc):
    """2^32 + 11 elements: the last ones' blocks and places, from the generator itself."""
    n = (1 << 32) + 11
    print(f"[dropout] {n} elements", flush=True)
    x = torch.ones(n, dtype=torch.float16, device=DEV)
    y = ssc.dropout_fwd(x, 0.5, torch.tensor([5, 6], dtype=torch.int64, device=DEV), 2)
    tail = y[-27:].cpu().numpy()
    for e in range(n - 27, n):
        word = S.philox([e // 8, 2, 6, 0], [5, 0])[e % 8 // 2]
        assert tail[e - (n - 27)] == (2.0 if (word >> (16 * (e % 2))) & 0xFFFF >= 32768 else 0.0), e
    kept = (y[:1 << 24] != 0).double().mean().item()
    assert abs(kept - 0.5) < 5 * 0.5 / 2 ** 12  # five standard deviations
