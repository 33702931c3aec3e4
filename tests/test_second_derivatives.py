"""The autograd wrappers have first derivatives only, and say so when a second is asked for.

The raw calls are replaced by stand-ins on the host: what is tested is what autograd records around them.
"""
import types

import pytest
import torch

import sparse_submanifold_convolution_amd as ssc
from sparse_submanifold_convolution_amd import attention as att
from sparse_submanifold_convolution_amd import binding as bind


def _attention(monkeypatch):
    monkeypatch.setattr(att, "cross_attention_fwd", lambda q, k, v, *r: (q.detach() * 2, torch.zeros(2, 3)))
    monkeypatch.setattr(att, "cross_attention_bwd", lambda q, k, v, *r: tuple(t.detach() * 2 for t in (q, k, v)))
    x = [torch.randn(3, 2, 8, requires_grad=True) for _ in range(3)]
    off = torch.tensor([0, 3], dtype=torch.int32)
    return x[0], ssc.cross_attention(*x, off, off)


def _norm_rope(monkeypatch):
    monkeypatch.setattr(att, "qk_norm_rope_fwd", lambda q, k, *r: (q.detach() * 2, k.detach() * 2))
    monkeypatch.setattr(att, "qk_norm_rope_bwd", lambda q, k, p, t, dq, dk, *r, **kw: (dq.detach() * 2, dk.detach() * 2, None, None))
    x = [torch.randn(3, 2, 8, requires_grad=True) for _ in range(2)]
    return x[0], sum(ssc.qk_norm_rope(*x))


def _subm(monkeypatch):
    monkeypatch.setattr(bind, "subm_conv3d_fwd", lambda plan, f, w, b: f.detach() * 2)
    monkeypatch.setattr(bind, "subm_conv3d_bwd", lambda plan, f, w, d, **kw: (d.detach() * 2, w.detach() * 2, None))
    f, w = torch.randn(3, 8, requires_grad=True), torch.randn(27, 8, 8, requires_grad=True)
    return f, ssc.subm_conv3d(f, types.SimpleNamespace(), w)


def _sparse(monkeypatch):
    monkeypatch.setattr(bind, "sparse_conv3d_fwd", lambda plan, f, w, b: f.detach() * 2)
    monkeypatch.setattr(bind, "sparse_conv3d_bwd", lambda plan, f, w, d, **kw: (d.detach() * 2, w.detach() * 2, None))
    f, w = torch.randn(3, 8, requires_grad=True), torch.randn(27, 8, 8, requires_grad=True)
    return f, bind.SparseConv3dFunction.apply(f, w, None, types.SimpleNamespace())


def _grid(monkeypatch):
    monkeypatch.setattr(bind, "grid_sample_fwd", lambda plan, f, p: f.detach() * 2)
    monkeypatch.setattr(bind, "grid_sample_bwd", lambda plan, p, d: d.detach() * 2)
    f = torch.randn(3, 8, requires_grad=True)
    return f, ssc.grid_sample(f, types.SimpleNamespace(), torch.zeros(3, 4))


CALLS = {"CrossAttentionFunction": _attention, "QKNormRopeFunction": _norm_rope, "SubmConv3dFunction": _subm,
         "SparseConv3dFunction": _sparse, "GridSampleFunction": _grid}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())
def test_second_derivatives_are_refused(call, monkeypatch):
    """A penalty on a gradient would otherwise train as if that gradient were constant."""
    x, y = call(monkeypatch)
    (first,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    assert torch.isfinite(first).all()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((y * y).sum() + first.square().sum()).backward()


def test_every_wrapper_is_covered():
    found = {n for m in (att, bind) for n, c in vars(m).items()
             if isinstance(c, type) and issubclass(c, torch.autograd.Function) and c.__module__ == m.__name__}
    assert found == set(CALLS)
