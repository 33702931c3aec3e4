"""The differentiable attention calls' handling of memory, on the host: no call here reaches the GPU."""
import pytest
import torch

import sparse_submanifold_convolution_amd as ssc
from sparse_submanifold_convolution_amd import attention as att


def _shifted(t):
    """t's values in a contiguous view that starts one element into its buffer."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    view = buf[1:].view(t.shape)
    view.copy_(t)
    assert view.is_contiguous() and view.data_ptr() % 16
    return view


@pytest.fixture
def seen(monkeypatch):
    """Replaces the raw calls by stand-ins that record the tensors they are given and return zeros."""
    args = {}

    def note(**kw):
        for name, t in kw.items():
            if t is not None:
                assert t.data_ptr() % 16 == 0, f"{name} reaches the call misaligned"
                args[name] = t

    def attn_fwd(q, k, v, *rest):
        note(q=q, k=k, v=v)
        return torch.zeros(q.shape, dtype=q.dtype), torch.zeros(q.shape[1], q.shape[0])

    def attn_bwd(q, k, v, out, lse, dout, *rest):
        note(q=q, k=k, v=v, dout=dout)
        return torch.zeros(q.shape, dtype=q.dtype), torch.zeros(k.shape, dtype=k.dtype), torch.zeros(v.shape, dtype=v.dtype)

    def rope_fwd(q, k, positions, table, qw, kw, *rest):
        note(q=q, k=k, qw=qw, kw=kw)
        return torch.zeros(q.shape, dtype=q.dtype), torch.zeros(k.shape, dtype=k.dtype)

    def rope_bwd(q, k, positions, table, dqo, dko, qw, kw, *rest, **kws):
        note(q=q, k=k, dqo=dqo, dko=dko, qw=qw, kw=kw)
        return torch.zeros(q.shape, dtype=q.dtype), torch.zeros(k.shape, dtype=k.dtype), torch.zeros_like(qw), torch.zeros_like(kw)

    for name, f in (("cross_attention_fwd", attn_fwd), ("cross_attention_bwd", attn_bwd), ("qk_norm_rope_fwd", rope_fwd),
                    ("qk_norm_rope_bwd", rope_bwd)):
        monkeypatch.setattr(att, name, f)
    return args


DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dt", DTYPES)
def test_attention_takes_views_that_start_anywhere(seen, dt):
    q, k, v = (torch.randn(n, 2, 16).to(dt) for n in (3, 5, 5))
    ins = [_shifted(t).requires_grad_() for t in (q, k, v)]
    off = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([0, 5], dtype=torch.int32)
    out = ssc.cross_attention(*ins, *off)
    g = torch.randn(out.shape).to(dt)
    out.backward(_shifted(g))
    for name, t in (("q", q), ("k", k), ("v", v), ("dout", g)):
        assert torch.equal(seen[name], t)


@pytest.mark.parametrize("dt", DTYPES)
def test_norm_rope_takes_views_that_start_anywhere(seen, dt):
    q, k = (torch.randn(3, h, 16).to(dt) for h in (4, 2))
    qw, kw = (torch.randn(h, 16).to(dt) for h in (4, 2))
    ins = [_shifted(t).requires_grad_() for t in (q, k, qw, kw)]
    qo, ko = ssc.qk_norm_rope(ins[0], ins[1], q_weight=ins[2], k_weight=ins[3])
    gq, gk = torch.randn(qo.shape).to(dt), torch.randn(ko.shape).to(dt)
    torch.autograd.backward([qo, ko], [_shifted(gq), _shifted(gk)])
    for name, t in (("q", q), ("k", k), ("qw", qw), ("kw", kw), ("dqo", gq), ("dko", gk)):
        assert torch.equal(seen[name], t)


def test_attention_copies_rows_too_far_apart(seen):
    """The first rows of long sequences: row strides past what the calls take (2^23 elements)."""
    far = torch.as_strided(torch.zeros(32 + (1 << 23) + 32, dtype=torch.float16), (2, 2, 16), ((1 << 23) + 32, 16, 1))
    far.copy_(torch.randn(2, 2, 16))
    off = torch.tensor([0, 2], dtype=torch.int32)
    ssc.cross_attention(far, far, far, off, off)
    for name in "qkv":
        assert torch.equal(seen[name], far) and seen[name].stride(0) <= 1 << 23
    near = torch.zeros(1 << 23, dtype=torch.float16).as_strided((2, 2, 16), ((1 << 23) - 32, 16, 1))
    ssc.cross_attention(near, near, near, off, off)
    assert seen["q"].data_ptr() == near.data_ptr()


def test_views_the_calls_take_are_not_copied(seen):
    packed = torch.randn(4, 6, 16).to(torch.bfloat16)
    q, k, v = packed[:, :2], packed[:, 2:4], packed[:, 4:]
    off = torch.tensor([0, 4], dtype=torch.int32)
    ssc.cross_attention(q, k, v, off, off)
    for name, t in (("q", q), ("k", k), ("v", v)):
        assert seen[name].data_ptr() == t.data_ptr() and seen[name].stride() == t.stride()
