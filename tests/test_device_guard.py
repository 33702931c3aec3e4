"""Calls launch on their tensors' GPU, also where another one is current (on the host: no call here reaches a GPU)."""
import ast
import contextlib
import inspect

import pytest
import torch

from sparse_submanifold_convolution_amd import attention as att
from sparse_submanifold_convolution_amd import binding as bind


@pytest.mark.parametrize("module", [bind, att], ids=["binding", "attention"])
def test_every_launch_is_made_on_its_tensors_device(module):
    """A default stream's handle names no GPU: whatever takes a stream is called with that stream's GPU current."""
    tree = ast.parse(inspect.getsource(module))
    inside = {}
    for node in ast.walk(tree):
        if isinstance(node, ast.With):
            for item in node.items:
                if isinstance(item.context_expr, ast.Call) and getattr(item.context_expr.func, "id", "") == "_on":
                    for child in ast.walk(node):
                        inside[child] = ast.unparse(item.context_expr.args[0])
    calls = [n for n in ast.walk(tree) if isinstance(n, ast.Call) and getattr(n.func, "id", "") == "_stream"]
    assert len(calls) >= 4
    for call in calls:
        assert inside.get(call) == ast.unparse(call.args[0]), f"line {call.lineno}"


def test_the_current_device_is_switched_only_where_it_differs(monkeypatch):
    switched = []

    @contextlib.contextmanager
    def device(d):
        switched.append(d)
        yield

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("cuda:0", "cpu"):
        with bind._on(torch.device(name)):
            pass
    assert switched == []
    with bind._on(torch.device("cuda:1")):
        assert switched == [torch.device("cuda:1")]


def test_attention_calls_run_inside_the_guard(monkeypatch):
    active, seen = [], []

    @contextlib.contextmanager
    def on(device):
        active.append(device)
        yield
        active.pop()

    class Library:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 512

            def call(*args):
                assert active == [torch.device("cpu")], name
                seen.append(name)
                return 0
            return call

    monkeypatch.setattr(att, "_on", on)
    monkeypatch.setattr(att, "_stream", lambda device: 0)
    monkeypatch.setattr(att, "lib", Library)
    q, off = torch.zeros(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32)
    out, lse = att.cross_attention_fwd(q, q, q, off, off)
    att.cross_attention_bwd(q, q, q, out, lse, out, off, off)
    att.qk_norm_rope_fwd(q, q)
    att.qk_norm_rope_bwd(q, q, None, None, q, q, q_weight=torch.ones(64))
    assert seen == ["ssc_cross_attn_fwd", "ssc_cross_attn_bwd", "ssc_qk_norm_rope_fwd", "ssc_qk_norm_rope_bwd"]
