"""Calls launch on their tensors' GPU, also where another one is current (on the host: no call here reaches a GPU)."""
import ast
import contextlib
import inspect

import pytest
import torch

from sparse_submanifold_convolution_amd import attention as att
from sparse_submanifold_convolution_amd import binding as bind


def _calls(module, name):
    tree = ast.parse(inspect.getsource(module))
    return tree, [n for n in ast.walk(tree) if isinstance(n, ast.Call) and getattr(n.func, "id", "") == name]


def test_every_launch_is_made_on_its_tensors_device():
    """A default stream's handle names no GPU: whatever takes a stream is called with that stream's GPU current."""
    tree, calls = _calls(bind, "_stream")
    inside = {}
    for node in ast.walk(tree):
        if isinstance(node, ast.With):
            for item in node.items:
                if isinstance(item.context_expr, ast.Call) and getattr(item.context_expr.func, "id", "") == "_on":
                    for child in ast.walk(node):
                        inside[child] = ast.unparse(item.context_expr.args[0])
    assert len(calls) >= 16
    for call in calls:
        assert inside.get(call) == ast.unparse(call.args[0]), f"line {call.lineno}"


def test_every_attention_launch_goes_through_the_guarded_one():
    tree, calls = _calls(att, "_launch")
    assert len(calls) == 4 and all(ast.unparse(c.args[1]) == "dev" for c in calls)
    named = [n.attr for n in ast.walk(tree) if isinstance(n, ast.Attribute) and n.attr.startswith("ssc_")]
    assert named and all(n.endswith("_workspace_bytes") for n in named)


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


def test_attention_launches_switch_the_device_only_where_it_differs(monkeypatch):
    active, seen = [], []

    @contextlib.contextmanager
    def device(d):
        active.append(d)
        yield
        active.pop()

    class Library:
        @staticmethod
        def ssc_call(*args):
            seen.append((list(active), args))
            return 0

        @staticmethod
        def ssc_status_string(code):
            return b""

        @staticmethod
        def ssc_bad(*args):
            return 2

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(att, "lib", Library)
    monkeypatch.setattr(bind, "lib", Library)
    att._launch("ssc_call", torch.device("cuda:0"), 1, 2)
    att._launch("ssc_call", torch.device("cuda:1"), 3)
    assert seen == [([], (1, 2, 100)), ([torch.device("cuda:1")], (3, 101))]
    with pytest.raises(ValueError):
        att._launch("ssc_call", torch.device("cpu"), 1)
    with pytest.raises(att.SSCError):
        att._launch("ssc_bad", torch.device("cuda:0"))
