"""The serial block of examples/: convolution, layer norm, windowed attention, dropout and gated scans together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import sequence as S

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("serial_voxels", os.path.join(ROOT, "examples", "serial_voxels.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rng(step=0):
    return torch.tensor([7, step], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_training_runs(example, dtype):
    losses = example.train(config=1, steps=3, dtype=dtype, report=lambda *a, **k: None)
    assert len(losses) == 3 and np.isfinite(losses).all()


def test_every_parameter_has_a_gradient(example):
    data = example.inputs(1, torch.float32, DEV)
    block = example.SerialBlock(data["feats"].shape[1], 2, 40, torch.float32, DEV)
    x, last = block(**data, rng=_rng())
    (x.square().mean() + last.square().mean()).backward()
    for name, p in block.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name


def test_block_gradient_matches_differences(example):
    """A directional difference of the whole block's loss in fp32, dropout's choice held, against its gradient.  The loss is
    a mean of squares of order one: with steps of 2^-5 along a unit direction the fourth-order difference is off by the
    step's fourth power and the fp32 loss's rounding over the step, both below one part in a hundred of the slope."""
    data = example.inputs(1, torch.float32, DEV)
    block = example.SerialBlock(data["feats"].shape[1], 2, 40, torch.float32, DEV)

    def loss():
        x, last = block(**data, rng=_rng())
        return x.double().square().mean() + last.double().square().mean()

    loss().backward()
    params = list(block.parameters())
    grads = [p.grad.clone() for p in params]
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in grads))
    start = [p.detach().clone() for p in params]
    h = 2.0 ** -5
    vals = []
    with torch.no_grad():
        for s in (-2, -1, 1, 2):
            for p, p0, g in zip(params, start, grads):
                p.copy_(p0 + s * h * g / norm)
            vals.append(loss().item())
    slope = (8 * (vals[2] - vals[1]) - (vals[3] - vals[0])) / (12 * h)
    assert abs(slope - norm.item()) <= 0.01 * norm.item()


def test_the_run_of_operators_against_the_oracle():
    """Norm, windowed attention, dropout with residual and norm, scan, dropout with residual: each fed by the one before, in
    fp32, against the same run in 64 bits.  The forward errors of fp32 operators of order-one values are some thousand half
    steps of 2^-24 at most in each (sums of 64 and 130 terms, decays of up to 0.98 over the rows) and pass through maps
    whose gain is at most some ten: 2^-24 x 2^12 x 10 = 2.5e-3 of the largest value bounds them with room."""
    import sparse_submanifold_convolution_amd as ssc
    g = torch.Generator().manual_seed(1)
    lens, c, h = [130, 0, 77, 1], 64, 2
    n, p, seed = sum(lens), 0.2, 99
    off = [0, 130, 130, 207, 208]
    x, w, b = torch.randn(n, c, generator=g), 1 + 0.1 * torch.randn(c, generator=g), 0.1 * torch.randn(c, generator=g)
    gate = torch.randn(n, c, generator=g) + 1
    dx, dw, db, dgate = (t.to(DEV) for t in (x, w, b, gate))
    doff = torch.tensor(off, dtype=torch.int32, device=DEV)
    rng = torch.tensor([seed, 3], dtype=torch.int64, device=DEV)
    y = ssc.layer_norm_fwd(dx, dw, db)
    qkv = y.view(n, h, c // h)
    a, _ = ssc.window_attention_fwd(qkv, qkv, qkv, doff, doff, 20, 5, 2)
    y, s = ssc.add_layer_norm_fwd(a.reshape(n, c), dx, dw, db, p=p, rng=rng, layer=4)
    z, last, _ = ssc.gated_scan_fwd(y, dgate, doff)
    out = ssc.dropout_fwd(z, p, rng, 5, s)

    nx, nw, nb = x.double().numpy(), w.double().numpy(), b.double().numpy()
    ry, _ = S.layer_norm_fwd(nx, nw, nb, 1e-5)
    r3 = ry.reshape(n, h, c // h)
    ra, _, _ = S.window_attention_fwd(r3, r3, r3, off, off, 20, 5, 2)
    rs = S.dropout_factor(n * c, p, seed, 3, 4).reshape(n, c) * ra.reshape(n, c) + nx
    ry, _ = S.layer_norm_fwd(rs, nw, nb, 1e-5)
    rz, rlast, _ = S.gated_scan_fwd(ry, gate.double().numpy(), off)
    rout = S.dropout_factor(n * c, p, seed, 3, 5).reshape(n, c) * rz + rs
    for got, ref in ((s, rs), (z, rz), (last, rlast), (out, rout)):
        assert np.abs(got.double().cpu().numpy() - ref).max() <= 2.5e-3 * np.abs(ref).max()


def test_a_captured_training_step(example):
    """Forward and backward of the run in one graph: replayed with new steps of rng, it gives the eager passes' results."""
    import sparse_submanifold_convolution_amd as ssc
    g = torch.Generator(device=DEV).manual_seed(3)
    n, c = 3000, 64
    x, gate, up = (torch.randn(n, c, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    w = torch.ones(c, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 1000, 3000], dtype=torch.int32, device=DEV)
    rng = _rng()

    def step():
        qkv = x.view(n, 2, 32)
        a, lse = ssc.window_attention_fwd(qkv, qkv, qkv, off, off, 64, 64, 4)
        y, s = ssc.add_layer_norm_fwd(a.reshape(n, c), x, w, w, p=0.1, rng=rng)
        z, last, carries = ssc.gated_scan_fwd(y, gate, off, need_carries=True)
        out = ssc.dropout_fwd(z, 0.1, rng, 1, s)
        dz = ssc.dropout_bwd(up, 0.1, rng, 1)
        dy, dgate, _ = ssc.gated_scan_bwd(y, gate, carries, dz, off)
        da, dx, dw, db = ssc.add_layer_norm_bwd(s, dy, up, w, w, p=0.1, rng=rng)
        dq, dk, dv = ssc.window_attention_bwd(qkv, qkv, qkv, a, lse, da.view(n, 2, 32), off, off, 64, 64, 4)
        return out, last, dgate, dx, dw, db, dq, dk, dv

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        rng.copy_(_rng(i))
        x.copy_(torch.randn(n, c, generator=g, device=DEV).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b), i
