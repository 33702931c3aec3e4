"""The voxel block of examples/: convolution, norm with rotation, self and cross attention and pooling together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("voxel_attention", os.path.join(ROOT, "examples", "voxel_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_training_lowers_the_loss(example, dtype):
    losses = example.train(config=1, steps=4, dtype=dtype, report=lambda *a, **k: None)
    assert np.isfinite(losses).all() and losses[-1] < losses[0]


def test_every_parameter_has_a_gradient(example):
    data = example.inputs(1, 20, 16, torch.float32, torch.device("cuda:0"))
    block = example.VoxelBlock(data["feats"].shape[1], 2, 16, torch.float32, torch.device("cuda:0"))
    x, token = block(**data)
    (x.square().mean() + token.square().mean()).backward()
    for name, p in block.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name


def test_block_gradient_matches_differences(example):
    """A directional difference of the whole block's loss in fp32 against its gradient.  The loss is a mean of squares of
    order one: with a step of 2^-5 along a unit direction scaled by the parameter count, the fourth-order difference is
    off by the step's fourth power and the fp32 loss's rounding over the step, both below one part in a hundred of the
    slope along the gradient itself."""
    dev = torch.device("cuda:0")
    data = example.inputs(1, 20, 16, torch.float32, dev)
    block = example.VoxelBlock(data["feats"].shape[1], 2, 16, torch.float32, dev)

    def loss():
        x, token = block(**data)
        return x.double().square().mean() + token.double().square().mean()

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
