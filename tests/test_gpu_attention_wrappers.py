"""The differentiable attention calls on tensors that start anywhere in their buffers."""
import pytest
import torch

from test_attention_wrappers import _shifted
from test_gpu_attention import DEV, _inputs, _to, ssc  # noqa: F401  (ssc is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_flat_parameters_and_joined_losses(ssc, dt):
    """Norm, rotation and attention on parameters of a flat buffer, their results read through one joined vector: the
    gradients arrive as views that start one element in.  Every result is that of aligned tensors, bit for bit."""
    q, k, v, _, qo, ko, m = _to(*_inputs(61, [30, 9], [50, 40], 4, 2, 32, dt, "random"))
    pos = torch.arange(3 * 90, dtype=torch.int32, device=DEV).view(90, 3)
    table = ssc.rope_table((5, 5, 6), device=DEV)
    g = torch.Generator(device=DEV).manual_seed(62)
    w = (1 + 0.1 * torch.randn(4, 32, device=DEV, generator=g)).to(q.dtype)
    results = []
    for place in (lambda t: t.clone(), _shifted):
        leaves = [place(t).requires_grad_() for t in (q, k, v, w)]
        qn, _ = ssc.qk_norm_rope(leaves[0], None, pos[:39], table, leaves[3])
        _, kn = ssc.qk_norm_rope(None, leaves[1], pos, table)
        out = ssc.cross_attention(qn, kn, leaves[2], qo, ko, m)
        joined = torch.cat([out.new_zeros(1), out.flatten(), qn.flatten()])
        upstream = torch.randn(joined.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(63)).to(q.dtype)
        joined.backward(upstream)
        results.append([out.detach(), *(t.grad for t in leaves)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_first_rows_of_long_sequences(ssc):
    """Query rows further apart than a call's row strides reach: the wrapper copies them."""
    far = torch.empty((1 << 23) + 64 + 64, dtype=torch.bfloat16, device=DEV).as_strided((2, 2, 32), ((1 << 23) + 64, 32, 1))
    q, k, v, _, qo, ko, _ = _to(*_inputs(64, [1, 1], [50, 40], 2, 2, 32, "bf16"))
    far.copy_(q)
    assert torch.equal(ssc.cross_attention(far, k, v, qo, ko), ssc.cross_attention(q, k, v, qo, ko))
