"""Rows all of whose scores are -inf: zeros, lse -inf and no gradient, while the other rows of their sample attend."""
import pytest
import torch

from test_gpu_attention import _inputs, _to, ssc  # noqa: F401  (ssc is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ql,kl,d", [([70, 9], [130, 40], 64), ([5, 3], [3000, 700], 96), ([2000], [60], 32)])
def test_scores_that_overflow(ssc, dt, ql, kl, d):
    """Finite queries and keys of 1e30 along one dimension: the product is past fp32's range on the negative side.  The
    other rows are zero along it, so that only rows 1 and (last) meet it."""
    q, k, v, do, qo, ko, _ = _inputs(71, ql, kl, 2, 1, d, dt)
    rows = [1, len(q) - 1]
    q[..., 0] = 0
    k[..., 0] = 1e30
    q[rows, :, 0] = -1e30
    q, k, v, do, qo, ko = _to(q, k, v, do, qo, ko)
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko)
    dq, dk, dv = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko)
    assert not out[rows].any() and (lse[:, rows] == -float("inf")).all() and not dq[rows].any()
    rest = [i for i in range(len(q)) if i not in rows]
    assert torch.isfinite(lse[:, rest]).all() and torch.isfinite(out).all()
    assert torch.isfinite(dk).all() and torch.isfinite(dv).all()
    do[rows] = 1000.0
    _, dk2, dv2 = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko)
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
