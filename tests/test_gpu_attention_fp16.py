"""fp16 attention gradients do not depend on rows they are not made of.

In fp16 dS carries a power of two that keeps it inside the type's range.  It follows the values of the sample and the
key head that dS belongs to, so the gradients of a sample and head are the same bits whatever other samples, other heads
and rows in no sample hold: the launches are the same and so is every number in them.
"""
import numpy as np
import pytest
import torch

from test_gpu_attention import DEV, _check, _inputs, _to, ssc  # noqa: F401  (ssc is a fixture)

pytestmark = pytest.mark.gpu

FORMS = [  # q_lens, kv_lens, head_dim
    ([70, 90], [130, 200], 64),           # rows
    ([3, 2], [5000, 4000], 64),           # few rows, key splits
    ([3000, 2500], [90, 60], 64),         # dK and dV splits
    ([70, 90], [130, 200], 96),           # 32-row tiles
    ([40, 33], [700, 800], 128),          # a pass each for dK and dV
]
IDS = [f"q{f[0][0]}-k{f[1][0]}-d{f[2]}" for f in FORMS]


def _run(ssc, case):
    q, k, v, do, qo, ko, m = _to(*case)
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
    return (out, *ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m))


@pytest.mark.parametrize("ql,kl,d", FORMS, ids=IDS)
@pytest.mark.parametrize("mask", [None, "random"])
def test_rows_of_no_sample_change_nothing(ssc, ql, kl, d, mask):
    """Large finite values and output gradients before the first and from the last offset."""
    q, k, v, do, qo, ko, m = _inputs(31, [5, *ql, 7], [9, *kl, 4], 4, 2, d, "f16", mask)
    qo, ko = qo[1:-1].clone(), ko[1:-1].clone()
    plain = _run(ssc, (q, k, v, do, qo, ko, m))
    v, do = v.clone(), do.clone()
    for t, off in ((v, ko), (do, qo)):
        t[:off[0]], t[off[-1]:] = 65504.0, -60000.0
    for a, b in zip(plain, _run(ssc, (q, k, v, do, qo, ko, m))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("ql,kl,d", FORMS, ids=IDS)
def test_a_sample_keeps_its_bits_beside_a_large_one(ssc, ql, kl, d):
    case = _inputs(32, ql, kl, 4, 2, d, "f16")
    plain = _run(ssc, case)
    q, k, v, do, qo, ko, m = (None if t is None else t.clone() for t in case)
    v[ko[1]:] *= 2.0 ** 7
    do[qo[1]:] *= 2.0 ** 12
    big = _run(ssc, (q, k, v, do, qo, ko, m))
    nq, nk = int(qo[1]), int(ko[1])
    for a, b, n in zip(plain, big, (nq, nq, nk, nk)):
        assert torch.equal(a[:n], b[:n])


def test_a_key_head_keeps_its_bits_beside_a_large_one(ssc):
    case = _inputs(33, [70, 9], [130, 500], 4, 2, 64, "f16", "random")
    plain = _run(ssc, case)
    q, k, v, do, qo, ko, m = (None if t is None else t.clone() for t in case)
    v[:, 1] *= 2.0 ** 7
    do[:, 2:] *= 2.0 ** 12
    big = _run(ssc, (q, k, v, do, qo, ko, m))
    for a, b, h in zip(plain, big, (2, 2, 1, 1)):
        assert torch.equal(a[:, :h], b[:, :h])


def test_a_sample_without_keys_changes_nothing(ssc):
    """Output gradients of rows whose keys are all masked, or that have none."""
    case = _inputs(34, [40, 30, 20], [200, 150, 0], 2, 2, 64, "f16")
    q, k, v, do, qo, ko, _ = case
    m = torch.ones(350, dtype=torch.bool)
    m[200:] = False
    plain = _run(ssc, (q, k, v, do, qo, ko, m))
    do = do.clone()
    do[40:] = 65504.0
    for a, b in zip(plain, _run(ssc, (q, k, v, do, qo, ko, m))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("samples,hq,hk", [(150, 2, 1), (70, 8, 8), (1, 16, 1)])
def test_samples_of_many_sizes_and_magnitudes(ssc, samples, hq, hk):
    """Ragged samples with empty ones, output gradients and values of each at its own power of two, against the oracle."""
    rng = np.random.default_rng(35)
    ql, kl = (rng.integers(0, 30, samples).tolist() for _ in range(2))
    if samples == 1:
        ql, kl = [1100], [900]
    q, k, v, do, qo, ko, m = _inputs(35, ql, kl, hq, hk, 32, "f16", "random")
    for b in range(samples):
        do[qo[b]:qo[b + 1]] *= 2.0 ** int(rng.integers(-5, 7))
        v[ko[b]:ko[b + 1]] *= 2.0 ** int(rng.integers(-3, 4))
    _check(ssc, (q, k, v, do, qo, ko, m))


def test_graph_replays_with_new_offsets(ssc):
    """A captured backward pass follows offsets and magnitudes that change between its replays."""
    q, k, v, do, _, _, m = _to(*_inputs(36, [400], [700], 4, 2, 64, "f16", "random"))
    qo, ko = (torch.tensor(o, dtype=torch.int32, device=DEV) for o in ([0, 100, 400], [0, 300, 700]))
    out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
        grads = ssc.cross_attention_bwd(q, k, v, out, lse, do, qo, ko, m)
    for i, (a, b) in enumerate([(100, 300), (1, 699), (399, 5), (0, 700), (250, 64)]):
        qo.copy_(torch.tensor([0, min(a, 400 - i), 400 - i], dtype=torch.int32))
        ko.copy_(torch.tensor([i, b, 700], dtype=torch.int32))
        do[:200] *= 2.0
        v[300:] *= 0.5
        graph.replay()
        torch.cuda.synchronize()
        eo, el = ssc.cross_attention_fwd(q, k, v, qo, ko, m)
        eager = (eo, el, *ssc.cross_attention_bwd(q, k, v, eo, el, do, qo, ko, m))
        torch.cuda.synchronize()
        for x, y in zip((out, lse, *grads), eager):
            assert torch.equal(x, y)
