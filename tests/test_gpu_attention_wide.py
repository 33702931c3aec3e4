"""GPU parity of attention with heads of 104 to 128: the few-rows form, masks, splits and grouped heads.

Oracle and tolerances are those of the other parity cases.
"""
import pytest

from test_gpu_attention import _check, _inputs, ssc  # noqa: F401  (ssc is a fixture)

pytestmark = pytest.mark.gpu

CASES = [  # q_lens, kv_lens, heads_q, heads_kv, head_dim, mask
    ([1], [3000], 2, 2, 128, None),                  # one token over long keys: key splits
    ([1], [3000], 2, 2, 128, "random"),
    ([1, 1, 1], [600, 0, 77], 8, 2, 128, "random"),  # one token a sample, grouped heads, a sample without keys
    ([5, 3], [2100, 1300], 4, 1, 120, "random"),
    ([2], [130], 3, 3, 104, None),                   # no split
    ([190, 70], [333, 129], 4, 2, 128, "random"),    # rows: eight forward waves, a pass each for dK and dV
    ([300], [65], 4, 1, 104, "random"),
    ([64], [900], 1, 1, 128, "none left"),
    ([40], [2500], 2, 2, 120, None),                 # rows with key splits
    ([1200], [40], 2, 1, 128, "random"),             # dK and dV splits
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"q{sum(c[0])}-k{sum(c[1])}-h{c[2]}.{c[3]}-d{c[4]}-{c[5]}" for c in CASES])
def test_parity(ssc, case, dt):
    ql, kl, hq, hk, d, mask = case
    print(f"[attention] {dt} q{ql} k{kl} heads {hq}/{hk} d{d} mask {mask}", flush=True)
    _check(ssc, _inputs(41, ql, kl, hq, hk, d, dt, mask))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [40, 64])
def test_few_rows_with_a_mask(ssc, d, dt):
    """The few-rows form of heads of 33 to 64 under a mask, with and without key splits."""
    _check(ssc, _inputs(42, [2, 3], [3000, 2500], 4, 2, d, dt, "random"))
    _check(ssc, _inputs(43, [7], [100], 2, 2, d, dt, "random"))
