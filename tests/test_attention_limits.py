"""The attention calls refuse on the host what a launch cannot hold: 2^32 threads in a dimension.

Shapes just below the limit are accepted (their workspace is sized), just past it no pass is started.
"""
import pytest

from test_attention_abi import FAKE, L, _attn, _rope  # noqa: F401  (L is a fixture)

# workgroups x threads of the first refused shape, as the launch plans have them
ATTN = [
    # few rows: 65536 / 32 + 65536 + 2 tiles of one head, 256 threads: 248 heads 4.291e9, 249 heads 4.308e9
    (dict(nq=65536, nk=65536, batch=65536, d=8), 248, 249),
    # rows, forward with eight waves: 2^28 / 256 + 8194 tiles, 512 threads: 7 heads 3.79e9, 8 heads 4.33e9 (fp32, and
    # dQ: four waves and twice the tiles, 3.77e9 and 4.31e9)
    (dict(nq=1 << 28, nk=8, batch=8192, d=128, qr=1024, qh=128, kr=1024, kh=128, vr=1024, vh=128), 7, 8),
    # dK and dV: 2^28 / 128 + 8194 tiles, 256 threads, over few query rows
    (dict(nq=8, nk=1 << 28, batch=8192, d=64), 7, 8),
]


@pytest.mark.parametrize("shape,most,past", ATTN)
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_attention_refuses_launches_past_the_grid(L, shape, most, past, dt):
    for backward in (0, 1):
        assert L.ssc_cross_attn_workspace_bytes(_attn(**shape, hq=most, hk=most, dt=dt), backward) > 0
        assert L.ssc_cross_attn_workspace_bytes(_attn(**shape, hq=past, hk=past, dt=dt), backward) == 0
    sh = _attn(**shape, hq=past, hk=past, dt=dt)
    assert L.ssc_cross_attn_fwd(sh, *[FAKE] * 9, 1 << 60, None) == 2
    assert L.ssc_cross_attn_bwd(sh, *[FAKE] * 13, 1 << 60, None) == 2


@pytest.mark.parametrize("d,most", [(64, 16), (128, 8), (8, 32)])
def test_norm_rope_refuses_launches_past_the_grid(L, d, most):
    """A group of lanes (a 16-byte vector each, at least four) walks a row's heads eight at a time; with 2^28 rows less
    64, two walks of 8 lanes, one of 16 or four of 4 are just below 2^32 threads."""
    n = (1 << 28) - 64
    assert L.ssc_qk_norm_rope_workspace_bytes(_rope(n=n, d=d, pairs=0, hq=most, hk=0)) > 0
    sh = _rope(n=n, d=d, pairs=0, hq=most, hk=1)
    assert L.ssc_qk_norm_rope_workspace_bytes(sh) == 0
    assert L.ssc_qk_norm_rope_fwd(sh, *[FAKE] * 9, None) == 2
    assert L.ssc_qk_norm_rope_bwd(sh, *[FAKE] * 14, 1 << 60, None) == 2
