"""dq and dk of 16-bit attention do not carry the rounding of the forward result that delta is formed from.

delta_i = dout_i . out_i with out as it was rounded to 16 bits is off by eps_i, which meets every key of a row with one
sign (the probabilities' rounding in the forward result does too).  The dQ pass takes it out again (and the rounding of
dS with it) and hands the dK pass the corrected delta.  The bounds below hold with the correction only.  Per row, with u
half a step of the type, f = 2^-24, relative errors ep of a probability, and E = 2 (u + ep) sum |dout| sum_j P_j |v_j|, a
bound of |eps| (the result's rounding and the probabilities'):
  a product dout . v and delta are off by D_j = (d + 4) f (sum |dout v_j| + sum |dout out|);
  dS formed with the rounded delta is at most W_j = (1 + ep) (|dS_j| + P_j (E + D_j)), and differs from
  dS_j + P_j eps by at most Z_j = ep W_j + P_j D_j; rounding it adds R_j = u W_j (and half of the smallest step);
  the sum of the rounded values is eps + sum (Z_j + R_j) + n f sum W_j at most apart, so that
  dq / scale is off by sum (Z_j + R_j) (|k_j| + K) + (u + 2 ep + n f) (E + sum W_j) K + (n + d) f sum W_j |k_j|,
  K = sum P_j |k_j|: eps itself is met by no more than the rounding u of the second sum's probabilities;
  the corrected delta is off by Y = ep E + sum Z_j + n f sum W_j + 4 f sum |dout out|, so that
  dk / scale is off by sum over rows of (u + ep + n f) |dS_j| + P_j (D_j + Y) times |q_i|.
Keys share a mean and values a large one, and dout has the signs of the result's rounding, so that eps outweighs what
rounding leaves; each test also shows, on the CPU, that the same formulas with the uncorrected delta lie outside the
bounds.
"""
import numpy as np
import pytest
import torch

from test_gpu_attention import DT, F, _f64, _to, _u, ssc  # noqa: F401  (ssc is a fixture)

pytestmark = pytest.mark.gpu

FORMS = [(64, 100), (64, 1000), (48, 3000), (3, 100), (3, 3000), (2, 10000)]  # rows, few rows; none, few, many key splits


def _case(nq, nk, d, dt):
    g = torch.Generator().manual_seed(51)
    q, k, v, do = (torch.randn(n, 1, d, generator=g, dtype=torch.float64) for n in (nq, nk, nk, nq))
    q, k, v = (t.to(DT[dt]) for t in (3 * q, 1.5 + k, 48 + v))
    s = d ** -0.5 * (q[:, 0].double() @ k[:, 0].double().T)
    out = torch.softmax(s, 1) @ v[:, 0].double()
    return q, k, v, (do.abs() * torch.sign(out.to(DT[dt]).double() - out)[:, None]).to(DT[dt])


# fp16's steps are an eighth of bf16's: over heads of 128 the bound of the fp32 products nearly reaches its eps
@pytest.mark.parametrize("dt,d", [("f16", 40), ("f16", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("nq,nk", FORMS)
def test_delta_is_corrected(ssc, nq, nk, d, dt):
    q, k, v, do = _case(nq, nk, d, dt)
    off = [torch.tensor([0, n], dtype=torch.int32) for n in (nq, nk)]
    gq, gk, gv, gdo, qo, ko = _to(q, k, v, do, *off)
    out, lse = ssc.cross_attention_fwd(gq, gk, gv, qo, ko)
    dq, dk, _ = ssc.cross_attention_bwd(gq, gk, gv, out, lse, gdo, qo, ko)

    q, k, v, do = (_f64(t)[:, 0] for t in (q, k, v, do))
    scale, u, n = d ** -0.5, _u(dt), max(nq, nk)
    s = scale * (q @ k.T)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    o = p @ v
    ds = p * (do @ v.T - (do * o).sum(1, keepdims=True))
    top = scale * (np.abs(q) @ np.abs(k).T).max(1, keepdims=True)
    ep = 4 * (2 * (d + 8) * F * top + 2.0 ** -21) + n * F + 8 * F * np.abs(s).max(1, keepdims=True)
    ado = (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
    E = 2 * (u + ep) * ado  # values are positive: sum P |v| = |out|
    D = (d + 4) * F * (np.abs(do) @ np.abs(v).T + ado)
    W = (1 + ep) * (np.abs(ds) + p * (E + D))
    Z = ep * W + p * D
    # fp16: the scaled dS is at least a quarter of 2^15.5 at its bound 2 |dout| |v|, its smallest step is 2^-24
    step = 2.0 ** -38 * 2 * np.linalg.norm(do, axis=1).max() * np.linalg.norm(v, axis=1).max() if dt == "f16" else 0.0
    R = u * W + step
    K = p @ np.abs(k)
    sW = W.sum(1, keepdims=True)
    tq = (Z + R) @ np.abs(k) + (Z + R).sum(1, keepdims=True) * K + (u + 2 * ep + n * F) * (E + sW) * K
    tq = scale * (tq + (n + d) * F * (W @ np.abs(k)))
    Y = ep * E + Z.sum(1, keepdims=True) + n * F * sW + 4 * F * ado
    tk = scale * (((u + ep + n * F) * np.abs(ds) + p * (D + Y) + step).T @ np.abs(q))
    rounded = _f64(torch.from_numpy(o).to(DT[dt]))
    off = p * (do @ v.T - (do * rounded).sum(1, keepdims=True))  # dS with the uncorrected delta
    least = 2.0 ** -25 if dt == "f16" else 1e-30
    for name, got, ref, tol, bad in (("dq", dq, scale * (ds @ k), tq, scale * (off @ k)),
                                     ("dk", dk, scale * (ds.T @ q), tk, scale * (off.T @ q))):
        tol = tol + u * np.abs(ref) + least
        err = np.abs(_f64(got)[:, 0] - ref)
        assert (err <= tol).all(), f"{name}: worst |err|/tol {(err / tol).max():.3g}"
        assert (np.abs(bad - ref) > tol).any(), f"{name}: the bound would not see the uncorrected delta"
