"""Calls of the serial operators on two streams at once, and on a stream that is not the one their tensors came from."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def ssc():
    import sparse_submanifold_convolution_amd as m
    m.lib()
    return m


def _work(ssc, seed):
    """Inputs, and a pass through every operator forward and backward."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, c = 5000, 128
    x, r, gate, up = (torch.randn(n, c, generator=g, device=DEV).to(torch.bfloat16) for _ in range(4))
    w = torch.randn(c, generator=g, device=DEV).to(torch.bfloat16)
    off = torch.tensor([0, 2000, 5000], dtype=torch.int32, device=DEV)
    rng = torch.tensor([seed, 1], dtype=torch.int64, device=DEV)

    def run():
        q = x.view(n, 2, 64)
        a, lse = ssc.window_attention_fwd(q, q, q, off, off, 100, 20, 4)
        y, s = ssc.add_layer_norm_fwd(a.reshape(n, c), r, w, w, p=0.3, rng=rng)
        z, last, car = ssc.gated_scan_fwd(y, gate, off, need_carries=True)
        d = ssc.dropout_fwd(z, 0.2, rng, 1, s)
        dx, dg, _ = ssc.gated_scan_bwd(y, gate, car, up, off)
        grads = ssc.add_layer_norm_bwd(s, dx, d, w, w, p=0.3, rng=rng)
        return (a, lse, y, s, z, last, d, dg, *grads,
                *ssc.window_attention_bwd(q, q, q, a, lse, grads[0].view(n, 2, 64), off, off, 100, 20, 4))

    return run


def test_two_streams_at_once(ssc):
    runs = [_work(ssc, i) for i in range(2)]
    want = [r() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(runs[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_backward_on_another_stream(ssc):
    """Autograd runs a backward pass on the stream its forward pass ran on; the leaves live on the default one."""
    x = torch.randn(3000, 64, device=DEV).requires_grad_()
    off = torch.tensor([0, 3000], dtype=torch.int32, device=DEV)

    def loss():
        y, last = ssc.gated_scan(ssc.layer_norm(x), x, off)
        q = y.view(3000, 1, 64)
        return ssc.window_attention(q, q, q, off, off, 30, 30, 2).square().sum() + last.sum()

    (want,) = torch.autograd.grad(loss(), x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        value = loss()
        (got,) = torch.autograd.grad(value, x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
