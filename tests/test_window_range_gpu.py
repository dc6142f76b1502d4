"""GPU gradients of attn_bwd_window over the range of their inputs: small and large upstream
gradients and values, where P and dS lie outside fp16's normal range.

Errors are root mean squares over a gradient, against the rounding of the exact gradient to the
type ("own").  dS enters dQ in two 16-bit parts (2^-22 of it in fp16), so dQ is off by its own
rounding alone.  dK and dV are sums of terms that are rounded once: a term's relative error and the
result's have the same size, and where the terms' signs are random their root mean squares add up
to sqrt(2) of own; half of a tenth is allowed on top.
"""
import pytest
import torch

import attention_forward_tiled_b200 as attn
from attention_forward_tiled_b200.inputs import DTYPES
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


def rms(x):
    return x.square().mean().sqrt().item()


def gradients(q, k, v, dout, window, sinks, scale=None):
    """The kernels' (dq, dk, dv), and their exact values, both float64."""
    args = [t.cuda() for t in (q, k, v)]
    o, lse = attn.attn_fwd_window(*args, window, sinks, scale=scale)
    got = attn.attn_bwd_window(*args, o, lse, dout.cuda(), window, sinks, scale=scale)
    assert attn.get_status() == 0
    exact = ref.backward(q, k, v, o.cpu(), lse.cpu(), dout, ref.visible(q.shape[1], k.shape[1], window, sinks), scale)
    return [g.cpu().to(ref.F) for g in got], exact


def check(got, exact, dtype, limits=(1.05, 1.5, 1.5), where=slice(None)):
    for name, g, e, limit in zip(("dq", "dk", "dv"), got, exact, limits):
        g, e = g[:, where], e[:, where]
        own = rms(e.to(dtype).to(ref.F) - e)
        assert torch.isfinite(g).all(), name
        assert rms(g - e) <= limit * own, f"{name}: {rms(g - e) / own:.2f} times its own rounding"


def make(B, H, Hkv, Nq, Nk, d, dtype, dout_size, v_size, seed):
    g = torch.Generator().manual_seed(seed)
    draw = lambda n, h, size: (size * torch.randn(B, n, h, d, generator=g)).to(DTYPES[dtype])  # noqa: E731
    return draw(Nq, H, 1.0), draw(Nk, Hkv, 1.0), draw(Nk, Hkv, v_size), draw(Nq, H, dout_size)


@pytest.mark.parametrize("H,Hkv,N,d,window,sinks", [
    (4, 1, 1024, 128, 256, 4),
    (2, 2, 2000, 64, 2 ** 31 - 1, 0),   # every earlier key: P of 2^-11 and less
    (3, 1, 700, 128, 2 ** 31 - 1, 0),
    (8, 2, 600, 64, 100, 200),
])
@pytest.mark.parametrize("dout_size,v_size", [(1.0, 1.0), (1e-3, 1.0), (1e-4, 1.0), (1.0, 1e-3), (50.0, 1.0)])
def test_fp16_gradients_of_small_and_large_inputs(H, Hkv, N, d, window, sinks, dout_size, v_size):
    q, k, v, dout = make(1, H, Hkv, N, N, d, "f16", dout_size, v_size, 3 + N)
    check(*gradients(q, k, v, dout, window, sinks), torch.float16)


@pytest.mark.parametrize("d", [64, 128])
def test_products_past_the_range_of_fp16(d):
    """dO V^T of some 2^21, dS past 65504, while the gradients (a small scale) are not."""
    q, k, v, dout = make(2, 4, 2, 300, 400, d, "f16", 500.0, 300.0, 5)
    got, exact = gradients(q, k, v, dout, 9, 2, scale=2.0 ** -14)
    assert all(e.abs().max() < 65504 for e in exact)
    check(got, exact, torch.float16)


def test_rows_of_different_sizes():
    """Upstream gradients of 1e-4 in the first half of the queries: their dq and the gradients of the keys that
    only they see keep their own precision."""
    N, window = 1024, 128
    q, k, v, dout = make(1, 4, 2, N, N, 128, "f16", 1.0, 1.0, 7)
    dout[:, :N // 2] = (dout[:, :N // 2].float() * 1e-4).half()
    got, exact = gradients(q, k, v, dout, window, 0)
    check(got, exact, torch.float16, where=slice(N // 2, N))
    check(got[:1], exact[:1], torch.float16, where=slice(0, N // 2))
    check(got, exact, torch.float16, where=slice(0, N // 2 - window - 128))


def test_zero_gradients_and_values():
    """dO = 0 leaves every gradient exactly zero, V = 0 (T = D = 0) dQ and dK.  dV then is a sum of products
    P dO of either sign: its error goes by the magnitudes that are summed (2^-11 of each, P's rounding), which
    can be any multiple of the sum itself, so check_backward's bound holds it."""
    for size in ((0.0, 1.0), (1.0, 0.0), (0.0, 0.0)):
        q, k, v, dout = make(1, 2, 1, 200, 300, 64, "f16", *size, 9)
        qd, kd, vd = (t.cuda() for t in (q, k, v))
        o, lse = attn.attn_fwd_window(qd, kd, vd, 100, 3)
        grads = attn.attn_bwd_window(qd, kd, vd, o, lse, dout.cuda(), 100, 3)
        assert attn.get_status() == 0
        ref.check_backward(grads, q, k, v, o.cpu(), lse.cpu(), dout, ref.visible(200, 300, 100, 3))
        assert (grads[0] == 0).all() and (grads[1] == 0).all()
        assert size[0] or (grads[2] == 0).all()


@pytest.mark.parametrize("dout_size,v_size", [(1e-6, 1.0), (1e6, 1.0), (1.0, 1e-6), (1e6, 1e6)])
def test_bf16_gradients_of_small_and_large_inputs(dout_size, v_size):
    """Values past 65504 take the split forward (few rows), as the tiled one keeps V in fp16."""
    few = v_size > 1.0
    q, k, v, dout = make(8 if few else 1, 4, 2, 16 if few else 500, 500, 128, "bf16", dout_size, v_size, 11)
    check(*gradients(q, k, v, dout, 200, 4), torch.bfloat16, limits=(1.05, 1.5, 1.5))


def test_bounds_under_captured_graphs_and_streams():
    """fp16 calls of very different sizes in two graphs and on two streams: each finds its own bounds."""
    calls, want = [], []
    for size, seed in ((1e-4, 1), (30.0, 2)):
        q, k, v, dout = (t.cuda() for t in make(2, 4, 2, 300, 500, 128, "f16", size, 1.0, seed))
        o, lse = attn.attn_fwd_window(q, k, v, 120, 4)
        out = [torch.empty_like(t) for t in (q, k, v)]
        calls.append(lambda a=(q, k, v, o, lse, dout), b=out, s=None: attn.attn_bwd_window(
            *a, 120, 4, dq=b[0], dk=b[1], dv=b[2], stream=s))
        want.append([t.clone() for t in calls[-1]()])

    def check():
        torch.cuda.synchronize()
        assert attn.get_status() == 0
        for call, w in zip(calls, want):
            for got, x in zip(call.__defaults__[1], w):
                assert torch.equal(got, x)
                got.fill_(3.0)

    check()
    graphs = []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        check()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for call, stream in zip(calls, streams):
            call(s=stream)
        check()
