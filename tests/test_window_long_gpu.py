"""GPU: keys whose elements are counted past 2^31, and queries likewise: the window at the end and the
sinks at the start against a sequence without what lies between (it is seen by nobody)."""
import pytest
import torch

import attention_forward_tiled_b200 as attn
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Nq,window,sinks", [(1, 700, 5), (300, 200, 130)])
def test_keys_past_32_bits(Nq, window, sinks):
    d, Hkv, H, tail = 64, 2, 4, 1024
    Nk = (1 << 31) // (Hkv * d) + 1000
    g = torch.Generator().manual_seed(Nq)
    q, dout = (torch.randn(1, Nq, H, d, generator=g).half() for _ in range(2))
    small = [torch.randn(1, sinks + tail, Hkv, d, generator=g).half() for _ in range(2)]
    k, v = (torch.zeros(1, Nk, Hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 31
    for x, s in zip((k, v), small):
        x[:, :sinks], x[:, -tail:] = s[:, :sinks].cuda(), s[:, sinks:].cuda()
    see = ref.visible(Nq, sinks + tail, window, sinks)
    out, lse = attn.attn_fwd_window(q.cuda(), k, v, window, sinks)
    assert attn.get_status() == 0
    ref.check_forward(out, lse, q, *small, see)
    dq, dk, dv = attn.attn_bwd_window(q.cuda(), k, v, out, lse, dout.cuda(), window, sinks)
    assert attn.get_status() == 0
    cut = [torch.cat((x[:, :sinks], x[:, -tail:]), 1) for x in (dk, dv)]
    ref.check_backward((dq, *cut), q, *small, out.cpu(), lse.cpu(), dout, see)
    for x in (dk, dv):
        assert torch.count_nonzero(x[:, sinks:-tail]) == 0


def test_queries_past_32_bits():
    """Heads enough that q's elements pass 2^31; only the first batch's first head and the last's last have
    queries and upstream gradients (which of them run as units of one tile differs, so bits may)."""
    d, H, Nq, B = 64, 256, 520, 256
    q = torch.zeros(B, Nq, H, d, dtype=torch.float16, device="cuda")
    assert q.numel() > 1 << 31
    g = torch.Generator().manual_seed(1)
    row, dout1 = (torch.randn(Nq, d, generator=g).half().cuda() for _ in range(2))
    k, v = (torch.randn(1, Nq, 1, d, generator=g).half().cuda().expand(B, -1, 4, -1).contiguous() for _ in range(2))
    dout = torch.zeros_like(q)
    for b, h in ((0, 0), (B - 1, H - 1)):
        q[b, :, h], dout[b, :, h] = row, dout1
    out, lse = attn.attn_fwd_window(q, k, v, 100, 3)
    dq, dk, dv = attn.attn_bwd_window(q, k, v, out, lse, dout, 100, 3)
    assert attn.get_status() == 0
    see = ref.visible(Nq, Nq, 100, 3)
    cpu = lambda x, b, h: x[b:b + 1, :, h:h + 1].cpu()  # noqa: E731
    for b, h, hk in ((0, 0, 0), (B - 1, H - 1, 3)):
        args = cpu(q, b, h), cpu(k, b, hk), cpu(v, b, hk)
        ref.check_forward(cpu(out, b, h), lse[b:b + 1, h:h + 1], *args, see)
        grads = cpu(dq, b, h), cpu(dk, b, hk), cpu(dv, b, hk)
        ref.check_backward(grads, *args, cpu(out, b, h), lse[b:b + 1, h:h + 1].cpu(), cpu(dout, b, h), see)
    for x in (dq, dk, dv):
        assert torch.count_nonzero(x[1:-1]) == 0
    assert torch.count_nonzero(dq[0, :, 1:]) == 0 and torch.count_nonzero(dq[-1, :, :-1]) == 0
