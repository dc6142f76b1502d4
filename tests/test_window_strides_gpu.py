"""GPU: strides of o in attn_bwd_window; those of dimensions of one element are never taken."""
import pytest
import torch

import attention_forward_tiled_b200 as attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Nq,H,strides", [
    (1, 70, 4, (70 * 320 + 3, 320, 64, 1)),   # cut from a padded buffer
    (2, 1, 4, (512, 5, 64, 1)),               # one query of each
    (2, 70, 1, (70 * 128, 128, 7, 1)),        # one head
])
def test_output_with_an_odd_stride_that_is_not_taken(B, Nq, H, strides):
    g = torch.Generator().manual_seed(2)
    q, k, v, dout = (torch.randn(B, n, h, 64, generator=g).half().cuda() for n, h in ((Nq, H), (70, 1), (70, 1), (Nq, H)))
    o, lse = attn.attn_fwd_window(q, k, v, 30, 2)
    wide = torch.zeros(B * 70 * 400, dtype=torch.float16, device="cuda")
    view = wide.as_strided(o.shape, strides)
    view.copy_(o)
    assert not view.is_contiguous()
    for a, b in zip(attn.attn_bwd_window(q, k, v, view, lse, dout, 30, 2), attn.attn_bwd_window(q, k, v, o, lse, dout, 30, 2)):
        assert torch.equal(a, b)
    assert attn.get_status() == 0
