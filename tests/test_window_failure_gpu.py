"""Failure detection of the windowed kernels and of attention over the 4-bit cache, without faulting the GPU.

The test hook lets the first tile of each CTA never count as landed, so the bounded wait for it runs
out after a short limit: the call must record ATTN_ERR_TIMEOUT, every warp must leave its loops, and
the context must stay usable: the same call then gives what it gave before.
"""
import pytest
import torch

import attention_forward_tiled_b200 as attn
from attention_forward_tiled_b200.inputs import DTYPES
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


def make(B, H, Hkv, Nq, Nk, d, dtype):
    g = torch.Generator().manual_seed(Nq + Nk)
    return [torch.randn(B, n, h, d, generator=g).to(DTYPES[dtype]).cuda()
            for n, h in ((Nq, H), (Nk, Hkv), (Nk, Hkv), (Nq, H))]


def expires(call):
    want = call()
    assert attn.get_status() == attn.ATTN_OK
    attn.debug_set(inject=1, wait_timeout_ns=20_000_000)  # 20 ms limit per wait
    try:
        call()
        status = attn.get_status()
    finally:
        attn.debug_set(0, 0)
    assert status == attn.ATTN_ERR_TIMEOUT
    assert attn.get_status() == attn.ATTN_OK  # reading the word cleared it
    for _ in range(2):
        got = call()
        assert attn.get_status() == attn.ATTN_OK
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,dtype,window,sinks", [
    (1, 4, 2, 300, 500, 128, "f16", 100, 4),
    (1, 4, 2, 300, 500, 64, "f16", 100, 4),
    (1, 8, 1, 200, 400, 128, "bf16", 50, 0),
    (1, 8, 1, 200, 400, 64, "bf16", 50, 0),
    (60, 4, 1, 256, 256, 128, "f16", 64, 2),      # several units to a CTA, some of one tile
    (2, 8, 2, 1, 2000, 128, "f16", 1500, 4),      # split: parts of an item
    (160, 4, 2, 1, 900, 64, "bf16", 800, 0),      # runs of several items
    (3, 4, 1, 1, 300, 128, "bf16", 200, 0),       # a CTA an item
])
def test_forward(B, H, Hkv, Nq, Nk, d, dtype, window, sinks):
    q, k, v, _ = make(B, H, Hkv, Nq, Nk, d, dtype)
    expires(lambda: attn.attn_fwd_window(q, k, v, window, sinks))


@pytest.mark.parametrize("B,H,Hkv,N,d,dtype,window,sinks", [
    (1, 4, 2, 300, 128, "f16", 100, 4),
    (1, 4, 1, 900, 64, "f16", 400, 3),            # queries of a key tile split over units, then joined
    (1, 4, 2, 300, 128, "bf16", 100, 4),
    (30, 8, 4, 200, 64, "bf16", 90, 0),           # several units to a CTA
])
def test_gradients(B, H, Hkv, N, d, dtype, window, sinks):
    q, k, v, dout = make(B, H, Hkv, N, N, d, dtype)
    o, lse = attn.attn_fwd_window(q, k, v, window, sinks)
    expires(lambda: attn.attn_bwd_window(q, k, v, o, lse, dout, window, sinks))


@pytest.mark.parametrize("lens,Lq,H,d,page,dtype", [
    ([1500, 70], 1, 4, 64, 16, "f16"),            # parts
    ([900] + [30] * 170, 3, 4, 64, 16, "bf16"),   # runs
    ([200, 5], 8, 8, 128, 8, "bf16"),             # a CTA an item of 32 rows
])
def test_attention_over_the_cache(lens, Lq, H, d, page, dtype):
    cache, table, sl = (t.cuda() for t in ref.make_cache(lens, 2, d, page, DTYPES[dtype], 4))
    q = torch.randn(len(lens), Lq, H, d, generator=torch.Generator().manual_seed(1)).to(DTYPES[dtype]).cuda()
    expires(lambda: attn.attn_fwd_paged_q4(q, cache, table, sl, causal=True))
