"""GPU: an empty request whose rows hold 2^31 pieces of four elements."""
import math

import pytest
import torch

import attention_forward_tiled_b200 as attn

pytestmark = pytest.mark.gpu


def test_rows_of_an_empty_request_past_32_bits():
    H, Lq, d = 1 << 22, 16, 128
    q = torch.empty(1, Lq, H, d, dtype=torch.float16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.zeros(1, H, Lq, device="cuda")
    cache = torch.empty(attn.q4_cache_shape(64, 16, 1, d), dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, 64, dtype=torch.int32, device="cuda")
    attn.attn_fwd_paged_q4(q, cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), causal=True, out=out, lse=lse)
    assert attn.get_status() == 0
    assert torch.count_nonzero(out) == 0 and (lse == -math.inf).all()
