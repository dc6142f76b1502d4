"""GPU: attn_fwd at d = 128 where a CTA meets many tiles in a row that store nothing: pairs whose
second tile has no query (up to 128 queries, an odd number of tiles, the last pairs run tile by
tile) and tiles above the causal diagonal.  They take turns with the one staging buffer of the
tiles that store (tests/test_staging_turns.py)."""
import math

import pytest
import torch

from attention_forward_tiled_b200 import attn_fwd, get_status
from tests.test_parity_gpu import run_and_compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,Nq,Nk,dtype,causal", [
    (12, 64, 16, 300, "f16", False),    # 768 pairs, several to a CTA, each with one tile of 16 rows
    (10, 48, 128, 200, "bf16", False),
    (6, 50, 100, 513, "f16", True),
    (5, 60, 384, 130, "bf16", False),   # three tiles a head: every other pair has one
    (3, 60, 700, 20, "f16", True),      # 680 rows above the diagonal
    (4, 40, 1000, 150, "bf16", True),
])
def test_tiles_that_store_nothing(B, H, Nq, Nk, dtype, causal):
    heads = [(b, h) for b in (0, B - 1) for h in (0, H // 2, H - 1)]
    q, k, v, out, lse = run_and_compare(B, H, Nq, Nk, 128, dtype, causal, 1 / math.sqrt(128), seed=Nq + Nk,
                                        path="prefill", heads=heads)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    for _ in range(5):
        again = attn_fwd(qd, kd, vd, causal=causal, scale=1 / math.sqrt(128), path="prefill")
        assert get_status() == 0
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
