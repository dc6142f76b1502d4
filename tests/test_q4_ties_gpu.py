"""GPU: codes of elements that lie a hair beside the border between two codes, against the exact
quotient in rational numbers (float64 cannot hold x - zero there: bf16 goes down to 2^-133)."""
from fractions import Fraction

import pytest
import torch

import attention_forward_tiled_b200 as attn
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


def exact_codes(row):
    """Codes of a group of 64 elements by the definition."""
    x = [Fraction(float(e)) for e in row]
    lo, hi = min(x), max(x)
    zero = Fraction(float(torch.tensor(float(lo), dtype=torch.float64).half()))
    scale = Fraction(float(torch.tensor(float((hi - lo) / 15), dtype=torch.float64).half()))
    return [min(max(round((e - zero) / scale), 0), 15) for e in x]  # round() of a Fraction: half to even


@pytest.mark.parametrize("lo,hi", [(-1.0, 29.0), (-3.0, 27.0), (-0.5, 14.5), (-6.5, 8.5), (-7.0, 23.0)])
def test_elements_beside_a_border(lo, hi):
    """zero = lo and scale = (hi - lo) / 15 put 0 on the border between two codes."""
    tiny = [s * 2.0 ** -e for e in (30, 45, 53, 60, 100, 126) for s in (1, -1)]
    row = torch.tensor([lo, hi, 0.0, -0.0] + tiny, dtype=torch.float64)
    row = torch.cat([row, torch.linspace(lo, hi, 64 - len(row), dtype=torch.float64)]).bfloat16()
    want = exact_codes(row)
    assert len(set(want[3:16])) == 2  # both codes beside the border occur
    k = row.view(1, 1, 1, 64).cuda()
    cache = torch.zeros(attn.q4_cache_shape(1, 8, 1, 64), dtype=torch.uint8, device="cuda")
    attn.attn_cache_write_q4(k, k, cache, torch.zeros(1, 1, dtype=torch.int32).cuda(),
                             torch.ones(1, dtype=torch.int32).cuda())
    assert attn.get_status() == 0
    flat = cache.cpu().view(-1)
    for at in ref.cache_offsets(cache.shape, 64, 0, 0, 0)[:2]:
        got = [int(b) >> h & 15 for b in flat[at:at + 32] for h in (0, 4)]
        assert got == want
