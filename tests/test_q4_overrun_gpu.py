"""GPU: writing to a 4-bit cache whose table is too short for the sequence."""
import pytest
import torch

import attention_forward_tiled_b200 as attn
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length,new", [(33, 4), (36, 4), (40, 4), (2 ** 31 - 1, 3), (40, 40), (35, 20)])
def test_tokens_past_the_table_are_not_written(length, new):
    """A table of 32 positions: tokens that lie past it are left out, the others go to their own rows, and no
    earlier token's row is touched."""
    cache, table, _ = ref.make_cache([32], 2, 64, 16, torch.float16, 3)
    g = torch.Generator().manual_seed(new)
    k, v = torch.randn(2, 1, new, 2, 64, generator=g).half()
    want = cache.clone()
    for i in range(new):
        pos = length - new + i
        if 0 <= pos < 32:
            for h in range(2):
                ref.cache_put(want, 64, int(table[0, pos // 16]), h, pos % 16, k[0, i, h], v[0, i, h])
    got = cache.cuda()
    attn.attn_cache_write_q4(k.cuda(), v.cuda(), got, table.cuda(), torch.tensor([length], dtype=torch.int32).cuda())
    assert attn.get_status() == 0 and torch.equal(got.cpu(), want)
