"""GPU precision of attn_fwd_window as include/attn.h states it, on both sides of the limit of 32
query rows of a key/value head: errors against the rounding of the exact output, and bf16 values
below fp16's normal range."""
import pytest
import torch

import attention_forward_tiled_b200 as attn
from attention_forward_tiled_b200.inputs import DTYPES
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


def run(Nq, d, dtype, v_size, H=4, Hkv=1, Nk=900, window=500, sinks=4):
    g = torch.Generator().manual_seed(Nq + d)
    q, k, v = ((s * torch.randn(2, n, h, d, generator=g)).to(DTYPES[dtype])
               for n, h, s in ((Nq, H, 1.0), (Nk, Hkv, 1.0), (Nk, Hkv, v_size)))
    out, _ = attn.attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), window, sinks)
    assert attn.get_status() == 0
    exact, _, p, _ = ref.forward(q, k, v, ref.visible(Nq, Nk, window, sinks))
    err = out.cpu().to(ref.F) - exact
    own = exact.to(q.dtype).to(ref.F) - exact
    return err, own, exact, torch.einsum("bhqk,bkhd->bqhd", p, ref.spread(v.to(ref.F).abs(), H))


def rms(x):
    return x.square().mean().sqrt().item()


@pytest.mark.parametrize("Nq", [1, 8, 9, 300])  # 4, 32, 36 and 1200 rows
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,limit", [
    # P is rounded to fp16 (2^-11 of each term at most) and the output by as much: where the terms' signs are
    # random, each leaves the same root mean square and the two add up to sqrt(2) of one
    ("f16", 1.5),
    # P's rounding (2^-11 in the tiled kernel, 2^-16 in the other) beside the output's 2^-8: sqrt(1 + 2^-6) and less
    ("bf16", 1.02),
])
def test_error_against_the_rounding_of_the_output(Nq, d, dtype, limit):
    err, own, _, _ = run(Nq, d, dtype, 1.0)
    assert rms(err) <= limit * rms(own)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("v_size", [1e-6, 1e-12])
def test_small_bf16_values(d, v_size):
    """Up to 32 rows bf16 V is used as it is; past that it is fp16, off by 2^-25 at most, which P sums up to 2^-25."""
    err, own, _, _ = run(8, d, "bf16", v_size)
    assert rms(err) <= 1.02 * rms(own)
    err, own, exact, mag = run(9, d, "bf16", v_size)
    bound = 2.0 ** -25 + 2.0 ** -9 * mag + 2.0 ** -8 * exact.abs()
    assert (err.abs() <= bound).all()
