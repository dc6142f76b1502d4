"""Time limits of the windowed operators and the 4-bit cache on the GPU: no large regression.

Cases and calls of perf/operators.py, timed as tests/test_zy_perf_floor.py times the dense ones.  Each
must take at most twice the time recorded for it on a B200; what the limit is for is said there.
"""
import pytest

import attention_forward_tiled_b200 as attn
from perf import operators
from tests.test_zy_perf_floor import FLOOR, seconds_per_call

pytestmark = pytest.mark.gpu

# us a call, back to back
RECORDED = {"window_fwd_4k": 336.0, "window_fwd_chunk": 35.0, "window_fwd_token": 18.5, "window_bwd_short": 36.0,
            "window_bwd_4k": 660.0, "cache_chunk": 52.0, "q4_token_4k": 39.0, "q4_draft_window": 37.5,
            "q4_token_long": 105.0}


@pytest.mark.parametrize("name", list(RECORDED))
def test_time(name, monkeypatch):
    case = next(c for c in operators.listed() if c["name"] == name)
    state = operators.prepare(case, 1)
    monkeypatch.setattr(operators, "own", True)
    us = 1e6 * seconds_per_call(lambda: operators.run(state))
    assert attn.get_status() == 0
    assert us * FLOOR <= RECORDED[name], f"{name}: {us:.1f} us against {RECORDED[name]:.1f} recorded"
    print(f"{name}: {us:.1f} us")
