"""The low-bit training example: it learns, with 8-bit moments as with 32-bit ones."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_trains_and_agrees():
    import low_bit_step as ex
    import zero_sharded_optimizer_bucket_gb300 as zs
    last = {}
    for bits in (32, 8):
        losses, model = ex.train(steps=150, bits=bits)
        first, last[bits] = sum(losses[:5]) / 5, sum(losses[-10:]) / 10
        # the untrained network is off by about the sum of both outputs'
        # variances (0.5 each); learning has to halve that at least
        assert last[bits] < 0.5 * first, (bits, first, last[bits])
        assert int(model.flags[0]) == 0 and bool(torch.isfinite(model.master).all())
    # moments of 8 bits cost little: less than half of what was learnt
    assert last[8] < 0.5 * (first + last[32])
    assert zs.zs_device_wait_timeouts() == 0


def test_first_step_of_both_forms():
    """From zero moments the first update is the same number with 8-bit moments as with 32-bit ones."""
    import low_bit_step as ex
    a, b = (ex.train(steps=1, bits=bits)[1].master for bits in (8, 32))
    assert torch.allclose(a, b, rtol=1e-5, atol=1e-7)
