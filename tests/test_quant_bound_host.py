"""How far the values of an appended block may be off, as paged_quant.h states it:
half a step of a code when a token is written, and half a step of the least codes
each time that the block's scale grows after that."""

import numpy as np
import pytest

from oracle import quant_cache as Q


def _appends(seed, sizes, D=256):
    """A block's 16 tokens written one by one, of these sizes: (values, held, scale)."""
    g = np.random.default_rng(seed)
    codes, scale = np.zeros((1, 16, 1, D), dtype=np.uint8), np.zeros((1, 1, 1))
    x = g.standard_normal((16, 1, D)) * np.asarray(sizes)[:, None, None]
    for i in range(16):
        Q.store(x[i:i + 1], [i], codes, scale)
    return x, Q.dequantised(codes, scale)[0], float(scale[0, 0, 0])


@pytest.mark.parametrize("growth", [1.0, 1.7, 2.0, 3.3, 8.0])
def test_bound_of_an_appended_block(growth):
    past = 0
    for seed in range(20):
        x, held, scale = _appends(seed, growth ** np.arange(16.0))
        off = np.abs(held - x)
        # 2^-4 of the value or 2^-10 of the scale that it was written with, the last one at most, and
        # 2^-10 x (new + new / 2 + ..) of the growths
        assert (off <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale) + 2.0 ** -9 * scale).all()
        past += int((off > np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)).sum())
    # (the first part alone does not bound them)
    assert past > 0


def test_growths_add_less_than_a_step_of_the_least_codes():
    # one value against the codes that it goes through, scale by scale: every start, ten doublings
    for start in Q.MAGNITUDES:
        held, s = start, 1.0
        for _ in range(10):
            s *= 2.0
            now = float(Q.values(Q.encode(np.array([held / s])))[0]) * s
            assert abs(now - held) <= 2.0 ** -10 * s
            held = now
            assert abs(held - start) < 2.0 ** -9 * s
