"""CPU tests of the check that the GPU tests of stored keys use (tests/close4.py)."""

import numpy as np
import pytest

from oracle import cache
from tests.close4 import close4


def _case(seed):
    r = np.random.default_rng(seed)
    want = r.standard_normal((3, 64))
    return want, 2.0 ** -8 * np.abs(want)


@pytest.mark.parametrize("seed", range(5))
def test_takes_every_rounding_within_the_slack(seed):
    want, slack = _case(seed)
    r = np.random.default_rng(100 + seed)
    for _ in range(5):
        near = want + slack * r.uniform(-1, 1, want.shape)
        # one scale for the group, as the largest value of either end of its range gives
        codes, scales = cache.quantise(near)
        top = [cache.quantise(np.abs(want) + d * slack)[1] for d in (-1, 1)]
        if any(not np.array_equal(scales, t) for t in top):
            continue
        close4(cache.dequantise(codes, scales), want, slack, seed)
    close4(cache.dequantise(*cache.quantise(want)), want, slack, seed)


@pytest.mark.parametrize("seed", range(5))
@pytest.mark.parametrize("wrong", [np.negative, np.abs, lambda x: -np.abs(x), lambda x: 2 * x,
                                   lambda x: np.where(np.arange(x.size).reshape(x.shape) == 7, -x, x)])
def test_rejects_wrong_signs_and_sizes(seed, wrong):
    want, slack = _case(seed)
    want[0, 7] = 1.5        # which no rounding takes to zero
    got = wrong(cache.dequantise(*cache.quantise(want)))
    with pytest.raises(AssertionError):
        close4(got, want, slack, seed)
