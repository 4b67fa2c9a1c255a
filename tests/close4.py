"""What a 4-bit cache may hold for values known within a slack, signs included."""

import numpy as np

from tests.test_gpu_norm import _close4


def close4(got, want, slack, what):
    """_close4, which compares magnitudes where a rounding is in doubt, and the signs: a held value that is not zero has that
    of the value it stands for, unless the slack leaves it open."""
    _close4(got, want, slack, what)
    clear = (np.abs(want) > slack) & (got != 0)
    assert np.array_equal(np.signbit(got[clear]), np.signbit(want[clear])), (what, "sign")
