"""Pins of the oracle's norms, 4-bit cache and windows, and the argument checks that need no GPU."""

import ctypes
import math

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import bf16, cache


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    assert np.allclose(cache.norm(x, None, 0.0), x / 2.5)
    assert np.allclose(cache.norm(x, np.array([1.0, 2.0, 0.0, 5.0]), 0.0, offset=1.0), [[[2.4, 4.8, 0, 0]]])
    assert np.allclose(cache.norm(0 * x, None, 1e-6), 0)


def test_norm_gradient_is_the_difference():
    """Central differences with steps of 2^-12: off by the third derivative, 2^-24 times a value of order 1."""
    r = np.random.default_rng(1)
    x, dy, w = r.standard_normal((2, 2, 8)), r.standard_normal((2, 2, 8)), r.standard_normal(8)
    freq, pos = np.array([1.0, 0.3, 0.1]), [5, -7]

    def value(x, w):
        return (cache.rotate(cache.norm(x, w, 0.1, 0.5), pos, freq, 1.3, True) * dy).sum()

    dx, dw = cache.norm_rotate_gradient(x, dy, pos, freq, w, 0.1, 0.5, 1.3, True)
    step = 2.0 ** -12
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = step
        assert abs((value(x + e, w) - value(x - e, w)) / (2 * step) - dx[at]) < 1e-5
    for j in range(8):
        e = np.zeros(8)
        e[j] = step
        assert abs((value(x, w + e) - value(x, w - e)) / (2 * step) - dw[j]) < 1e-5


def test_e2m1_by_hand():
    """Exponent and fraction of each code by the format's rule (bias 1), and the largest value's place under the scale."""
    for code in range(8):
        e, m = code >> 1, code & 1
        assert cache.E2M1[code] == (m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))
    x = np.zeros((5, 32))
    x[0, :9] = [6, -6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]         # ties: to the even code
    x[1, :2] = [6.03125, 0.5]                                      # above 6: the next power of two
    x[2, 0] = 2.0 ** -130                                          # under the least scale: 2^-125 / 32 is nearest 0
    x[3, 0] = np.inf
    x[4, 5] = 1.5 * 2.0 ** 127
    codes, scales = cache.quantise(x)
    assert scales.ravel().tolist() == [127, 128, 2, 255, 252]
    got = cache.dequantise(codes, scales)
    assert got[0, :9].tolist() == [6, -6, 4, 4, 2, 2, 1, 1, 0]
    assert got[1, :2].tolist() == [6, 0] and codes[2, 0] == 0 and np.isnan(got[3]).all() and got[4, 5] == x[4, 5]
    assert codes[0, 1] == 15 and cache.quantise(np.full((1, 32), -0.0))[0][0, 0] == 8
    assert cache.unpacked(np.array([0x72, 0x0F], np.uint8)).tolist() == [2, 7, 15, 0]


def test_quantised_values_stay():
    r = np.random.default_rng(2)
    x = bf16.decode(bf16.encode(r.standard_normal((6, 64)) * 2.0 ** r.integers(-20, 20, (6, 1))))
    codes, scales = cache.quantise(x)
    y = cache.dequantise(codes, scales)
    assert np.array_equal(cache.dequantise(*cache.quantise(y)), y)
    # half a step is at most 1 (between 4 and 6) in units of the scale
    assert np.all(np.abs(y - x) <= np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1))


def test_window_by_hand():
    see = cache.seen_in_window(3, 8, 2, 3, 1)
    assert see.astype(int).tolist() == [[1, 0, 0, 0, 1, 1, 1, 0], [1, 0, 0, 0, 0, 1, 1, 1], [0] * 8]
    assert np.array_equal(cache.seen_in_window(4, 9, 4, 100, 0), cache.seen_by(4, 9, 4, None))
    assert cache.seen_in_window(1, 5, 1, 1, 0).astype(int).tolist() == [[0, 0, 0, 0, 1]]


def test_null_handle_is_refused_before_any_device_work():
    lib = rk.lib()
    norm, kv = rk._lib.PredNorm(None, 1e-6, 0.0), rk._lib.PredKvCache()
    n, c = ctypes.byref(norm), ctypes.byref(kv)
    assert lib.pred_norm_rotate(None, n, None, 1, 64, 1, 1, None, 1, 64, None) == rk.PRED_ERR_NULL_ARG
    assert lib.pred_norm_rotate_backward(None, n, None, 1, 64, 1, 1, None, 1, 64, 1, 64, None, None, 0,
                                         None) == rk.PRED_ERR_NULL_ARG
    assert lib.pred_norm_rotate_workspace_bytes(None, 5, 5) == 0
    assert lib.pred_norm_rotate_store(None, n, n, None, 1, 64, 1, 64, 1, 64, 1, None, 1, c, 1,
                                      None) == rk.PRED_ERR_NULL_ARG
    assert lib.pred_store(None, 1, 64, 1, 64, 1, 1, c, None) == rk.PRED_ERR_NULL_ARG
    assert lib.pred_load(None, c, 1, 1, 1, 1, None) == rk.PRED_ERR_NULL_ARG
    assert lib.pred_attend_window(None, c, 1, 1, None, 1, 1, None, None, 4, 1, 1.0, 1, None, None, 0,
                                  None) == rk.PRED_ERR_NULL_ARG
    assert lib.pred_attend_window_workspace_bytes(None, 1, 1, 1, 4, 1) == 0
    assert lib.pred_attend_window_kernel_name(None, c, 1) is None
    assert "NULL" in rk.pred_last_error()
