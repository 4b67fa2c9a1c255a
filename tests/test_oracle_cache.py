"""Pins of the cache operators' oracle, and the library's host-only parts against it (no GPU needed)."""

import math

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import cache

KINDS = [("none", 1.0, 0.0, 0.0, 0.0), ("linear", 4.0, 0.0, 0.0, 0.0), ("ntk", 8.0, 0.0, 0.0, 0.0),
         ("llama3", 8.0, 1.0, 4.0, 8192.0), ("yarn", 16.0, 1.0, 32.0, 8192.0)]


def test_rotation_by_hand():
    """A quarter turn sends (1, 0) to (0, 1) and (0, 1) to (-1, 0); both pairings; the transpose goes back."""
    x = np.array([[[1.0, 0.0, 5.0], [0.0, 1.0, 6.0]]])
    got = cache.rotate(x, [1], np.array([math.pi / 2]))
    assert np.allclose(got, [[[0, 1, 5], [-1, 0, 6]]], atol=1e-15)
    assert np.allclose(cache.rotate(got, [1], np.array([math.pi / 2]), backward=True), x, atol=1e-15)
    y = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    f = np.array([math.pi, math.pi / 2])
    assert np.allclose(cache.rotate(y, [1], f, interleaved=True), [[[-1, -2, -4, 3]]], atol=1e-14)
    assert np.allclose(cache.rotate(y, [1], f), [[[-1, -4, -3, 2]]], atol=1e-14)
    assert np.allclose(cache.rotate(y, [3], f, mscale=2.0), [[[-2, 8, -6, -4]]], atol=1e-14)


@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("kind", KINDS, ids=[k[0] for k in KINDS])
def test_library_turns_are_the_frequencies(rot, kind):
    """turns * 2^-64 * 2 pi is the frequency.  Either side rounds a double a few times (pow, log, the interpolation's
    products: relative 2^-48 covers 32 roundings of 2^-53), and the fraction is cut to whole units of 2^-64 turns, an
    absolute 2 pi 2^-64 that is 2^-42 of the lowest frequencies here (4e-7 turns a position and below)."""
    if kind[0] == "ntk" and rot == 2:
        with pytest.raises(rk.PredError):
            rk.pred_rope_turns(rot, 500000.0, *kind)
        return
    turns, mscale = rk.pred_rope_turns(rot, 500000.0, *kind)
    want, want_scale = cache.frequencies(rot, 500000.0, *kind)
    got = turns.astype(np.float64) * 2.0 ** -64 * 2 * math.pi
    assert turns.dtype == np.uint64 and turns.shape == (rot // 2,)
    assert np.all(np.abs(got - want) <= 2.0 ** -48 * want + 2 * math.pi * 2.0 ** -64), np.abs(got / want - 1).max()
    assert mscale == np.float32(want_scale)


def test_far_positions_keep_their_angle():
    """The angle of a far position from the integer product, against the same frequency in exact rational arithmetic:
    off by the position times the fraction's own error, 2^-53 relative and 2^-64 turns."""
    from fractions import Fraction
    turns, _ = rk.pred_rope_turns(128, 10000.0)
    f, _ = cache.frequencies(128, 10000.0)
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    for pos in (1, 1000003, 2 ** 31 - 1, -7):
        for i in (0, 13, 63):
            got = Fraction((pos * int(turns[i])) % 2 ** 64, 2 ** 64)
            want = pos * Fraction(float(f[i])) / two_pi
            off = abs((got - want + Fraction(1, 2)) % 1 - Fraction(1, 2))
            assert off <= abs(pos) * (Fraction(2) ** -50 * Fraction(float(f[i])) + Fraction(2) ** -64)


def test_scaling_endpoints():
    """llama3: short wavelengths keep their frequency, long ones are divided; yarn: the first pairs keep theirs,
    the last are divided; a factor of 1 changes nothing."""
    base, _ = cache.frequencies(128, 500000.0)
    f, _ = cache.frequencies(128, 500000.0, "llama3", 8.0, 1.0, 4.0, 8192.0)
    assert f[0] == base[0] and f[-1] == base[-1] / 8 and np.all(np.diff(f) < 0)
    f, m = cache.frequencies(128, 500000.0, "yarn", 16.0, 1.0, 32.0, 8192.0)
    assert f[0] == base[0] and abs(f[-1] - base[-1] / 16) < 1e-18 and abs(m - (1 + 0.1 * math.log(16))) < 1e-15
    for kind in ("linear", "ntk"):
        assert np.allclose(cache.frequencies(128, 1e4, kind, 1.0)[0], cache.frequencies(128, 1e4)[0], rtol=1e-15)


@pytest.mark.parametrize("args", [(3, 1e4), (0, 1e4), (65538, 1e4), (64, 1.0), (64, float("nan")), (64, float("inf")),
                                  (64, 1e4, 9), (64, 1e4, "linear", 0.0), (64, 1e4, "ntk", -1.0),
                                  (64, 1e4, "linear", float("inf")), (64, 1e4, "llama3", 8.0, 4.0, 1.0, 8192.0),
                                  (64, 1e4, "llama3", 8.0, 1.0, 4.0, 0.0), (64, 1e4, "yarn", 8.0, 0.0, 32.0, 8192.0),
                                  (64, 1e4, "yarn", 8.0, 1.0, 32.0, float("nan"))])
def test_turns_refusals(args):
    with pytest.raises(rk.PredError) as e:
        rk.pred_rope_turns(*args)
    assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE


def test_null_handles_are_refused():
    lib = rk.lib()
    null = rk.PRED_ERR_NULL_ARG
    assert lib.pred_rope_turns(64, 1e4, None, None, None) == null
    assert lib.pred_rotate(None, None, None, 0, 1, 1, None, None, 0, None) == null
    assert lib.pred_rotate_store(None, None, None, 0, None, 0, None, 0, 1, None, None, None, None, None) == null
    assert lib.pred_attend(None, None, None, 1, None, None, 1, 1, None, None, 1.0, None, None, None, None, 0, None) == null
    assert lib.pred_accumulate_weight(None, None, None, 1, None, None, 1, 1, 1.0, None, None, None) == null
    assert lib.pred_evict_blocks(None, None, None, None, 1, 1, 1, 0, 1, None, None, None, None, None, 0, None) == null
    assert lib.pred_attend_workspace_bytes(None, 1, 1, 1) == 0
    assert lib.pred_attend_kernel_name(None, None, 1, 0) is None


def test_evict_workspace_sizes():
    assert rk.pred_evict_workspace_bytes(32768, 64) == 0
    assert rk.pred_evict_workspace_bytes(32769, 3) == 32769 * 3 * 8
    assert rk.pred_evict_workspace_bytes(40000, 0) == 0


def test_e4m3_table():
    v = cache.e4m3_values()
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and v[0xB8] == -1
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and np.isfinite(np.delete(v, [0x7F, 0xFF])).all()
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, v, equal_nan=True)


def test_softmax_by_hand():
    """Two tokens with scores 0 and log 3 weigh 1/4 and 3/4; a row that sees neither has output 0 and lse -inf."""
    q = np.array([[1.0], [1.0], [1.0]])
    k, v = np.array([[0.0], [math.log(3)]]), np.array([[4.0], [-8.0]])
    seen = np.array([[True, True], [True, False], [False, False]])
    out, lse, x, absolute = cache.attend_one(q, k, v, seen, 1.0)
    assert np.allclose(out[:, 0], [1 - 6, 4, 0]) and np.allclose(lse[:2], [math.log(4), 0]) and lse[2] == -np.inf
    assert np.allclose(absolute[0], 1 + 6)
    blocks = cache.block_lse_one(x, 1)
    assert blocks.shape == (2, 3) and blocks[1, 1] == -np.inf and abs(blocks[1, 0] - math.log(3)) < 1e-15


def test_what_rows_see():
    see = cache.seen_by(4, 5, 3, None)
    assert see.astype(int).tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0]]
    see = cache.seen_by(3, 5, 3, [1, 0b11, 0b101])
    assert see.astype(int).tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 0, 1]]
    assert not cache.seen_by(2, 0, 0, None).any()


def test_eviction_by_hand():
    """Blocks 1 .. 3 of 5 may go; the budget takes two: the lowest, and of two equal ones the lower index."""
    table, mass = [10, 11, 12, 13, 14, 99], [0.0, 3.0, 2.0, 2.0, 0.0, 7.0]
    got = cache.evict(table, mass, 5 * 4 - 1, 4, 4, 1, 1)
    assert got == ([10, 11, 13, 14, 12, 99], [0.0, 3.0, 2.0, 0.0, 0.0, 7.0], 15, 1)
    got = cache.evict(table, mass, 20, 4, 1, 1, 1)      # all candidates, no more
    assert got == ([10, 14, 11, 12, 13, 99], [0.0, 0.0, 0.0, 0.0, 0.0, 7.0], 8, 3)
    nan = cache.evict([0, 1, 2], [1.0, float("nan"), -1.0], 12, 4, 2, 0, 1)
    assert nan[0] == [0, 2, 1] and nan[3] == 1
    assert cache.evict([5], [1.0], 0, 4, 0, 0, 1) == ([5], [1.0], 0, 0)


def test_weights_of_all_blocks_sum_to_the_rows():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(6, 40))
    blocks = cache.block_lse_one(x, 7)
    lse = np.log(np.exp(x).sum(1))
    mass = cache.accumulate(np.zeros(6), lse.reshape(3, 2), blocks.reshape(6, 3, 2), 6, 0.5, [0, 2])
    assert abs(mass.sum() - 4) < 1e-12      # two accepted rows of two heads, each a whole softmax
