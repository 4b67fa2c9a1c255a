"""GPU tests of attention over the paged cache where a row's sums meet their limits.  Inputs, oracle and tolerances are
tests/test_gpu_cache.py's."""

import pytest

import rank_kv_block_amd as rk
from tests.test_gpu_cache import FP8, Case, _gpu, _handle, _say  # noqa: F401 (_gpu: a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


AIM = 64.0      # the queries' first value: a key's first value times this decides its score


def _aim(c, s, token, score):
    """Makes a token of sequence s score about `score` with every query of an aimed case."""
    page = int(c.tables[s, token // c.B])
    c.k[page, token % c.B] = 0
    c.k[page, token % c.B, :, 0] = torch.tensor(score / (AIM * c.scale * c.scales[0])).to(c.k.dtype)


def _aimed(c):
    c.q *= 0.25
    c.q[..., 0] = AIM
    c.k[..., 0] = 0
    return c


WIDE = [
    # Hq, Hk, D, B, M, dtype, kernel
    (32, 8, 64, 64, 4, torch.bfloat16, "attend_stream_kernel"),
    (16, 8, 128, 64, 8, torch.bfloat16, "attend_stream_kernel"),
    (8, 8, 128, 96, 20, FP8, "attend_stream_kernel"),
    (32, 8, 64, 128, 5, FP8, "attend_stream_kernel"),
    (16, 4, 64, 96, 24, torch.bfloat16, "attend_tree_kernel"),
    (8, 4, 128, 96, 30, FP8, "attend_tree_kernel"),
    (16, 4, 128, 128, 20, torch.bfloat16, "attend_tree_kernel"),
    (8, 4, 64, 64, 64, torch.bfloat16, "attend_tree_kernel"),
    (8, 4, 64, 192, 64, FP8, "attend_tree_kernel"),
    (4, 2, 80, 96, 20, torch.bfloat16, "attend_plain_kernel"),
]


@pytest.mark.parametrize("seen", ["hidden", "first", "last"])
@pytest.mark.parametrize("Hq,Hk,D,B,M,dtype,name", WIDE)
def test_attend_wide_block_far_below_and_hidden(Hq, Hk, D, B, M, dtype, name, seen):
    """The last block's tokens lie 150 below the row's maximum, and part of it are drafted tokens that rows do not see:
    its sum is that of the tokens they do see, whichever of its tiles these are in.  Drafts of every place in the block;
    rows see no drafted token, those of the first half, or those of the last.  The batch is large enough for runs of
    several blocks, so a wave has met the maximum before."""
    S, n = 28, 16
    most = n * B
    # the draft behind the block's middle, in its last tile, over its start, filling the block as far as it goes
    ends = [most, most - B // 2 + M // 2, most - B + M, most - B + min(B, M + 32), most - 1]
    lens = [min(most, max(ends[s % 5], most - B + 1)) for s in range(S)]
    _say("wide block", Hq, Hk, D, B, M, dtype, name, seen, lens[:5])
    c = Case(S, M, Hq, Hk, D, B, n, dtype, tree="tree", lens=lens, drafts=[M] * S)
    half = (1 << (M // 2)) - 1
    word = {"hidden": 0, "first": half, "last": ((1 << M) - 1) & ~half}[seen]
    c.tree[:] = word - (1 << 64) if word >> 63 else word
    c.tree[:, 1::7] = 0         # and some rows that see none
    _aimed(c)
    for s in range(5):
        for token in range(most - B, lens[s]):
            _aim(c, s, token, -150.0)
    with _handle(Hq, Hk, D, B, c.N) as p:
        assert rk.pred_attend_kernel_name(p.handle, c.kv, M, True) == name
        c.run(p)
        rk.pred_device_error(p.handle)
        c.check(seqs=range(5))
        # finite wherever the last block holds a token of the context, which every row sees
        for s in range(5):
            if lens[s] - M > most - B:
                assert torch.isfinite(c.block_lse[s, n - 1]).all()
