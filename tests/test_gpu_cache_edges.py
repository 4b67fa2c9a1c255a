"""GPU tests of attention over the paged cache where a row's sums meet their limits.  Inputs, oracle and tolerances are
tests/test_gpu_cache.py's."""

import pytest

import rank_kv_block_amd as rk
from tests.test_gpu_cache import FP8, Case, Serving, _cache_tensors, _gpu, _handle, _say  # noqa: F401 (_gpu: a fixture)

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


INFINITE = [
    # Hq, Hk, D, B, n, M, dtype, kernel: short contexts of one run, and long ones of many
    (4, 2, 64, 16, 8, 1, torch.bfloat16, "attend_stream_kernel"),
    (32, 8, 128, 16, 8, 1, torch.bfloat16, "attend_stream_kernel"),
    (8, 2, 128, 32, 70, 1, torch.bfloat16, "attend_stream_kernel"),
    (8, 2, 64, 64, 40, 6, torch.bfloat16, "attend_stream_kernel"),
    (4, 4, 128, 16, 9, 20, torch.bfloat16, "attend_stream_kernel"),
    (8, 2, 128, 16, 8, 13, torch.bfloat16, "attend_tree_kernel"),        # a wave pair for the rows
    (8, 2, 64, 32, 6, 40, torch.bfloat16, "attend_tree_kernel"),
    (16, 2, 128, 16, 130, 20, torch.bfloat16, "attend_tree_kernel"),
    (8, 1, 64, 7, 300, 64, torch.bfloat16, "attend_tree_kernel"),
    (16, 4, 128, 1024, 2, 10, torch.bfloat16, "attend_tree_kernel"),
    (4, 2, 80, 16, 20, 3, torch.bfloat16, "attend_plain_kernel"),
    (4, 1, 256, 24, 50, 1, torch.bfloat16, "attend_plain_kernel"),
    (8, 2, 128, 16, 130, 4, FP8, "attend_stream_kernel"),
    (16, 2, 64, 16, 130, 20, FP8, "attend_tree_kernel"),
    (4, 2, 80, 16, 20, 3, FP8, "attend_plain_kernel"),
]


@pytest.mark.parametrize("Hq,Hk,D,B,n,M,dtype,name", INFINITE)
def test_attend_values_that_are_not_finite(Hq, Hk, D, B, n, M, dtype, name):
    """Infinities and NaN in values that rows see, in the context and in the draft, at tokens of ordinary weight and at
    tokens whose weight is below float32's range: an infinity is that element's result, two of opposite signs and NaN
    are NaN, and every other element, sum and row keeps its bits.  (Weights are positive: e^-150 of them here.)"""
    inf, nan = float("inf"), float("nan")
    _say("not finite", Hq, Hk, D, B, n, M, dtype, name)
    length = n * B - 3
    c = Case(2, M, Hq, Hk, D, B, n, dtype, tree="tree", lens=[length, length], drafts=[M, max(1, M // 2)])
    ctx = length - M
    _aimed(c)
    far = min(ctx // 3, 640)        # whole tiles, and in the long contexts whole runs, far below the others
    for t in range(far):
        _aim(c, 0, t, -150.0)
    with _handle(Hq, Hk, D, B, c.N) as p:
        weights = name != "attend_tree_kernel" or B != 7
        assert rk.pred_attend_kernel_name(p.handle, c.kv, M, weights) == name
        c.run(p, weights)
        clean = [t.clone() for t in (c.out, c.lse, c.block_lse)]
        assert all(torch.isfinite(t).all() for t in (clean[0], clean[1][0]))
        one = inf if dtype == torch.bfloat16 else nan
        places = [(ctx - 1, 3, one), (far + 1, 5, -one), (ctx // 2, 7, nan), (far, 9, one), (ctx - 2, 9, -one), (0, 11, one),
                  (far - 1, 13, -one), (far // 2, 15, one), (1, 15, -one)]
        want = {3: one, 5: -one, 7: nan, 9: nan, 11: one, 13: -one, 15: nan}
        for t, d, value in places:
            c.v[int(c.tables[0, t // B]), t % B, :, d] = torch.tensor(value).to(dtype)
        sees = [False] * M
        if M > 1:       # a drafted token that only its own subtree sees
            t = ctx + M // 2
            c.v[int(c.tables[0, t // B]), t % B, :, 17] = torch.tensor(one).to(dtype)
            sees = [bool(w >> (M // 2) & 1) for w in c.tree[0].tolist()]
        c.run(p, weights)
        rk.pred_device_error(p.handle)
        expected = clean[0].clone()
        for d, value in want.items():
            expected[0, :, :, d] = value
        for i in range(M):
            if sees[i]:
                expected[0, i, :, 17] = one
        for d in range(D):
            same = (c.out[..., d] == expected[..., d]) | (c.out[..., d].isnan() & expected[..., d].isnan())
            assert same.all(), (d, c.out[0, :, :, d], expected[0, :, :, d])
        assert torch.equal(c.lse, clean[1]) and torch.equal(c.block_lse, clean[2])


def test_kernel_names_only_for_what_attend_takes():
    """A head size, a number of rows or a cache that pred_attend refuses has no kernel."""
    for D, M, good in ((256, 64, True), (264, 1, False), (512, 1, False), (128, 0, False), (128, 65, False)):
        with _handle(2, 1, D, 16, 2) as p:
            kv = rk.KVCache(*_cache_tensors(2, 16, 1, D, torch.bfloat16, "tokens", fill=0.0))
            if good:
                assert rk.pred_attend_kernel_name(p.handle, kv, M) == "attend_plain_kernel"
                continue
            with pytest.raises(rk.PredError):
                rk.pred_attend_kernel_name(p.handle, kv, M)
            q = torch.zeros((1, M, 2, D), dtype=torch.bfloat16, device="cuda")
            with pytest.raises(rk.PredError):
                rk.pred_attend(p.handle, kv, q, None, None, None, None, 1.0, torch.zeros_like(q))
            kv = rk.KVCache(kv.k, kv.v, 2.0, 1.0)       # a bf16 cache has scales of 1
            with pytest.raises(rk.PredError):
                rk.pred_attend_kernel_name(p.handle, kv, 1)


def test_two_graphs_keep_their_workspaces():
    """The serving step captured twice, each graph with a workspace of its own that lives as long as it does: the graphs
    take turns, other tensors come and go between the replays, and every replay is the eager step's result."""
    a, b = Serving(torch.bfloat16), Serving(torch.bfloat16)
    for w in (a, b):
        w.feed(0)
        w.device_step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        b.ws = torch.empty_like(b.ws)
        state = [t.clone() for t in (b.tables, b.mass, b.lens)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.device_step()
        graphs.append((graph, b.ws))
        for t, old in zip((b.tables, b.mass, b.lens), state):
            t.copy_(old)
    assert graphs[0][1].data_ptr() != graphs[1][1].data_ptr()
    for step in range(1, 30):
        a.feed(step)
        a.device_step()
        b.feed(step)
        others = [torch.full_like(b.ws, 255) for _ in range(4)]
        graphs[step % 2][0].replay()
        torch.cuda.synchronize()
        assert all((t == 255).all() for t in others), step
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y), step
    a.p.close()
    b.p.close()
