"""GPU tests of attention over a cache held in 4 bits against the float64 oracle, with the tolerances of
tests/test_gpu_cache.py: a 4-bit value is read without loss, so nothing is added to them."""

import math

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import cache
from tests.test_gpu_cache import Case, HALF_BF16, _f64, _handle, _rope, _say
from tests.test_gpu_norm import cache4, values4

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


class Case4(Case):
    """The same over random bytes: every code, scales that differ between the groups of a token."""

    def __init__(self, S, M, Hq, Hk, D, B, n, layout="heads", tree="chain", **kw):
        super().__init__(S, M, Hq, Hk, D, B, n, torch.bfloat16, "tokens", tree, **kw)
        self.bits = cache4(self.N, B, Hk, D, layout)
        for t in self.bits[:2]:
            t.copy_(torch.randint(0, 256, t.shape, generator=self.g, dtype=torch.uint8))
        for t in self.bits[2:]:
            t.copy_(torch.randint(122, 127, t.shape, generator=self.g, dtype=torch.uint8))
        self.kv = rk.KVCache(*self.bits[:2], 1.0, 1.0, *self.bits[2:])
        self.read()

    def read(self):
        """The values as bf16, which holds them all."""
        for x, bits, scales in (("k", 0, 2), ("v", 1, 3)):
            setattr(self, x, torch.from_numpy(values4(self.bits[bits], self.bits[scales])).bfloat16().cuda())


ATTEND = [
    # S, M, Hq, Hk, D, B, n, layout, tree, the kernel without block sums
    (1, 1, 4, 1, 64, 16, 5, "heads", "chain", "tree"),
    (3, 1, 32, 8, 128, 16, 20, "heads", "chain", "stream"),
    (3, 1, 32, 8, 128, 16, 20, "tokens", "chain", "stream"),
    (2, 1, 16, 2, 128, 32, 40, "padded", "chain", "stream"),
    (2, 1, 8, 8, 128, 64, 9, "tokens", "chain", "stream"),
    (1, 1, 40, 8, 128, 16, 130, "heads", "chain", "stream"),
    (2, 1, 8, 2, 64, 8, 33, "padded", "chain", "tree"),
    (2, 1, 8, 2, 128, 8, 33, "heads", "chain", "tree"),
    (4, 3, 20, 4, 128, 16, 12, "heads", "tree", "stream"),
    (4, 8, 8, 2, 128, 48, 7, "tokens", "bits", "stream"),
    (2, 7, 8, 2, 64, 32, 12, "heads", "bits", "tree"),
    (3, 13, 16, 2, 128, 32, 9, "tokens", "tree", "tree"),
    (2, 64, 8, 1, 128, 16, 21, "heads", "tree", "tree"),
    (2, 64, 8, 2, 64, 16, 21, "padded", "bits", "tree"),
    (2, 33, 12, 4, 128, 8, 21, "padded", "chain", "tree"),
    (2, 17, 10, 2, 64, 64, 5, "heads", "bits", "tree"),
    (2, 1, 6, 2, 96, 16, 9, "heads", "chain", "plain"),
    (2, 5, 4, 1, 256, 16, 9, "tokens", "tree", "plain"),
    (2, 2, 4, 2, 32, 7, 19, "padded", "bits", "plain"),
    (2, 2, 4, 2, 128, 7, 19, "padded", "bits", "tree"),
    (2, 3, 4, 2, 128, 24, 9, "tokens", "tree", "tree"),
    (2, 2, 4, 2, 64, 1, 70, "heads", "chain", "tree"),
    (1, 2, 4, 2, 128, 512, 2, "heads", "tree", "stream"),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("S,M,Hq,Hk,D,B,n,layout,tree,name", ATTEND)
def test_attend(S, M, Hq, Hk, D, B, n, layout, tree, name, weights):
    _say("attend 4", S, M, Hq, Hk, D, B, n, layout, tree, weights)
    c = Case4(S, M, Hq, Hk, D, B, n, layout, tree)
    with _handle(Hq, Hk, D, B, c.N) as p:
        got = rk.pred_attend_kernel_name(p.handle, c.kv, M, weights)
        _say(got)
        assert got == f"attend_{name}_kernel" or (weights and got == "attend_plain_kernel" and B not in (8, 16) and B % 32)
        c.run(p, weights)
        rk.pred_device_error(p.handle)
        c.check(weights)


@pytest.mark.parametrize("seed", range(12))
def test_attend_random_shapes(seed):
    r = np.random.default_rng(400 + seed)
    Hk, g = int(r.integers(1, 9)), int(r.integers(1, 9))
    D = int(r.choice([64, 128, 128, 32 * int(r.integers(1, 9))]))
    B = int(r.choice([8, 16, 32, 64, int(r.integers(1, 70))]))
    M = int(r.choice([1, int(r.integers(1, 65))]))
    S = int(r.integers(1, 5))
    n = max(1, min(int(r.integers(1, 3000 // B + 2)), 2 ** 20 // (S * B * Hk * D) + 1))
    n = max(n, -(-M // B))
    layout, tree = str(r.choice(["tokens", "heads", "padded"])), str(r.choice(["chain", "tree", "bits"]))
    weights = bool(r.integers(2))
    _say("attend 4 random", seed, S, M, Hk * g, Hk, D, B, n, layout, tree, weights)
    c = Case4(S, M, Hk * g, Hk, D, B, n, layout, tree, seed=seed)
    with _handle(Hk * g, Hk, D, B, c.N) as p:
        c.run(p, weights)
        rk.pred_device_error(p.handle)
        c.check(weights)


SHAPES = [(32, 8, 128, 16, 1), (16, 2, 128, 16, 3), (16, 2, 128, 16, 40), (8, 2, 64, 32, 64), (4, 1, 64, 16, 1),
          (6, 2, 96, 16, 2)]


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_attend_short_sequences(Hq, Hk, D, B, M):
    lens = [0, 1, 1, 2, B - 1, B, B + 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130]
    lens = lens + lens
    drafts = [min(M, x) for x in lens[:17]] + [min(M, x, 1 + i % 3) if i % 4 else 0 for i, x in enumerate(lens[17:])]
    _say("attend 4 short", Hq, Hk, D, B, M)
    c = Case4(len(lens), M, Hq, Hk, D, B, -(-130 // B), tree="bits" if M > 1 else "chain", lens=lens, drafts=drafts)
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        rk.pred_device_error(p.handle)
        c.check()
        assert torch.all(c.out[0] == 0) and torch.all(torch.isneginf(c.lse[0]))


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_masked_places_do_not_matter(Hq, Hk, D, B, M):
    """NaN groups past a sequence's end, in slots of no sequence and in drafted tokens that a row does not see: every row
    that does not see them keeps its bits; one that sees a NaN value is NaN in its 32 places."""
    n, S = max(5, -(-M // B) + 2), 3
    c = Case4(S, M, Hq, Hk, D, B, n, tree="tree" if M > 1 else "chain", lens=[n * B - B // 2, n * B - 1, M + 2],
              drafts=[M, max(1, M // 2), M])
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        c.check()
        clean = [t.clone() for t in (c.out, c.lse, c.block_lse)]
        for s in range(S):
            for t in range(int(c.lens[s]), n * B):
                for scales in c.bits[2:]:
                    scales[int(c.tables[s, t // B]), t % B] = 255
        used = set(c.tables.flatten().tolist())
        for page in set(range(c.N)) - used:
            for scales in c.bits[2:]:
                scales[page] = 255
        c.run(p)
        for got, want in zip((c.out, c.lse, c.block_lse), clean):
            assert torch.equal(got, want)
        # a value of the context that every row sees
        page = int(c.tables[1, 0])
        old = c.bits[3][page, 0].clone()
        c.bits[3][page, 0, :, 0] = 255
        c.run(p)
        rows = int(c.drafts[1])
        assert torch.isnan(c.out[1, :rows, :, :32]).all() and torch.isfinite(c.out[1, :rows, :, 32:]).all()
        assert torch.equal(c.out[0], clean[0][0]) and torch.equal(c.out[2], clean[0][2]) and torch.equal(c.lse, clean[1])
        c.bits[3][page, 0] = old
        if M == 1:
            return
        s, j = 0, M // 2
        t = int(c.lens[s]) - int(c.drafts[s]) + j
        page = int(c.tables[s, t // B])
        sees = [bool(int(w) >> j & 1) for w in c.tree[s].tolist()]
        for scales, value in ((c.bits[3], True), (c.bits[2], False)):
            old = scales[page, t % B].clone()
            scales[page, t % B, :, 0] = 255
            c.run(p)
            for i in range(M):
                if not sees[i]:
                    assert torch.equal(c.out[s, i], clean[0][s, i]) and torch.equal(c.lse[s, i], clean[1][s, i]), (value, i)
                elif value:
                    assert torch.isnan(c.out[s, i, :, :32]).all() and torch.isfinite(c.out[s, i, :, 32:]).all()
                    assert torch.equal(c.lse[s, i], clean[1][s, i])
                else:
                    assert torch.isnan(c.out[s, i]).all()
            assert torch.equal(c.out[1:], clean[0][1:])
            scales[page, t % B] = old


@pytest.mark.parametrize("Hq,Hk,D,B,M", [(32, 8, 128, 16, 1), (16, 2, 128, 16, 40), (4, 1, 64, 16, 1)])
def test_long_context_with_bad_entries(Hq, Hk, D, B, M):
    """Contexts of many runs; entries outside the cache are left out."""
    n, S = 700, 2
    c = Case4(S, M, Hq, Hk, D, B, n, tree="tree", lens=[n * B, n * B - 37], drafts=[M, max(1, M // 2)])
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        rk.pred_device_error(p.handle)
        c.check()
        at = [5, 70, 333, 602]
        tables = c.tables.clone()
        for x, bad in zip(at, (-1, c.N, 2 ** 31 - 1, -2 ** 31)):
            c.tables[:, x] = bad
        c.run(p)
        with pytest.raises(rk.PredError):
            rk.pred_device_error(p.handle)
        assert torch.isneginf(c.block_lse[:, at]).all()
        got = c.out.clone()
        keep = [x for x in range(n) if x not in at]
        c.tables = torch.cat((tables[:, keep], tables[:, at]), 1).contiguous()
        c.lens = c.lens - B * len(at)
        c.run(p)
        c.check()
        # one rounding of each, and sums of another order: 2^-9 of values under 4
        assert torch.all((got.float() - c.out.float()).abs() <= 2 * HALF_BF16 * c.out.float().abs() + 2.0 ** -9)


def test_serving_loop_in_4_bits():
    """Prompt and steps as a program runs them: norms, rotation and store, attention with block sums, accumulated weight,
    eviction; the cache read back is what the oracle attends over."""
    S, Hq, Hk, D, B, n, steps = 3, 8, 2, 128, 16, 6, 5
    g = torch.Generator().manual_seed(5)
    N = S * n + 2
    k, v, ks, vs = cache4(N, B, Hk, D)
    kv = rk.KVCache(k, v, 1.0, 1.0, ks, vs)
    rope, freq, _ = _rope(D)
    qw, kw = ((1 + 0.2 * torch.randn((D,), generator=g)).bfloat16().cuda() for _ in range(2))
    q_norm, k_norm = rk.Norm(qw, 1e-6), rk.Norm(kw, 1e-6)
    tables = torch.randperm(N, generator=g)[:S * n].view(S, n).int().cuda()
    lens = torch.tensor([70, 33, 64], dtype=torch.int32).cuda()
    mass, gone = torch.zeros((S, n), device="cuda"), torch.empty((S,), dtype=torch.int32, device="cuda")
    with _handle(Hq, Hk, D, B, N) as p:
        h = p.handle
        ws = torch.empty((max(1, rk.pred_attend_workspace_bytes(h, S, 1, n)),), dtype=torch.uint8, device="cuda")

        def put(tokens, positions, slots):
            q, kk, vv = (torch.randn((tokens, x, D), generator=g).bfloat16().cuda() for x in (Hq, Hk, Hk))
            out = torch.empty_like(q)
            rk.pred_norm_rotate_store(h, q_norm, k_norm, rope, q, kk, vv, positions, slots, kv, out)
            return out

        for s in range(S):
            t = torch.arange(int(lens[s]))
            put(len(t), t.int().cuda(), (tables[s].cpu().long()[t // B] * B + t % B).cuda())
        for step in range(steps):
            at = lens.cpu().long()
            slots = tables.cpu().long()[torch.arange(S), at // B] * B + at % B
            q = put(S, lens.clone(), slots.cuda())
            lens += 1
            out = torch.empty_like(q).view(S, 1, Hq, D)
            lse, block_lse = torch.empty((S, 1, Hq), device="cuda"), torch.full((S, n, 1, Hq), -math.inf, device="cuda")
            rk.pred_attend(h, kv, q.view(S, 1, Hq, D), None, tables, lens, None, D ** -0.5, out, lse, block_lse, ws)
            for s in range(S):
                length = int(lens[s])
                t = torch.arange(length)
                back = [torch.empty((length, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                rk.pred_load(h, kv, (tables[s].cpu().long()[t // B] * B + t % B).cuda(), *back)
                kk, vv = (_f64(x) for x in back)
                for x in range(Hk):
                    qq = _f64(q[s, 4 * x:4 * x + 4])
                    want, want_lse, _, absolute = cache.attend_one(qq, kk[:, x], vv[:, x], np.ones((4, length), bool), D ** -0.5)
                    rel = 2.0 ** -15 + 2 * (D + 4) * 2.0 ** -24 * D ** -0.5 * (np.abs(qq) @ np.abs(kk[:, x]).T).max()
                    assert np.all(np.abs(_f64(out[s, 0, 4 * x:4 * x + 4]) - want) <= HALF_BF16 * np.abs(want) + rel * absolute)
                    Case._close_log(_f64(lse[s, 0, 4 * x:4 * x + 4]), want_lse, rel, (step, s, x))
            rk.pred_accumulate_weight(h, lse, block_lse, None, lens, 0.9, mass)
            rk.pred_evict_blocks(h, tables, mass, lens, 4, 1, 1, tables, mass, lens, gone)
        rk.pred_device_error(h)
        assert int(lens.max()) <= 4 * B
