"""GPU tests of attention with a sliding window and sinks against the float64 oracle.

Tolerances: those of tests/test_gpu_cache.py; the chunk kernel's weights are one bf16 term, half a step of which is 2^-8
relative, so an output may be off by that times the weighted mean of the absolute values more."""

import math

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import cache
from tests.test_gpu_cache import FP8, Case, HALF_BF16, _f64, _handle, _say
from tests.test_gpu_cache4 import Case4

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16 = torch.bfloat16
ALL = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


class _Windowed:
    """A case's run and check with a window."""

    def run(self, p, window, sinks, lse=True, offset=0):
        need = rk.pred_attend_window_workspace_bytes(p.handle, self.S, self.M, self.n, window, sinks)
        ws = torch.full((max(need, 1),), 0x7F, dtype=torch.uint8, device="cuda")
        self.out.fill_(9.0)
        self.lse.fill_(9.0)
        rk.pred_attend_window(p.handle, self.kv, self.q, self.tables, self.lens, self.drafts, window, sinks, self.scale,
                              self.out, self.lse if lse else None, ws if need else None, n_blocks=self.n)

    def check(self, p, window, sinks):
        chunk = rk.pred_attend_window_kernel_name(p.handle, self.kv, self.M) == "attend_chunk_kernel"
        q, k, v = _f64(self.q), _f64(self.k) * self.scales[0], _f64(self.v) * self.scales[1]
        out, lse = _f64(self.out), _f64(self.lse)
        g = self.Hq // self.Hk
        for s in range(self.S):
            length, rows = int(self.lens[s]), int(self.drafts[s])
            pages = np.arange(-(-length // self.B)) if self.tables is None else self.tables[s, :-(-length // self.B)].cpu().numpy()
            seen = np.repeat(cache.seen_in_window(self.M, length, rows, window, sinks), g, axis=0)
            ok = (pages >= 0) & (pages < self.N)        # entries that may be anything where nothing is seen
            for b in np.nonzero(~ok)[0]:
                assert not seen[:, b * self.B:(b + 1) * self.B].any()
            pages = np.where(ok, pages, 0)
            for h in range(self.Hk):
                kk = k[pages, :, h].reshape(-1, self.D)[:length]
                vv = v[pages, :, h].reshape(-1, self.D)[:length]
                qq = q[s, :, h * g:h * g + g].reshape(-1, self.D)
                want, want_lse, absolute, delta = self._attend(qq, kk, vv, seen)
                rel = 2 * delta + 2.0 ** -20 + 2.0 ** -16 + (length + 64) * 2.0 ** -24
                got = out[s, :, h * g:h * g + g].reshape(-1, self.D)
                tol = HALF_BF16 * np.abs(want) + (rel + HALF_BF16 * chunk) * absolute
                bad = ~(np.abs(got - want) <= tol)
                assert not bad.any(), ("out", s, h, np.argwhere(bad)[:4], (np.abs(got - want) - tol).max())
                self._close_log(lse[s, :, h * g:h * g + g].reshape(-1), want_lse, rel, ("lse", s, h))

    def _attend(self, q, k, v, seen):
        """cache.attend_one for many rows, by matrices."""
        x = np.where(seen, self.scale * (q @ k.T), -np.inf) if len(k) else np.zeros(seen.shape)
        delta = (self.D + 4) * 2.0 ** -24 * self.scale * (np.abs(q) @ np.abs(k).T)[seen].max() if seen.any() else 0.0
        m = np.where(seen.any(1), x.max(1, initial=-np.inf), 0.0)
        p = np.exp(x - m[:, None])
        total = p.sum(1)
        with np.errstate(divide="ignore"):
            lse = np.where(total > 0, m + np.log(total), -np.inf)
        p = p / np.where(total > 0, total, 1.0)[:, None]
        return p @ v, lse, p @ np.abs(v), delta


class Win(_Windowed, Case):
    pass


class Win4(_Windowed, Case4):
    pass


def make(kind, S, M, Hq, Hk, D, B, n, layout="tokens", **kw):
    if kind == "fp4":
        return Win4(S, M, Hq, Hk, D, B, n, layout, **kw)
    return Win(S, M, Hq, Hk, D, B, n, FP8 if kind == "fp8" else BF16, layout, **kw)


CASES = [
    # S, M, Hq, Hk, D, B, n, kind, layout, window, sinks, the kernel
    (1, 1, 4, 1, 64, 16, 64, "bf16", "tokens", 256, 4, "stream"),
    (3, 1, 32, 8, 128, 16, 60, "bf16", "tokens", 100, 4, "stream"),
    (3, 1, 32, 8, 128, 16, 60, "fp8", "heads", 33, 0, "stream"),
    (3, 1, 32, 8, 128, 16, 60, "fp4", "heads", 200, 20, "stream"),
    (2, 4, 8, 2, 128, 32, 40, "bf16", "padded", 1, 0, "stream"),
    (2, 4, 8, 2, 64, 8, 99, "bf16", "heads", 31, 70, "stream"),
    (2, 3, 20, 4, 128, 16, 50, "fp8", "tokens", ALL, 0, "stream"),
    (2, 16, 2, 2, 128, 16, 300, "bf16", "tokens", 700, 4, "stream"),
    (3, 5, 16, 2, 128, 16, 50, "bf16", "tokens", 130, 4, "chunk"),
    (2, 1, 40, 2, 128, 16, 50, "bf16", "heads", 64, 1, "chunk"),
    (2, 1, 8, 2, 64, 16, 40, "fp4", "heads", 100, 4, "chunk"),
    (2, 3, 8, 2, 128, 7, 99, "fp8", "padded", 100, 9, "chunk"),
    (3, 100, 8, 2, 128, 16, 40, "bf16", "tokens", 100, 4, "chunk"),
    (3, 100, 8, 2, 128, 16, 40, "fp8", "heads", 64, 0, "chunk"),
    (3, 100, 8, 2, 128, 16, 40, "fp4", "tokens", 65, 130, "chunk"),
    (2, 300, 10, 2, 64, 32, 20, "bf16", "padded", 77, 4, "chunk"),
    (2, 300, 10, 2, 64, 32, 20, "fp4", "padded", 1, 1, "chunk"),
    (2, 513, 3, 3, 64, 16, 40, "fp8", "tokens", 40, 0, "chunk"),
    (1, 700, 4, 4, 128, 16, 60, "bf16", "tokens", ALL, 0, "chunk"),
    (1, 33, 300, 1, 128, 16, 10, "bf16", "tokens", 50, 4, "chunk"),
    (2, 65, 8, 1, 128, 24, 30, "bf16", "heads", 300, 4, "chunk"),
    (2, 65, 8, 1, 128, 1, 400, "bf16", "tokens", 63, 4, "chunk"),
    # groups that fill the chip: no walk is split
    (1, 2100, 32, 8, 128, 16, 160, "bf16", "heads", 700, 4, "chunk"),
    (1, 2055, 32, 8, 64, 32, 70, "fp4", "tokens", ALL, 0, "chunk"),
    (5, 1000, 28, 7, 64, 16, 64, "fp8", "tokens", 90, 4, "chunk"),
    (4, 1030, 32, 8, 128, 16, 70, "fp4", "heads", 300, 4, "chunk"),
    (2, 5, 6, 2, 80, 16, 20, "bf16", "tokens", 100, 4, "plain"),
    (2, 40, 4, 2, 256, 16, 9, "fp8", "heads", 20, 3, "plain"),
    (2, 9, 4, 2, 96, 7, 19, "fp4", "padded", 50, 10, "plain"),
]


@pytest.mark.parametrize("S,M,Hq,Hk,D,B,n,kind,layout,window,sinks,name", CASES)
def test_window(S, M, Hq, Hk, D, B, n, kind, layout, window, sinks, name):
    _say("window", S, M, Hq, Hk, D, B, n, kind, layout, window, sinks)
    c = make(kind, S, M, Hq, Hk, D, B, n, layout)
    with _handle(Hq, Hk, D, B, c.N) as p:
        assert rk.pred_attend_window_kernel_name(p.handle, c.kv, M) == f"attend_{name}_kernel"
        c.run(p, window, sinks)
        rk.pred_device_error(p.handle)
        c.check(p, window, sinks)
        out = c.out.clone()
        c.run(p, window, sinks, lse=False)
        assert torch.equal(out, c.out) and torch.all(c.lse == 9.0)


@pytest.mark.parametrize("seed", range(30))
def test_random_shapes(seed):
    r = np.random.default_rng(700 + seed)
    Hk, g = int(r.integers(1, 6)), int(r.integers(1, 9))
    kind = str(r.choice(["bf16", "fp8", "fp4"]))
    D = int(r.choice([64, 128, 128, 32 * int(r.integers(1, 9))]))
    B = int(r.choice([8, 16, 32, 64, int(r.integers(1, 70))]))
    M = int(r.choice([1, int(r.integers(1, 20)), int(r.integers(1, 400))]))
    S = int(r.integers(1, 5))
    n = max(1, min(int(r.integers(1, 2000 // B + 2)), 2 ** 20 // (S * B * Hk * D) + 1))
    n = max(n, -(-M // B))
    layout = str(r.choice(["tokens", "heads", "padded"]))
    window = int(r.choice([1, 2, int(r.integers(1, 70)), int(r.integers(1, 1500)), ALL]))
    sinks = int(r.choice([0, 1, 4, int(r.integers(0, 100)), 10 ** 9]))
    _say("window random", seed, S, M, Hk * g, Hk, D, B, n, kind, layout, window, sinks)
    c = make(kind, S, M, Hk * g, Hk, D, B, n, layout, seed=seed)
    with _handle(Hk * g, Hk, D, B, c.N) as p:
        c.run(p, window, sinks)
        rk.pred_device_error(p.handle)
        c.check(p, window, sinks)


SHAPES = [(32, 8, 128, 16, 1), (16, 2, 128, 16, 2), (16, 2, 128, 16, 40), (8, 2, 64, 32, 130), (4, 1, 64, 16, 1), (6, 2, 96, 16, 2)]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_short_sequences(Hq, Hk, D, B, M, kind):
    """Lengths around every tile's edges with rows of every number, none among them; sequences that are all rows."""
    lens = [0, 1, 1, 2, B - 1, B, B + 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 300]
    lens = lens + lens
    rows = [min(M, x) for x in lens[:18]] + [min(M, x, 1 + 7 * (i % 5)) if i % 4 else 0 for i, x in enumerate(lens[18:])]
    _say("window short", Hq, Hk, D, B, M, kind)
    c = make(kind, len(lens), M, Hq, Hk, D, B, -(-300 // B), lens=lens, drafts=rows)
    with _handle(Hq, Hk, D, B, c.N) as p:
        for window, sinks in ((1, 0), (3, 5), (32, 4), (64, 64), (129, 1), (ALL, 0)):
            c.run(p, window, sinks)
            rk.pred_device_error(p.handle)
            c.check(p, window, sinks)
            assert torch.all(c.out[0] == 0) and torch.all(torch.isneginf(c.lse[0]))


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_a_window_of_everything_is_attention(Hq, Hk, D, B, M):
    """Against pred_attend where that takes as many rows: the same tokens, one rounding each and sums of another order;
    the stream kernel's walk is the same, so its bits are."""
    M = min(M, 64)
    c = make("bf16", 3, M, Hq, Hk, D, B, max(30, M))
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p, ALL, 0)
        got = c.out.clone(), c.lse.clone()
        Case.run(c, p, False)
        same = rk.pred_attend_window_kernel_name(p.handle, c.kv, M) == rk.pred_attend_kernel_name(p.handle, c.kv, M)
        if same:
            assert torch.equal(c.out, got[0]) and torch.equal(c.lse, got[1])
        else:
            assert torch.all((c.out.float() - got[0].float()).abs() <= 3 * HALF_BF16 * c.out.float().abs() + HALF_BF16)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_masked_places_do_not_matter(Hq, Hk, D, B, M, kind):
    """NaN and infinities in tokens outside the window, past the end, in later rows' tokens and in the queries of rows past
    row_len; entries outside the cache for blocks that nobody sees, which raise no error."""
    n, S, window, sinks = max(12, -(-M // B) + 12), 3, 50, 5
    lens = [n * B - B // 2, n * B - 1, M + 60]
    c = make(kind, S, M, Hq, Hk, D, B, n, lens=lens, drafts=[M, max(1, M // 2), M])
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p, window, sinks)
        c.check(p, window, sinks)
        clean = c.out.clone(), c.lse.clone()

        def spoil(page, off, what="both"):
            if kind == "fp4":
                for scales in ([c.bits[2]] if what == "k" else [c.bits[3]] if what == "v" else c.bits[2:]):
                    scales[page, off] = 255
                return
            bad = torch.full((), float("nan") if kind == "fp8" or off % 2 else float("inf")).to(c.k.dtype)
            if what != "v":
                c.k[page, off] = bad
            if what != "k":
                c.v[page, off] = bad

        for s in range(S):
            lowest = lens[s] - int(c.drafts[s]) - window + 1
            for t in list(range(lens[s], n * B)) + list(range(sinks, lowest)):
                spoil(int(c.tables[s, t // B]), t % B)
            c.q[s, int(c.drafts[s]):] = float("nan")
        c.run(p, window, sinks)
        rk.pred_device_error(p.handle)
        assert torch.equal(c.out, clean[0]) and torch.equal(c.lse, clean[1])
        # blocks of which nobody sees a token
        tables = c.tables.clone()
        for s in range(S):
            lowest = lens[s] - int(c.drafts[s]) - window + 1
            for b in range(-(-sinks // B), lowest // B):
                c.tables[s, b] = (-1, c.N, 2 ** 31 - 1)[b % 3]
        c.run(p, window, sinks)
        rk.pred_device_error(p.handle)
        assert torch.equal(c.out, clean[0]) and torch.equal(c.lse, clean[1])
        c.tables = tables
        # one token that some rows see: its value, then its key
        s = 0
        t = lens[0] - max(1, M // 2)
        page = int(c.tables[s, t // B])
        first = lens[0] - int(c.drafts[0])
        sees = [t <= first + i < t + window for i in range(M)]
        keep = [x.clone() for x in (c.bits if kind == "fp4" else (c.k, c.v))]
        for what in ("v", "k"):
            spoil(page, t % B, what)
            c.run(p, window, sinks)
            for i in range(M):
                if not sees[i]:
                    assert torch.equal(c.out[s, i], clean[0][s, i]) and torch.equal(c.lse[s, i], clean[1][s, i]), (what, i)
                elif what == "v":
                    assert not torch.isfinite(c.out[s, i]).any() and torch.equal(c.lse[s, i], clean[1][s, i])
            assert torch.equal(c.out[1:], clean[0][1:])
            for x, y in zip(c.bits if kind == "fp4" else (c.k, c.v), keep):
                x.copy_(y)


@pytest.mark.parametrize("M", [1, 3, 40])
def test_infinite_values_that_a_row_sees(M):
    """An infinity is a row's result whatever its weight, NaN and both signs are NaN; in the sinks, at either end of the
    window and inside, over runs and in the pairs of waves."""
    Hq, Hk, D, B, n, window, sinks = 8, 2, 128, 16, 80, 300, 4
    c = make("bf16", 1, M, Hq, Hk, D, B, n, lens=[n * B - 3], drafts=[M], q_scale=30.0)
    length = n * B - 3
    with _handle(Hq, Hk, D, B, c.N) as p:
        for at in (0, 3, length - M - window + 1, length - M - window + 2, length - 200, length - M, length - 1):
            page, off = int(c.tables[0, at // B]), at % B
            old = c.v[page, off].clone()
            c.v[page, off, :, 5] = float("inf")
            c.v[page, off, :, 6] = -float("inf")
            c.v[page, off, :, 7] = float("nan")
            c.run(p, window, sinks)
            for i in range(M):
                pos = length - M + i
                if at <= pos and (at > pos - window or at < sinks):
                    assert torch.all(c.out[0, i, :, 5] == float("inf")) and torch.all(c.out[0, i, :, 6] == -float("inf")), (at, i)
                    assert torch.isnan(c.out[0, i, :, 7]).all() and torch.isfinite(c.out[0, i, :, 8:]).all()
                else:
                    assert torch.isfinite(c.out[0, i]).all(), (at, i)
            c.v[page, off] = old


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_bad_entries_and_lengths(Hq, Hk, D, B, M):
    """An invalid entry of a block that is seen is left out and raises the error word; lengths are clamped."""
    n, window, sinks = max(12, -(-M // B) + 3), 60, 4
    c = make("bf16", 2, M, Hq, Hk, D, B, n, ragged=False)
    with _handle(Hq, Hk, D, B, c.N) as p:
        for at in (0, n - 2):
            tables = c.tables.clone()
            c.tables[:, at] = -1
            c.run(p, window, sinks)
            with pytest.raises(rk.PredError) as e:
                rk.pred_device_error(p.handle)
            assert "block-table" in str(e.value) and torch.isfinite(c.out).all()
            c.tables = tables
        for lens, rows in (([n * B + 1, 5], [1, 1]), ([-3, 5], [0, 1]), ([5, 5], [1, -1]), ([5, 5], [1, M + 1]), ([0, 5], [1, 1])):
            c.lens, c.drafts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, rows))
            c.run(p, window, sinks)
            with pytest.raises(rk.PredError):
                rk.pred_device_error(p.handle)
            c.lens = c.lens.clamp(0, n * B)
            c.drafts = torch.minimum(c.drafts.clamp(0, M), c.lens)
            c.check(p, window, sinks)


@pytest.mark.parametrize("Hq,Hk,D,B,M,kind,window", [(8, 2, 128, 16, 1, "bf16", 9000), (8, 2, 128, 16, 1, "fp4", ALL),
                                                      (8, 2, 128, 16, 30, "bf16", ALL), (8, 2, 64, 16, 30, "fp4", 7000),
                                                      (4, 4, 128, 32, 200, "fp8", 9000)])
def test_long_contexts_in_runs(Hq, Hk, D, B, M, kind, window):
    """Walks that are split over workgroups and joined, of sequences of uneven length."""
    lens = [12000, 11999, 257, 5]
    c = make(kind, 4, M, Hq, Hk, D, B, -(-12000 // B), lens=lens, drafts=[M, 1, min(M, 257), min(M, 5)])
    with _handle(Hq, Hk, D, B, c.N) as p:
        assert rk.pred_attend_window_workspace_bytes(p.handle, 4, M, c.n, window, 4) > 0
        c.run(p, window, 4)
        rk.pred_device_error(p.handle)
        c.check(p, window, 4)
        first = c.out.clone()
        c.run(p, window, 4)
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("S,M,Hq,Hk,D,B,n,kind,window,sinks", [
    (150, 1, 8, 2, 128, 16, 12, "bf16", 60, 4), (65, 3, 8, 2, 64, 16, 9, "fp8", 50, 0), (130, 20, 4, 2, 64, 16, 12, "fp4", 33, 5),
    (300, 1, 4, 1, 128, 16, 60, "fp4", 700, 4), (129, 40, 2, 1, 128, 32, 12, "bf16", ALL, 0)])
def test_many_sequences(S, M, Hq, Hk, D, B, n, kind, window, sinks):
    """More sequences than a wave has lanes."""
    _say("window many", S, M, Hq, Hk, D, B, n, kind, window, sinks)
    c = make(kind, S, M, Hq, Hk, D, B, n)
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p, window, sinks)
        rk.pred_device_error(p.handle)
        c.check(p, window, sinks)


@pytest.mark.parametrize("kind,N", [("bf16", 80000), ("fp4", 300000)])
@pytest.mark.parametrize("M", [1, 40])
def test_far_pages(kind, N, M):
    """A sequence scattered over more than 4 GiB of keys: the bits of the same pages close together, with the window and
    without; tokens stored and read back there."""
    Hq, Hk, D, B, n = 16, 8, 128, 32, 250
    c = make(kind, 1, M, Hq, Hk, D, B, n)
    near = c.tables[0].long()
    far = torch.linspace(600, N - 1, n).long().cuda()
    slots = (near[-3:, None] * B + torch.arange(B, device="cuda")).flatten()
    x, y = (torch.randn((3 * B, Hk, D), generator=c.g).bfloat16().cuda() for _ in range(2))

    def run(slots):
        with _handle(Hq, Hk, D, B, c.N) as p:
            got = []
            for window in (3000, ALL):
                c.run(p, window, 4)
                got += [c.out.clone(), c.lse.clone()]
            Case.run(c, p, False)
            got += [c.out.clone(), c.lse.clone()]
            back = [torch.zeros_like(x) for _ in range(4)]
            rk.pred_load(p.handle, c.kv, slots, *back[:2])
            rk.pred_store(p.handle, x, y, slots, c.kv)
            rk.pred_load(p.handle, c.kv, slots, *back[2:])
            rk.pred_device_error(p.handle)
            return got + back

    small = c.bits if kind == "fp4" else (c.k, c.v)
    big = [torch.zeros((N, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in small]
    for t, b in zip(small, big):
        b[far] = t[near]
    want = run(slots)
    c.N, c.tables = N, far.int().view(1, n)
    c.kv = rk.KVCache(*big[:2], 1.0, 1.0, *big[2:])
    for a, b in zip(run((far[-3:, None] * B + torch.arange(B, device="cuda")).flatten()), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,kind", [(1, "bf16"), (1, "fp4"), (40, "bf16"), (300, "fp4")])
def test_nobody_has_anything(M, kind):
    """Lengths of zero, no row of any sequence, a table of no blocks: zeros and -inf everywhere, no error."""
    S, Hq, Hk, D, B, n = 70, 8, 2, 128, 16, 3
    c = make(kind, S, M, Hq, Hk, D, B, n, lens=[0] * S, drafts=[0] * S)
    with _handle(Hq, Hk, D, B, c.N) as p:
        for lens in (c.lens, torch.full_like(c.lens, 20)):
            c.lens = lens
            c.run(p, 30, 4)
            assert torch.all(c.out == 0) and torch.all(torch.isneginf(c.lse))
        c.out.fill_(9.0)
        c.lse.fill_(9.0)
        c.lens.zero_()
        rk.pred_attend_window(p.handle, c.kv, c.q, c.tables[:, :0].contiguous(), c.lens, None, 30, 4, c.scale, c.out, c.lse, None)
        rk.pred_device_error(p.handle)
        assert torch.all(c.out == 0) and torch.all(torch.isneginf(c.lse))


def test_no_table_no_lengths():
    for M in (1, 70):
        c = make("bf16", 2, M, 8, 2, 128, 16, 9, identity=True, ragged=False, drafts=[M, M])
        with _handle(8, 2, 128, 16, 9) as p:
            ws = torch.empty((max(1, rk.pred_attend_window_workspace_bytes(p.handle, 2, M, 9, 50, 2)),), dtype=torch.uint8, device="cuda")
            rk.pred_attend_window(p.handle, c.kv, c.q, None, None, None, 50, 2, c.scale, c.out, c.lse, ws)
            c.check(p, 50, 2)


def test_chunks_of_a_prompt_are_the_prompt():
    """A prompt in one call and in chunks, its last token also as a decode step: each row within the roundings."""
    Hq, Hk, D, B, n, window, sinks, P = 8, 2, 128, 16, 30, 100, 4, 470
    c = make("bf16", 1, P, Hq, Hk, D, B, n, lens=[P], drafts=[P])
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p, window, sinks)
        c.check(p, window, sinks)
        whole = c.out[0].float()
        for chunk in (1, 37, 128):
            for at in ([P - 1] if chunk == 1 else range(0, P, chunk)):
                rows = min(chunk, P - at)
                q = c.q[:, at:at + rows].contiguous()
                out = torch.empty_like(q)
                lens = torch.tensor([at + rows], dtype=torch.int32, device="cuda")
                ws = torch.empty((max(1, rk.pred_attend_window_workspace_bytes(p.handle, 1, rows, n, window, sinks)),), dtype=torch.uint8,
                                 device="cuda")
                rk.pred_attend_window(p.handle, c.kv, q, c.tables, lens, None, window, sinks, c.scale, out, None, ws)
                # |v| < 5: two roundings of the output, and of the weights
                assert torch.all((out[0].float() - whole[at:at + rows]).abs() <= 2 * HALF_BF16 * whole[at:at + rows].abs() + HALF_BF16 * 2)


def test_steps_in_a_graph_and_on_another_stream():
    """A decode step and a chunk captured with workspaces of their own, replayed with eager work between."""
    Hq, Hk, D, B, n, window, sinks = 8, 2, 128, 16, 300, 3000, 4
    one, many = (make("bf16", 2, M, Hq, Hk, D, B, n, lens=[n * B, n * B - 77], drafts=[M, M], seed=M) for M in (1, 40))
    with _handle(Hq, Hk, D, B, max(one.N, many.N)) as p:
        ws = [[torch.empty((rk.pred_attend_window_workspace_bytes(p.handle, 2, c.M, n, window, sinks),), dtype=torch.uint8, device="cuda")
               for c in (one, many)] for _ in range(2)]

        def step(which):
            for c, w in zip((one, many), ws[which]):
                rk.pred_attend_window(p.handle, c.kv, c.q, c.tables, c.lens, c.drafts, window, sinks, c.scale, c.out, c.lse, w)

        step(0)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(0)
        s = torch.cuda.Stream()
        for i in range(4):
            for c in (one, many):
                c.q.copy_(torch.randn(c.q.shape, generator=c.g))
                c.lens -= 31
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                step(1)
            s.synchronize()
            want = [t.clone() for c in (one, many) for t in (c.out, c.lse)]
            for c in (one, many):
                c.out.zero_()
                c.lse.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip([t for c in (one, many) for t in (c.out, c.lse)], want):
                assert torch.equal(a, b), i


def test_more_rows_than_a_launch_has_threads():
    """2^24 rows of heads for the kernel that gives each a workgroup of 256: refused, and nothing written."""
    Hq, D, B, M = 64, 32, 16, 1 << 18
    q = torch.zeros((1, M, Hq, D), dtype=BF16, device="cuda")
    out = torch.full_like(q, 9.0)
    k, v = (torch.zeros((1, B, 1, D), dtype=BF16, device="cuda") for _ in range(2))
    lens, tab = torch.ones((1,), dtype=torch.int32, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    with _handle(Hq, 1, D, B, 1) as p:
        with pytest.raises(rk.PredError):
            rk.pred_attend_window(p.handle, rk.KVCache(k, v), q, tab, lens, None, 5, 0, 1.0, out)
        assert torch.all(out == 9.0)
        rows = M - 1
        rk.pred_attend_window(p.handle, rk.KVCache(k, v), q[:, :rows], tab, lens, None, 5, 0, 1.0, out[:, :rows])
        rk.pred_device_error(p.handle)
        assert torch.all(out[:, :rows] == 0) and torch.all(out[:, rows:] == 9.0)


def test_two_calls_at_once():
    """Two batches of one handle on two streams, each with its workspace, many times over: the bits of one after another."""
    Hq, Hk, D, B, n = 8, 2, 128, 16, 300
    cases = [make(kind, 2, M, Hq, Hk, D, B, n, lens=[n * B, n * B - 9], drafts=[M, M], seed=M)
             for M, kind in ((1, "bf16"), (40, "fp4"), (1, "fp4"), (33, "bf16"))]
    with _handle(Hq, Hk, D, B, cases[0].N) as p:
        want = []
        for c in cases:
            c.run(p, 3000, 4)
            want.append((c.out.clone(), c.lse.clone()))
            c.ws = torch.empty((rk.pred_attend_window_workspace_bytes(p.handle, 2, c.M, n, 3000, 4),), dtype=torch.uint8, device="cuda")
            c.out.zero_()
            c.lse.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in cases]
        for _ in range(10):
            for c, s in zip(cases, streams):
                rk.pred_attend_window(p.handle, c.kv, c.q, c.tables, c.lens, c.drafts, 3000, 4, c.scale, c.out, c.lse, c.ws, stream=s)
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cases, want):
            assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_refusals():
    D, B, Hk, N = 64, 16, 2, 8
    z = dict(device="cuda")
    with _handle(4, Hk, D, B, N) as p:
        h = p.handle
        k, v = (torch.zeros((N, B, Hk, D), dtype=BF16, **z) for _ in range(2))
        kv = rk.KVCache(k, v)
        q = torch.zeros((1, 3, 4, D), dtype=BF16, **z)
        out, lens = torch.zeros_like(q), torch.full((1,), 5, dtype=torch.int32, **z)
        tab = torch.zeros((1, N), dtype=torch.int32, **z)
        ws = torch.empty((rk.pred_attend_window_workspace_bytes(h, 1, 3, N, 100, 4) + 16,), dtype=torch.uint8, **z)

        def attend(**kw):
            a = dict(cache=kv, q=q, block_tables=tab, kv_len=lens, row_len=None, window=100, n_sinks=4, scale=1.0, out=out, workspace=ws)
            a.update(kw)
            rk.pred_attend_window(h, **a)

        attend()
        for kw, err in ((dict(q=q[0]), TypeError), (dict(q=q.float()), TypeError), (dict(out=out[..., :32]), ValueError),
                        (dict(out=out.cpu()), ValueError), (dict(kv_len=lens.long()), TypeError), (dict(block_tables=tab[0]), ValueError),
                        (dict(row_len=lens.expand(2).contiguous()), ValueError), (dict(window=0), rk.PredError), (dict(window=-5), rk.PredError),
                        (dict(n_sinks=-1), rk.PredError), (dict(scale=math.inf), rk.PredError), (dict(out=q), rk.PredError),
                        (dict(block_tables=None, n_blocks=N + 1), rk.PredError), (dict(workspace=None), rk.PredError),
                        (dict(workspace=ws[1:]), rk.PredError),
                        (dict(q=torch.zeros((1, 0, 4, D), dtype=BF16, **z), out=torch.zeros((1, 0, 4, D), dtype=BF16, **z)), rk.PredError)):
            with pytest.raises(err):
                attend(**kw)
        assert rk.pred_attend_window_workspace_bytes(h, 1, 3, N, 0, 4) == 0
        assert rk.pred_attend_window_workspace_bytes(h, 1, 2 ** 24 + 1, N, 9, 4) == 0
        with pytest.raises(rk.PredError):
            rk.pred_attend_window_kernel_name(h, kv, 0)
        attend(q=torch.zeros((0, 3, 4, D), dtype=BF16, **z), out=torch.zeros((0, 3, 4, D), dtype=BF16, **z),
               block_tables=torch.zeros((0, N), dtype=torch.int32, **z), kv_len=lens[:0], workspace=None)       # no sequence
        rk.pred_device_error(h)
    with _handle(2, 1, 264, 16, 2) as p:
        k = torch.zeros((2, 16, 1, 264), dtype=BF16, **z)
        q = torch.zeros((1, 1, 2, 264), dtype=BF16, **z)
        with pytest.raises(rk.PredError) as e:
            rk.pred_attend_window(p.handle, rk.KVCache(k, k), q, None, None, None, 5, 0, 1.0, torch.empty_like(q))
        assert e.value.code == rk.PRED_ERR_UNSUPPORTED
