"""GPU tests of the paged KV cache operators against the float64 oracle (oracle/cache.py).

Tolerances, fixed before the first run:
* bf16 results: half a step, 2^-8 relative, plus the float32 arithmetic before the one rounding; e4m3 results: half a
  step, 2^-4 relative or 2^-10 in the subnormals, plus the same.
* float32 arithmetic of a rotation: two products and a sum of values rounded to 2^-24, and a cosine and sine whose
  angle is cut at 2^-31 half turns and rounded to 2^-24 relative (under pi 2^-24 of a turn): 2^-20 (|a| + |b|) mscale.
* a score is a float32 sum of D exact products: off by at most (D + 4) 2^-24 scale sum |q k|, delta below.  A softmax
  weight is then off by 2 delta relative, plus 2^-20 for exp2 and the scaled argument, plus 2^-16 where the weights
  enter the matrix cores as two bf16 terms and (T + 64) 2^-24 for a sum over T tokens; an output by that times the sum
  of weights times |v|, a log-sum-exp by the same absolutely plus 2^-22 of its own size.
"""

import math

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import bf16, cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FP8 = torch.float8_e4m3fn
E4M3 = cache.e4m3_values()
HALF_BF16 = 2.0 ** -8


def _say(*a):
    print("[case]", *a, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


def _f64(t):
    """A GPU tensor's values, float64 on the host."""
    if t.dtype == FP8:
        return E4M3[t.detach().cpu().contiguous().view(torch.uint8).numpy()]
    return t.detach().cpu().double().numpy()


def _handle(Hq, Hk, D, B, N):
    return rk.Predictor(rk.dims(1, Hq, Hk, D, 8, B, N), seed=1)


def _rope(rot, theta=10000.0, kind="none", args=(), interleaved=False, backward=False):
    turns, mscale = rk.pred_rope_turns(rot, theta, kind, *args)
    freq, m = cache.frequencies(rot, theta, kind, *args)
    return rk.Rope(torch.from_numpy(turns.view(np.int64)).cuda(), rot, interleaved, mscale, backward), freq, m


def _cache_tensors(N, B, Hk, D, dtype, layout, gen=None, fill=None):
    """k, v [N, B, Hk, D] views of memory in the given order."""
    def values(shape):
        x = torch.randn(shape, generator=gen) if fill is None else torch.full(shape, fill)
        return (x * (16 if dtype == FP8 else 1)).to(dtype).cuda()
    if layout == "tokens":
        return values((N, B, Hk, D)), values((N, B, Hk, D))
    if layout == "heads":
        return values((N, Hk, B, D)).transpose(1, 2), values((N, Hk, B, D)).transpose(1, 2)
    both = values((N, 2, B, Hk, D + 16))[..., :D]        # k and v of a block side by side, rows padded
    return both[:, 0], both[:, 1]


# ---------------------------------------------------------------- rotation

def _rotation_tolerance(x, want, rot, interleaved, mscale):
    pair = np.zeros_like(x)
    half = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    both = np.abs(a) + np.abs(b)
    if interleaved:
        pair[..., 0:rot:2], pair[..., 1:rot:2] = both, both
    else:
        pair[..., :half], pair[..., half:rot] = both, both
    return 2.0 ** -20 * abs(mscale) * pair


ROTATIONS = [
    # n, heads, D, rot, interleaved, kind, scaling arguments, first position
    (1, 4, 64, 64, False, "none", (), 0),
    (5, 3, 64, 32, True, "linear", (4.0,), 77),
    (67, 8, 128, 128, False, "llama3", (8.0, 1.0, 4.0, 8192.0), 131000),
    (33, 5, 128, 64, True, "yarn", (16.0, 1.0, 32.0, 4096.0), 999000),
    (9, 2, 80, 80, False, "ntk", (8.0,), 2 ** 31 - 10),
    (9, 1, 80, 20, False, "none", (), 31),      # pairs that do not fill a piece
    (4, 7, 96, 6, True, "none", (), 5),
    (3, 33, 8, 2, False, "none", (), 5),
    (2, 3, 512, 512, True, "none", (), 4000),
    (2, 3, 512, 256, False, "none", (), 4000),
    (300, 40, 128, 128, True, "none", (), -150),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("n,heads,D,rot,inter,kind,args,first", ROTATIONS)
def test_rotate(n, heads, D, rot, inter, kind, args, first, backward):
    _say("rotate", n, heads, D, rot, inter, kind, first, backward)
    g = torch.Generator().manual_seed(n * 1000 + D + rot)
    rope, freq, mscale = _rope(rot, 500000.0, kind, args, inter, backward)
    store = torch.randn((n, heads + 2, D), generator=g).bfloat16().cuda()
    x = store[:, 1:heads + 1]                       # tokens apart
    pos = torch.arange(first, first + n, dtype=torch.int64)
    positions = ((pos + 2 ** 31) % 2 ** 32 - 2 ** 31).to(torch.int32).cuda()    # int32, wrapping at its end
    with _handle(8, 2, D, 16, 4) as p:
        out = torch.full((n, heads + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
        rk.pred_rotate(p.handle, rope, x, positions, out[:, :heads])
        want = cache.rotate(_f64(x), positions.cpu().numpy(), freq, mscale, inter, backward)
        tol = HALF_BF16 * np.abs(want) + _rotation_tolerance(_f64(x), want, rot, inter, mscale)
        err = np.abs(_f64(out[:, :heads]) - want)
        assert np.all(err <= tol), (err - tol).max()
        assert np.array_equal(_f64(out[..., rot:])[:, :heads], _f64(x[..., rot:]))      # passed values are copies
        assert torch.all(out[:, heads:] == 7)                                       # the row's rest stays
        keep = store.clone()
        rk.pred_rotate(p.handle, rope, x, positions, x)                             # in place
        assert torch.equal(x, out[:, :heads])
        assert torch.equal(store[:, 0], keep[:, 0]) and torch.equal(store[:, -1], keep[:, -1])


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_gradient_is_the_difference(inter):
    """The map is linear: <out(x + e) - out(x), u> for unit steps e is the gradient for u.  Powers of two for x, e and
    u make every difference one of two bf16 roundings of values under 8: off by 2 * 2^-8 * 8 at most."""
    rope, _, _ = _rope(16, 100.0, interleaved=inter)
    back, _, _ = _rope(16, 100.0, interleaved=inter, backward=True)
    D = 16
    pos = torch.tensor([3], dtype=torch.int32, device="cuda")
    with _handle(2, 1, D, 16, 4) as p:
        u = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
        for at in range(D):
            u.zero_()
            u[0, 0, at] = 1
            grad = torch.empty_like(u)
            rk.pred_rotate(p.handle, back, u, pos, grad)
            x = torch.full((D, 1, D), 0.5, dtype=torch.bfloat16, device="cuda")
            y = x.clone()
            y[torch.arange(D), 0, torch.arange(D)] += 4
            many = pos.expand(D).contiguous()
            outs = [torch.empty_like(x), torch.empty_like(x)]
            for t, o in zip((x, y), outs):
                rk.pred_rotate(p.handle, rope, t, many, o)
            diff = (_f64(outs[1]) - _f64(outs[0]))[:, 0, at] / 4
            assert np.all(np.abs(diff - _f64(grad)[0, 0]) <= 2 * HALF_BF16 * 8 / 4 + HALF_BF16)


STORES = [
    # n, Hq, Hk, D, B, rot, interleaved, dtype, layout, fused
    (1, 4, 1, 64, 16, 64, False, torch.bfloat16, "tokens", True),
    (37, 8, 2, 64, 16, 32, True, torch.bfloat16, "heads", False),
    (37, 8, 2, 128, 16, 128, False, FP8, "tokens", True),
    (130, 32, 8, 128, 32, 64, True, FP8, "heads", True),
    (20, 5, 1, 80, 7, 20, False, torch.bfloat16, "padded", False),
    (20, 10, 2, 96, 1, 96, True, FP8, "padded", False),
    (65, 64, 8, 128, 8, 128, False, torch.bfloat16, "padded", True),
]


@pytest.mark.parametrize("n,Hq,Hk,D,B,rot,inter,dtype,layout,fused", STORES)
def test_rotate_store(n, Hq, Hk, D, B, rot, inter, dtype, layout, fused):
    _say("store", n, Hq, Hk, D, B, rot, inter, dtype, layout, fused)
    g = torch.Generator().manual_seed(n + D)
    N = n // B + 4
    rope, freq, _ = _rope(rot, 10000.0, interleaved=inter)
    k_cache, v_cache = _cache_tensors(N, B, Hk, D, dtype, layout, fill=3.0)
    scales = (0.0625, 0.37) if dtype == FP8 else (1.0, 1.0)
    qkv = torch.randn((n, Hq + 2 * Hk, D), generator=g)
    qkv[n // 2, Hq] = 1000.0 * torch.sign(qkv[n // 2, Hq])      # beyond e4m3's range
    qkv = qkv.bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = torch.randperm(N * B, generator=g)[:n]
    if n > 4:
        slots[1] = -1
    positions = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32).cuda()
    with _handle(Hq, Hk, D, B, N) as p:
        kv = rk.KVCache(k_cache, v_cache, *scales)
        q_out = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
        before = [_f64(k_cache), _f64(v_cache)]
        rk.pred_rotate_store(p.handle, rope, q, k, v, positions, slots.cuda(), kv, q_out)
        rk.pred_device_error(p.handle)
        alone = torch.empty_like(q_out)
        rk.pred_rotate(p.handle, rope, q, positions, alone)
        assert torch.equal(alone, q_out)
        pos = positions.cpu().numpy()
        turned = cache.rotate(_f64(k), pos, freq, 1.0, inter)
        slack = _rotation_tolerance(_f64(k), turned, rot, inter, 1.0)
        for got, old, want, extra, scale in ((_f64(k_cache), before[0], turned, slack, scales[0]),
                                             (_f64(v_cache), before[1], _f64(v), 0 * slack, scales[1])):
            got, old = got.reshape(N * B, Hk, D), old.reshape(N * B, Hk, D)
            want, extra = want / scale, extra / scale
            if dtype == FP8:
                want = np.clip(want, -448, 448)
                tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + extra + 2.0 ** -22 * np.abs(want)
            else:
                tol = HALF_BF16 * np.abs(want) + extra
            hit = np.zeros(N * B, bool)
            for t, slot in enumerate(slots.tolist()):
                if slot >= 0:
                    hit[slot] = True
                    assert np.all(np.abs(got[slot] - want[t]) <= tol[t]), (t, slot)
            assert np.array_equal(got[~hit], old[~hit])
        # in place, and a second call over other slots of the same tokens
        if not fused:
            rk.pred_rotate_store(p.handle, rope, q, k, v, positions, slots.cuda(), kv, q)
            assert torch.equal(q, q_out)


def test_store_rounds_every_e4m3_step():
    """Values a quarter and three quarters of the way between neighbours, ties, and what is beyond the range, through
    the value path (no rotation): nearest, ties to even, clamped; NaN stays NaN."""
    D, B = 64, 16
    grid = np.sort(np.unique(E4M3[np.isfinite(E4M3)]))
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, mid, [464.0, -464.0, 2.0 ** 100, -2.0 ** 100, np.inf, -np.inf, np.nan]])
    # a step between e4m3 neighbours is 16 bf16 steps or more, so every midpoint is a bf16 value
    x = np.concatenate([x, np.zeros(-len(x) % D)]).reshape(-1, 1, D)
    n = len(x)
    with _handle(1, 1, D, B, n // B + 1) as p:
        k_cache, v_cache = _cache_tensors(n // B + 1, B, 1, D, FP8, "tokens", fill=0.0)
        kv = rk.KVCache(k_cache, v_cache, 1.0, 1.0)
        v = torch.from_numpy(x).bfloat16().cuda()
        assert np.array_equal(_f64(v), x, equal_nan=True)
        rope, _, _ = _rope(64)
        zeros = torch.zeros((n,), dtype=torch.int32, device="cuda")
        q_out = torch.empty_like(v)
        rk.pred_rotate_store(p.handle, rope, v, v, v, zeros, torch.arange(n).cuda(), kv, q_out)
        got = _f64(v_cache).reshape(-1, 1, D)[:n]
        for a, b in zip(x.ravel(), got.ravel()):
            if np.isnan(a):
                assert np.isnan(b)
                continue
            a = min(max(a, -448.0), 448.0)
            at = np.searchsorted(grid, a)
            if grid[at] == a:
                assert b == a
            else:       # a midpoint: the neighbour whose pattern is even
                pair = [y for y in (grid[at - 1], grid[at]) if any(E4M3[i] == y for i in range(0, 256, 2))]
                assert b in pair, (a, b)


def test_store_leaves_bad_slots_out():
    Hk, D, B, N, n = 2, 64, 16, 4, 6
    rope, _, _ = _rope(64)
    with _handle(4, Hk, D, B, N) as p:
        k_cache, v_cache = _cache_tensors(N, B, Hk, D, torch.bfloat16, "tokens", fill=3.0)
        kv = rk.KVCache(k_cache, v_cache)
        x = torch.randn((n, 4, D), device="cuda").bfloat16()
        slots = torch.tensor([N * B, -2, 5, 2 ** 40, -1, -2 ** 40], device="cuda")
        pos = torch.zeros((n,), dtype=torch.int32, device="cuda")
        out = torch.empty_like(x)
        rk.pred_rotate_store(p.handle, rope, x, x[:, :Hk].contiguous(), x[:, :Hk].contiguous(), pos, slots, kv, out)
        with pytest.raises(rk.PredError) as e:
            rk.pred_device_error(p.handle)
        assert e.value.code == rk.PRED_ERR_DEVICE and "slot" in str(e.value)
        assert torch.equal(out, x)      # position 0 turns nothing
        flat = v_cache.view(N * B, Hk, D)
        assert torch.equal(flat[5], x[2, :Hk])
        flat[5] = 3.0
        assert torch.all(flat == 3.0)
        slots.fill_(-1)
        rk.pred_rotate_store(p.handle, rope, x, x[:, :Hk].contiguous(), x[:, :Hk].contiguous(), pos, slots, kv, out)
        rk.pred_device_error(p.handle)      # padding is no error
        assert torch.all(flat == 3.0)


# ---------------------------------------------------------------- attention

class Case:
    """A batch over a cache: inputs on the GPU, the oracle's values on the host."""

    def __init__(self, S, M, Hq, Hk, D, B, n, dtype=torch.bfloat16, layout="tokens", tree="chain", ragged=True,
                 lens=None, drafts=None, seed=0, identity=False, q_scale=2.0):
        g = self.g = torch.Generator().manual_seed(seed + S * 7 + M * 131 + D + n)
        self.S, self.M, self.Hq, self.Hk, self.D, self.B, self.n = S, M, Hq, Hk, D, B, n
        self.N = n if identity else S * n + 3
        self.k, self.v = _cache_tensors(self.N, B, Hk, D, dtype, layout, g)
        self.scales = (0.0625, 0.11) if dtype == FP8 else (1.0, 1.0)
        self.kv = rk.KVCache(self.k, self.v, *self.scales)
        self.tables = None if identity else torch.randperm(self.N, generator=g)[:S * n].view(S, n).int().cuda()
        most = n * B
        if lens is None:
            lens = torch.randint(min(M, most), most + 1, (S,), generator=g) if ragged else torch.full((S,), most)
            lens[0] = most
        self.lens = torch.as_tensor(lens).int().cuda()
        if drafts is None:
            drafts = torch.randint(1, M + 1, (S,), generator=g)
            drafts[0] = M
            drafts = torch.minimum(drafts, self.lens.cpu().long())
        self.drafts = torch.as_tensor(drafts).int().cuda()
        self.tree = None
        if tree != "chain":
            words = torch.zeros((S, M), dtype=torch.int64)
            for s in range(S):
                for j in range(M):
                    bit = 1 << j if j < 63 else -(1 << 63)
                    parent = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
                    words[s, j] = (int(words[s, parent]) if parent >= 0 else 0) | bit
            if tree == "bits":      # any bits, rows that see no drafted token among them
                words = torch.randint(-2 ** 63, 2 ** 63 - 1, (S, M), generator=g)
                words[:, M // 2] = 0
            self.tree = words.cuda()
        self.q = (q_scale * torch.randn((S, M, Hq, D), generator=g)).bfloat16().cuda()
        self.scale = 1 / math.sqrt(D)
        self.out = torch.full_like(self.q, 9.0)
        self.lse = torch.full((S, M, Hq), 9.0, device="cuda")
        self.block_lse = torch.full((S, n, M, Hq), 9.0, device="cuda")

    def run(self, p, weights=True):
        need = rk.pred_attend_workspace_bytes(p.handle, self.S, self.M, self.n)
        ws = torch.empty((max(need, 1),), dtype=torch.uint8, device="cuda")
        for t in (self.out, self.lse, self.block_lse):
            t.fill_(9.0)
        rk.pred_attend(p.handle, self.kv, self.q, self.tree, self.tables, self.lens, self.drafts, self.scale, self.out,
                       self.lse, self.block_lse if weights else None, ws, n_blocks=self.n)
        return ws

    def check(self, weights=True, seqs=None):
        q, k, v = _f64(self.q), _f64(self.k) * self.scales[0], _f64(self.v) * self.scales[1]
        out, lse, blk = _f64(self.out), _f64(self.lse), _f64(self.block_lse)
        g = self.Hq // self.Hk
        for s in range(self.S) if seqs is None else seqs:
            length, drafted = int(self.lens[s]), int(self.drafts[s])
            used = -(-length // self.B)
            pages = np.arange(used) if self.tables is None else self.tables[s, :used].cpu().numpy()
            words = None if self.tree is None else self.tree[s].tolist()
            seen = np.repeat(cache.seen_by(self.M, length, drafted, words), g, axis=0)
            for h in range(self.Hk):
                kk = k[pages, :, h].reshape(-1, self.D)[:length]
                vv = v[pages, :, h].reshape(-1, self.D)[:length]
                qq = q[s, :, h * g:h * g + g].reshape(-1, self.D)
                want, want_lse, x, absolute = cache.attend_one(qq, kk, vv, seen, self.scale)
                delta = 0.0
                if length:
                    delta = (self.D + 4) * 2.0 ** -24 * self.scale * (np.abs(qq) @ np.abs(kk).T).max()
                rel = 2 * delta + 2.0 ** -20 + 2.0 ** -16 + (length + 64) * 2.0 ** -24
                got = out[s, :, h * g:h * g + g].reshape(-1, self.D)
                tol = HALF_BF16 * np.abs(want) + rel * absolute
                bad = np.abs(got - want) > tol
                assert not bad.any(), ("out", s, h, np.argwhere(bad)[:4], (np.abs(got - want) - tol).max())
                got = lse[s, :, h * g:h * g + g].reshape(-1)
                self._close_log(got, want_lse, rel, ("lse", s, h))
                if weights:
                    got = blk[s, :used, :, h * g:h * g + g].reshape(used, self.M * g)
                    self._close_log(got, cache.block_lse_one(x, self.B), rel, ("block_lse", s, h))
            if weights:
                assert np.all(blk[s, used:] == 9.0), ("blocks past the sequence", s)

    @staticmethod
    def _close_log(got, want, rel, what):
        none = np.isneginf(want)
        assert np.array_equal(none, np.isneginf(got)), what
        err = np.abs(got[~none] - want[~none])
        assert np.all(err <= rel + 2.0 ** -22 * np.abs(want[~none])), (what, err.max())


ATTEND = [
    # S, M, Hq, Hk, D, B, n, dtype, layout, tree
    (1, 1, 4, 1, 64, 16, 5, torch.bfloat16, "tokens", "chain"),
    (3, 1, 32, 8, 128, 16, 20, torch.bfloat16, "tokens", "chain"),
    (3, 1, 32, 8, 128, 16, 20, FP8, "tokens", "chain"),
    (2, 1, 16, 2, 128, 32, 40, torch.bfloat16, "heads", "chain"),
    (2, 1, 8, 2, 64, 8, 33, torch.bfloat16, "padded", "chain"),
    (2, 1, 8, 2, 64, 16, 33, FP8, "heads", "chain"),
    (2, 1, 8, 8, 128, 64, 9, FP8, "padded", "chain"),
    (1, 1, 40, 8, 128, 16, 130, torch.bfloat16, "tokens", "chain"),
    (4, 3, 20, 4, 128, 16, 12, torch.bfloat16, "tokens", "tree"),
    (4, 4, 16, 2, 128, 16, 12, FP8, "heads", "bits"),
    (2, 7, 8, 2, 64, 32, 12, torch.bfloat16, "heads", "bits"),
    (3, 13, 16, 2, 128, 32, 9, torch.bfloat16, "tokens", "tree"),
    (2, 64, 8, 1, 128, 16, 21, torch.bfloat16, "tokens", "tree"),
    (2, 64, 8, 2, 64, 16, 21, FP8, "tokens", "bits"),
    (2, 33, 12, 4, 128, 8, 21, FP8, "padded", "chain"),
    (2, 17, 10, 2, 64, 64, 5, torch.bfloat16, "padded", "bits"),
    (1, 64, 2, 2, 128, 16, 6, torch.bfloat16, "tokens", "chain"),
    (2, 1, 6, 2, 80, 16, 9, torch.bfloat16, "tokens", "chain"),      # plain kernel: head size
    (2, 5, 4, 1, 256, 16, 9, FP8, "heads", "tree"),
    (2, 3, 4, 2, 128, 24, 9, torch.bfloat16, "tokens", "tree"),      # blocks that end inside a tile
    (2, 2, 4, 2, 128, 7, 19, torch.bfloat16, "padded", "bits"),
    (2, 2, 4, 2, 64, 1, 70, FP8, "tokens", "chain"),
    (2, 20, 4, 2, 64, 40, 7, torch.bfloat16, "tokens", "bits"),
    (1, 2, 4, 2, 128, 512, 2, torch.bfloat16, "tokens", "tree"),
    (1, 40, 4, 1, 64, 96, 5, FP8, "tokens", "tree"),
]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("S,M,Hq,Hk,D,B,n,dtype,layout,tree", ATTEND)
def test_attend(S, M, Hq, Hk, D, B, n, dtype, layout, tree, weights):
    _say("attend", S, M, Hq, Hk, D, B, n, dtype, layout, tree, weights)
    c = Case(S, M, Hq, Hk, D, B, n, dtype, layout, tree)
    with _handle(Hq, Hk, D, B, c.N) as p:
        _say(rk.pred_attend_kernel_name(p.handle, c.kv, M, weights))
        c.run(p, weights)
        rk.pred_device_error(p.handle)
        c.check(weights)
        assert weights or torch.all(c.block_lse == 9.0)


@pytest.mark.parametrize("seed", range(24))
def test_attend_random_shapes(seed):
    r = np.random.default_rng(100 + seed)
    Hk, g = int(r.integers(1, 9)), int(r.integers(1, 9))
    D = int(r.choice([64, 128, 128, 64, 8 * int(r.integers(1, 33))]))
    B = int(r.choice([8, 16, 32, 64, int(r.integers(1, 70))]))
    M = int(r.choice([1, int(r.integers(1, 65))]))
    S = int(r.integers(1, 5))
    n = max(1, min(int(r.integers(1, 3000 // B + 2)), 2 ** 20 // (S * B * Hk * D) + 1))
    n = max(n, -(-M // B))
    dtype = FP8 if r.integers(2) else torch.bfloat16
    layout, tree = str(r.choice(["tokens", "heads", "padded"])), str(r.choice(["chain", "tree", "bits"]))
    weights = bool(r.integers(2))
    _say("attend random", seed, S, M, Hk * g, Hk, D, B, n, dtype, layout, tree, weights)
    c = Case(S, M, Hk * g, Hk, D, B, n, dtype, layout, tree, seed=seed)
    with _handle(Hk * g, Hk, D, B, c.N) as p:
        c.run(p, weights)
        rk.pred_device_error(p.handle)
        c.check(weights)


SHAPES = [(4, 1, 64, 16, 1), (32, 8, 128, 16, 1), (16, 2, 128, 16, 3), (16, 2, 128, 16, 40), (8, 2, 64, 32, 64),
          (6, 2, 80, 16, 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_attend_short_sequences(Hq, Hk, D, B, M, dtype):
    """Every length from none to a few tiles' edges, drafts of every size among them: lengths of 0 and 1, a sequence
    that is all draft, rows that see nothing."""
    lens = [0, 1, 1, 2, B - 1, B, B + 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130]
    lens = lens + lens
    drafts = [min(M, x) for x in lens[:17]] + [min(M, x, 1 + i % 3) if i % 4 else 0 for i, x in enumerate(lens[17:])]
    n = -(-130 // B)
    _say("attend short", Hq, Hk, D, B, M, dtype)
    c = Case(len(lens), M, Hq, Hk, D, B, n, dtype, tree="bits" if M > 1 else "chain", lens=lens, drafts=drafts)
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        rk.pred_device_error(p.handle)
        c.check()
        assert torch.all(c.out[0] == 0) and torch.all(torch.isneginf(c.lse[0]))


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_attend_defaults(Hq, Hk, D, B, M):
    """No table (the identity), no lengths (all blocks full), no draft lengths (all rows), no lse."""
    n = 6 if M <= 6 * B else -(-M // B)
    c = Case(2, M, Hq, Hk, D, B, n, identity=True, ragged=False, drafts=[M, M])
    with _handle(Hq, Hk, D, B, n) as p:
        ws = torch.empty((rk.pred_attend_workspace_bytes(p.handle, 2, M, n),), dtype=torch.uint8, device="cuda")
        c.run(p, False)
        first = c.out.clone()
        c.out.fill_(9.0)
        rk.pred_attend(p.handle, c.kv, c.q, None, None, None, None, c.scale, c.out, workspace=ws)
        assert torch.equal(first, c.out)
        c.check(False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_attend_masked_places_do_not_matter(Hq, Hk, D, B, M, dtype):
    """NaN and infinities past a sequence's end, in slots of no sequence, in drafted tokens a row does not see and in
    the queries of rows past the draft: every row that does not see them keeps its bits; a row that sees a NaN value
    is NaN in that place."""
    n, S = max(5, -(-M // B) + 2), 3
    c = Case(S, M, Hq, Hk, D, B, n, dtype, tree="tree" if M > 1 else "chain",
             lens=[n * B - B // 2, n * B - 1, M + 2], drafts=[M, max(1, M // 2), M])
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        c.check()
        clean = [t.clone() for t in (c.out, c.lse, c.block_lse)]
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")]) if dtype == torch.bfloat16 else torch.full(
            (3,), float("nan"))
        for s in range(S):
            length = int(c.lens[s])
            for t in range(length, n * B):      # past the end
                page = int(c.tables[s, t // B])
                c.k[page, t % B] = bad[t % 3].to(dtype)
                c.v[page, t % B] = bad[(t + 1) % 3].to(dtype)
            c.q[s, int(c.drafts[s]):] = float("nan")
        used = set(c.tables.flatten().tolist())
        for page in set(range(c.N)) - used:
            c.k[page], c.v[page] = bad[0].to(dtype), bad[0].to(dtype)
        c.run(p)
        for got, want in zip((c.out, c.lse, c.block_lse), clean):
            assert torch.equal(got, want)
        if M == 1:
            return
        # a drafted token that only its own subtree sees
        s, j = 0, M // 2
        t = int(c.lens[s]) - int(c.drafts[s]) + j
        page = int(c.tables[s, t // B])
        sees = [bool(int(w) >> j & 1) for w in c.tree[s].tolist()]
        for place, value in ((c.v, "value"), (c.k, "key")):
            old = place[page, t % B].clone()
            place[page, t % B, :, 3] = float("nan")
            c.run(p)
            for i in range(M):
                if not sees[i]:
                    assert torch.equal(c.out[s, i], clean[0][s, i]), (value, i)
                    assert torch.equal(c.lse[s, i], clean[1][s, i]), (value, i)
                elif value == "value":
                    assert torch.isnan(c.out[s, i, :, 3]).all()
                    rest = [d for d in range(D) if d != 3]
                    # the rest of the row, by the sums of the other path: two bf16 roundings of one value
                    a, b = c.out[s, i][:, rest].double(), clean[0][s, i][:, rest].double()
                    assert torch.all((a - b).abs() <= 2 * HALF_BF16 * b.abs() + 2.0 ** -8 * 0.05), (value, i)
                    assert torch.equal(c.lse[s, i], clean[1][s, i])
                else:
                    assert torch.isnan(c.out[s, i]).all()
            assert torch.equal(c.out[1:], clean[0][1:])
            place[page, t % B] = old


def test_attend_far_scores():
    """Scores hundreds apart (weights that underflow) and all equal: the log-sum-exp of a block far below the row's
    stays finite and right."""
    for q_scale in (0.0, 60.0):
        for M in (1, 12):
            c = Case(1, M, 16, 2, 128, 16, 30, tree="tree", q_scale=q_scale)
            with _handle(16, 2, 128, 16, c.N) as p:
                c.run(p)
                c.check()
                assert torch.isfinite(c.block_lse[:, :5]).all()


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_attend_bad_tables_and_lengths(Hq, Hk, D, B, M):
    """A block with an invalid entry is left out; lengths out of range are clamped; both raise the error word."""
    n = max(4, -(-M // B) + 3)
    c = Case(2, M, Hq, Hk, D, B, n, tree="chain", ragged=False)
    with _handle(Hq, Hk, D, B, c.N) as p:
        for bad in (-1, c.N, 2 ** 31 - 1):
            tables = c.tables.clone()
            c.tables[:, 1] = bad
            c.run(p)
            with pytest.raises(rk.PredError) as e:
                rk.pred_device_error(p.handle)
            assert "block-table" in str(e.value)
            assert torch.isneginf(c.block_lse[:, 1]).all() and torch.isfinite(c.out).all()
            got = c.out.clone()
            # the same without the block: its tokens taken out of the table
            c.tables = torch.cat((tables[:, :1], tables[:, 2:], tables[:, 1:2]), 1).contiguous()
            lens, c.lens = c.lens, c.lens - B
            c.run(p)
            rk.pred_device_error(p.handle)
            c.check()
            # one rounding of each, and sums of another order: 2^-9 of values under 4
            assert torch.all((got.float() - c.out.float()).abs() <= 2 * HALF_BF16 * c.out.float().abs() + 2.0 ** -9)
            c.tables, c.lens = tables, lens
        for lens, drafts in (([n * B + 1, 5], [1, 1]), ([-3, 5], [0, 1]), ([5, 5], [1, -1]), ([5, 5], [1, M + 1]),
                             ([0, 5], [1, 1])):
            c.lens, c.drafts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, drafts))
            c.run(p)
            with pytest.raises(rk.PredError) as e:
                rk.pred_device_error(p.handle)
            assert "length" in str(e.value)
            c.lens = c.lens.clamp(0, n * B)
            c.drafts = torch.minimum(c.drafts.clamp(0, M), c.lens)
            c.check(weights=False)


@pytest.mark.parametrize("Hq,Hk,D,M,dtype", [(32, 8, 128, 1, torch.bfloat16), (8, 2, 64, 5, FP8), (16, 2, 128, 40, torch.bfloat16),
                                             (16, 2, 128, 8, torch.bfloat16), (16, 2, 128, 40, FP8), (8, 2, 64, 64, torch.bfloat16)])
def test_attend_long_context_with_bad_entries(Hq, Hk, D, M, dtype):
    """Invalid entries here and there in a long table, alone, side by side and at both ends, with NaN in every block that
    no sequence has (block 0 among them): the other blocks' tokens against the oracle."""
    _say("attend bad entries", Hq, Hk, D, M, dtype)
    B, n, S = 16, 130, 2
    c = Case(S, M, Hq, Hk, D, B, n, dtype, tree="tree", lens=[n * B, n * B - 37], drafts=[M, max(1, M // 2)])
    c.tables = (1 + torch.randperm(c.N - 1, generator=c.g)[:S * n]).view(S, n).int().cuda()
    bad = [[0, 17, 18, 61, 62, 63, 64, 100], [3, 4, 5, 6, 7, 8, 9, 90, 126]]
    for s in range(S):
        for at, b in enumerate(bad[s]):
            c.tables[s, b] = (-1, c.N, 2 ** 31 - 1)[at % 3]
    used = set(c.tables.flatten().tolist())
    for page in set(range(c.N)) - used:
        c.k[page], c.v[page] = (torch.full((), float("nan")).to(dtype) for _ in range(2))
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        with pytest.raises(rk.PredError) as e:
            rk.pred_device_error(p.handle)
        assert "block-table" in str(e.value)
    q, out, lse, blk = _f64(c.q), _f64(c.out), _f64(c.lse), _f64(c.block_lse)
    g = Hq // Hk
    for s in range(S):
        length, drafted = int(c.lens[s]), int(c.drafts[s])
        used_blocks = -(-length // B)
        pages = c.tables[s, :used_blocks].cpu().numpy().copy()
        pages[bad[s]] = [i for i in range(1, c.N) if i in used][0]      # any block: its tokens are not seen
        k = _f64(c.k[torch.from_numpy(pages).long().cuda()]) * c.scales[0]
        v = _f64(c.v[torch.from_numpy(pages).long().cuda()]) * c.scales[1]
        seen = cache.seen_by(M, length, drafted, c.tree[s].tolist())
        for b in bad[s]:
            seen[:, b * B:b * B + B] = False
        seen = np.repeat(seen, g, axis=0)
        for h in range(Hk):
            kk, vv = k[:, :, h].reshape(-1, D)[:length], v[:, :, h].reshape(-1, D)[:length]
            qq = q[s, :, h * g:h * g + g].reshape(-1, D)
            want, want_lse, x, absolute = cache.attend_one(qq, kk, vv, seen, c.scale)
            delta = (D + 4) * 2.0 ** -24 * c.scale * (np.abs(qq) @ np.abs(kk).T).max()
            rel = 2 * delta + 2.0 ** -20 + 2.0 ** -16 + (length + 64) * 2.0 ** -24
            got = out[s, :, h * g:h * g + g].reshape(-1, D)
            assert np.all(np.abs(got - want) <= HALF_BF16 * np.abs(want) + rel * absolute), ("out", s, h)
            Case._close_log(lse[s, :, h * g:h * g + g].reshape(-1), want_lse, rel, ("lse", s, h))
            got = blk[s, :used_blocks, :, h * g:h * g + g].reshape(used_blocks, M * g)
            Case._close_log(got, cache.block_lse_one(x, B), rel, ("block_lse", s, h))


def test_attend_long_sequence_far_slots():
    """A cache whose slots lie beyond 2^32 bytes: 40000 blocks of 128 KiB, a sequence scattered over them."""
    Hq, Hk, D, B, N, n = 16, 8, 128, 32, 40000, 300
    k = torch.zeros((N, B, Hk, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Case(1, 2, Hq, Hk, D, B, n, tree="chain")
    far = (torch.arange(n) * 131 + 600).int()
    far[-1] = N - 1
    k[far.long().cuda()], v[far.long().cuda()] = c.k[c.tables[0].long()], c.v[c.tables[0].long()]
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        first = [t.clone() for t in (c.out, c.lse, c.block_lse)]
    c.k, c.v, c.N = k, v, N
    c.kv, c.tables = rk.KVCache(k, v), far.view(1, n).cuda()
    with _handle(Hq, Hk, D, B, N) as p:
        c.run(p)
        rk.pred_device_error(p.handle)
        for got, want in zip((c.out, c.lse, c.block_lse), first):
            assert torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 16, 64])
def test_attend_long_context_split(M):
    """Contexts long enough to be split over workgroups, sampled sequences against the oracle; the same bits again."""
    c = Case(3, M, 8, 2, 128, 16, 900, tree="tree" if M > 1 else "chain", lens=[14400, 5, 9001][:3] if M == 1 else
             [14400, M + 100, 9001])
    with _handle(8, 2, 128, 16, c.N) as p:
        c.run(p)
        c.check()
        again = [t.clone() for t in (c.out, c.lse, c.block_lse)]
        c.run(p)
        for got, want in zip((c.out, c.lse, c.block_lse), again):
            assert torch.equal(got, want)


@pytest.mark.parametrize("S,M,Hq,Hk,D,B,n,dtype", [
    (65, 1, 4, 1, 64, 16, 40, torch.bfloat16), (150, 3, 4, 2, 128, 16, 40, FP8), (700, 1, 8, 1, 64, 8, 30, torch.bfloat16),
    (129, 20, 4, 2, 64, 16, 40, FP8), (300, 64, 2, 1, 128, 32, 12, torch.bfloat16)])
def test_attend_many_sequences(S, M, Hq, Hk, D, B, n, dtype):
    """More sequences than a wave has lanes, of very different lengths (one of every block, others of nothing): sampled
    sequences against the oracle, the ends of each 64 among them; the same bits again."""
    _say("attend many", S, M, Hq, Hk, D, B, n, dtype)
    g = torch.Generator().manual_seed(S + M)
    lens = torch.randint(0, 3 * B, (S,), generator=g)
    lens[S // 2] = lens[1] = n * B
    lens[[0, 2, 63, S - 1]] = torch.tensor([0, 1, n * B - 1, 5])
    drafts = torch.minimum(torch.randint(0, M + 1, (S,), generator=g), lens)
    c = Case(S, M, Hq, Hk, D, B, n, dtype, tree="tree", lens=lens, drafts=drafts)
    with _handle(Hq, Hk, D, B, c.N) as p:
        c.run(p)
        rk.pred_device_error(p.handle)
        c.check(seqs=sorted({0, 1, 2, 3, 62, 63, 64, S // 2, S // 2 + 1, S - 2, S - 1}))
        again = [t.clone() for t in (c.out, c.lse, c.block_lse)]
        c.run(p)
        for got, want in zip((c.out, c.lse, c.block_lse), again):
            assert torch.equal(got, want)


KERNELS = [     # Hq, Hk, D, B, M, dtype, with block_lse, the kernel
    (32, 8, 128, 16, 1, torch.bfloat16, True, "attend_stream_kernel"),
    (32, 8, 128, 16, 8, FP8, True, "attend_stream_kernel"),        # 32 queries for each kv head
    (32, 8, 128, 16, 9, FP8, True, "attend_tree_kernel"),
    (8, 2, 64, 8, 1, torch.bfloat16, True, "attend_stream_kernel"),
    (8, 2, 64, 8, 1, FP8, True, "attend_tree_kernel"),             # a wave-load is 16 tokens
    (8, 2, 64, 8, 64, FP8, False, "attend_tree_kernel"),
    (4, 2, 128, 7, 2, torch.bfloat16, False, "attend_tree_kernel"),
    (4, 2, 128, 7, 2, torch.bfloat16, True, "attend_plain_kernel"),
    (4, 2, 64, 1, 1, FP8, False, "attend_tree_kernel"),
    (4, 2, 80, 16, 1, torch.bfloat16, False, "attend_plain_kernel"),
]


@pytest.mark.parametrize("Hq,Hk,D,B,M,dtype,weights,name", KERNELS)
def test_attend_kernel_of_a_shape(Hq, Hk, D, B, M, dtype, weights, name):
    """The kernel that runs for a shape, over a context of many runs and a short one, against the oracle."""
    _say("attend kernel", Hq, Hk, D, B, M, dtype, weights, name)
    n = 1500 // B
    c = Case(2, M, Hq, Hk, D, B, n, dtype, tree="tree", lens=[n * B, M], drafts=[M, M])
    with _handle(Hq, Hk, D, B, c.N) as p:
        assert rk.pred_attend_kernel_name(p.handle, c.kv, M, weights) == name
        c.run(p, weights)
        rk.pred_device_error(p.handle)
        c.check(weights)


@pytest.mark.parametrize("M", [1, 40])
def test_attend_block_beyond_two_gib(M):
    """A block whose tokens lie 4 MiB apart, 2.5 GiB in all: offsets inside it pass 31 bits."""
    Hq, Hk, D, B, apart = 4, 2, 64, 640, 1 << 21
    c = Case(1, M, Hq, Hk, D, B, 1, identity=True, tree="tree")
    for name in ("k", "v"):
        far = torch.empty((B * apart,), dtype=torch.bfloat16, device="cuda")
        far = far.as_strided((1, B, Hk, D), (B * apart, apart, D, 1))
        far.copy_(getattr(c, name))
        setattr(c, name, far)
    c.kv = rk.KVCache(c.k, c.v)
    with _handle(Hq, Hk, D, B, 1) as p:
        assert rk.pred_attend_kernel_name(p.handle, c.kv, M) == "attend_tree_kernel"
        c.run(p, weights=False)
        rk.pred_device_error(p.handle)
        c.check(weights=False)


@pytest.mark.parametrize("Hq,Hk,D,B,M", SHAPES)
def test_attend_scales(Hq, Hk, D, B, M):
    """A scale of zero weighs every seen token alike; a negative one turns the order round."""
    n = 4
    for scale in (0.0, -0.3):
        c = Case(2, M, Hq, Hk, D, B, n, lens=[n * B, n * B // 2 + 1], drafts=[1, min(M, n * B // 2 + 1)])
        c.scale = scale
        with _handle(Hq, Hk, D, B, c.N) as p:
            c.run(p)
            rk.pred_device_error(p.handle)
            c.scale = scale
            _check_scaled(c)


def _check_scaled(c):
    """Case.check, whose tolerance takes the scale's magnitude."""
    q, k, v, out, lse = _f64(c.q), _f64(c.k), _f64(c.v), _f64(c.out), _f64(c.lse)
    g = c.Hq // c.Hk
    for s in range(c.S):
        length, drafted = int(c.lens[s]), int(c.drafts[s])
        pages = c.tables[s, :-(-length // c.B)].cpu().numpy()
        seen = np.repeat(cache.seen_by(c.M, length, drafted, None), g, axis=0)
        for h in range(c.Hk):
            kk, vv = (t[pages, :, h].reshape(-1, c.D)[:length] for t in (k, v))
            qq = q[s, :, h * g:h * g + g].reshape(-1, c.D)
            want, want_lse, _, absolute = cache.attend_one(qq, kk, vv, seen, c.scale)
            delta = (c.D + 4) * 2.0 ** -24 * abs(c.scale) * (np.abs(qq) @ np.abs(kk).T).max()
            rel = 2 * delta + 2.0 ** -20 + 2.0 ** -16 + (length + 64) * 2.0 ** -24
            got = out[s, :, h * g:h * g + g].reshape(-1, c.D)
            assert np.all(np.abs(got - want) <= HALF_BF16 * np.abs(want) + rel * absolute), ("out", s, h)
            Case._close_log(lse[s, :, h * g:h * g + g].reshape(-1), want_lse, rel, ("lse", s, h))


# ---------------------------------------------------------------- weight and eviction

@pytest.mark.parametrize("S,M,Hq,B,n", [(1, 1, 4, 16, 7), (3, 1, 32, 16, 300), (2, 5, 5, 8, 33), (2, 64, 8, 16, 50),
                                        (2, 64, 64, 32, 17), (1, 3, 1, 1, 20), (1, 2, 300, 16, 9), (1, 1, 6, 16, 1)])
@pytest.mark.parametrize("accepted", [False, True])
def test_accumulate_weight(S, M, Hq, B, n, accepted):
    _say("weight", S, M, Hq, B, n, accepted)
    g = torch.Generator().manual_seed(S + M + Hq + n)
    lens = torch.randint(0, n * B + 1, (S,), generator=g)
    lens[0] = n * B - (B > 1)
    blk = 3 * torch.randn((S, n, M, Hq), generator=g)
    blk[torch.rand(blk.shape, generator=g) < 0.1] = -math.inf
    lse = torch.logsumexp(blk, 1)
    lse[0, M // 2] = -math.inf          # a row that saw nothing
    blk[0, :, M // 2] = -math.inf
    used = -(-lens // B)
    for s in range(S):
        blk[s, int(used[s]):] = math.nan    # never written
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (S,), generator=g) if accepted else None
    mass = torch.rand((S, n), generator=g) * 5
    with _handle(Hq, 1, 64, B, 16) as p:
        args = [lse.cuda(), blk.cuda(), None if words is None else words.cuda(), lens.int().cuda(), 0.75]
        old, new = mass.cuda(), torch.full((S, n), 9.0, device="cuda")
        rk.pred_accumulate_weight(p.handle, *args, old, new)
        rk.pred_device_error(p.handle)
        got = _f64(new)
        for s in range(S):
            rows = [i for i in range(M) if words is None or int(words[s]) >> i & 1]
            u = int(used[s])
            want = cache.accumulate(mass[s].numpy(), lse[s].double().numpy(), blk[s].double().numpy(), u, 0.75, rows)
            # exp of a difference rounded to 2^-24 of sizes up to 20, 2 ulps of exp, a sum of M Hq terms
            rel = 40 * 2.0 ** -24 + 2.0 ** -21 + (M * Hq + 8) * 2.0 ** -24
            assert np.all(np.abs(got[s, :u] - want[:u]) <= rel * np.abs(want[:u]) + 1e-30)
            assert np.array_equal(got[s, u:], mass[s, u:].double().numpy())
        rk.pred_accumulate_weight(p.handle, *args, old)         # in place
        assert torch.equal(old, new)


EVICT = [
    # S, n, B, budget, first, last
    (1, 1, 16, 0, 0, 1), (2, 5, 16, 3, 0, 1), (3, 64, 8, 40, 4, 5), (4, 100, 16, 0, 2, 3), (2, 2048, 16, 1000, 4, 8),
    (2, 2049, 16, 2000, 0, 1), (1, 8192, 16, 8191, 1, 1), (2, 8193, 1, 100, 0, 1), (1, 32768, 32, 20000, 7, 64),
    (2, 32769, 1, 30000, 3, 2), (1, 70001, 4, 1, 1000, 1000), (3, 300, 16, 299, 500, 1), (3, 300, 16, 10, 0, 2 ** 31 - 1),
    (3, 70, 16, 10 ** 12, 0, 1),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("values", ["spread", "ties", "odd"])
@pytest.mark.parametrize("S,n,B,budget,first,last", EVICT)
def test_evict_blocks(S, n, B, budget, first, last, values, in_place):
    _say("evict", S, n, B, budget, first, last, values, in_place)
    g = torch.Generator().manual_seed(S + n + B)
    tables = torch.randint(-2 ** 31, 2 ** 31 - 1, (S, n), generator=g).int()
    mass = torch.randn((S, n), generator=g).exp()
    if values == "ties":
        mass = torch.randint(0, 3, (S, n), generator=g).float()
    if values == "odd":
        some = torch.tensor([0.0, -0.0, math.nan, math.inf, -math.inf, 1e-42, -1.0, 3.0])
        mass = some[torch.randint(0, 8, (S, n), generator=g)]
    lens = torch.randint(0, n * B + 1, (S,), generator=g).int()
    lens[0] = n * B - (B > 1)
    with _handle(4, 1, 64, B, 16) as p:
        t, m, l = tables.cuda(), mass.cuda(), lens.cuda()
        outs = (t, m, l) if in_place else (torch.full_like(t, 5), torch.full_like(m, 5), torch.full_like(l, 5))
        gone = torch.full((S,), -7, dtype=torch.int32, device="cuda")
        need = rk.pred_evict_workspace_bytes(n, S)
        ws = torch.empty((need,), dtype=torch.uint8, device="cuda") if need else None
        rk.pred_evict_blocks(p.handle, t, m, l, budget, first, last, *outs, gone, ws)
        rk.pred_device_error(p.handle)
        for s in range(S):
            want = cache.evict(tables[s].tolist(), mass[s].tolist(), int(lens[s]), B, budget, first, last)
            assert outs[0][s].tolist() == want[0]
            assert np.array_equal(outs[1][s].cpu().numpy(), np.array(want[1], np.float32), equal_nan=True)
            assert int(outs[2][s]) == want[2] and int(gone[s]) == want[3]


def test_evict_takes_the_first_victims():
    """Evicted blocks are pred_select_victims's of the same scores, and the predictor's own scores serve as mass."""
    n, B = 600, 16
    scores = torch.randn((2, n), device="cuda")
    with _handle(4, 1, 64, B, 16) as p:
        victims = torch.empty((2, 90), dtype=torch.int32, device="cuda")
        rk.pred_select_victims(p.handle, scores, 90, victims)
        tables = torch.arange(2 * n, dtype=torch.int32, device="cuda").view(2, n).contiguous()
        lens = torch.full((2,), n * B, dtype=torch.int32, device="cuda")
        gone = torch.empty_like(lens)
        # nothing protected but the last block, which these scores place among the kept
        scores[:, -1] = 50.0
        rk.pred_select_victims(p.handle, scores, 90, victims)
        rk.pred_evict_blocks(p.handle, tables, scores, lens, n - 90, 0, 1, tables, scores, lens, gone)
        for s in range(2):
            assert sorted(victims[s].tolist()) == [x - s * n for x in tables[s, n - 90:].tolist()]
        assert lens.tolist() == [(n - 90) * B] * 2 and gone.tolist() == [90, 90]


def test_bad_lengths_are_clamped():
    with _handle(4, 1, 64, 16, 16) as p:
        tables = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10).contiguous()
        mass = torch.rand((2, 10), device="cuda")
        gone = torch.empty((2,), dtype=torch.int32, device="cuda")
        for lens, want in (([161, -1], [5, 0]), ([2 ** 31 - 1, 3], [5, 0])):
            l = torch.tensor(lens, dtype=torch.int32, device="cuda")
            out = torch.empty_like(l)
            rk.pred_evict_blocks(p.handle, tables, mass, l, 5, 0, 1, tables.clone(), mass.clone(), out, gone)
            with pytest.raises(rk.PredError) as e:
                rk.pred_device_error(p.handle)
            assert "length" in str(e.value) and gone.tolist() == want
            blk, lse = torch.zeros((2, 10, 1, 4), device="cuda"), torch.zeros((2, 1, 4), device="cuda")
            new = torch.empty_like(mass)
            rk.pred_accumulate_weight(p.handle, lse, blk, None, l, 1.0, mass, new)
            with pytest.raises(rk.PredError):
                rk.pred_device_error(p.handle)
            assert torch.equal(new[0], mass[0] + 4) and (lens[1] > 0 or torch.equal(new[1], mass[1]))


# ---------------------------------------------------------------- refusals

def test_refusals():
    D, B, Hk, N = 64, 16, 2, 8
    z = dict(device="cuda")
    with _handle(4, Hk, D, B, N) as p:
        h = p.handle
        k, v = _cache_tensors(N, B, Hk, D, torch.bfloat16, "tokens", fill=0.0)
        kv = rk.KVCache(k, v)
        rope, _, _ = _rope(64)
        q = torch.zeros((1, 1, 4, D), dtype=torch.bfloat16, **z)
        out, lse = torch.zeros_like(q), torch.zeros((1, 1, 4), **z)
        lens = torch.ones((1,), dtype=torch.int32, **z)
        tab = torch.zeros((1, N), dtype=torch.int32, **z)
        ws = torch.empty((rk.pred_attend_workspace_bytes(h, 1, 1, N) + 16,), dtype=torch.uint8, **z)

        def attend(**kw):
            a = dict(cache=kv, q=q, tree=None, block_tables=tab, kv_len=lens, draft_len=None, scale=1.0, out=out,
                     workspace=ws)
            a.update(kw)
            rk.pred_attend(h, **a)

        attend()
        for kw, err in ((dict(q=q[0]), TypeError), (dict(q=q.float()), TypeError), (dict(out=out[..., :32]), ValueError),
                        (dict(out=out.cpu()), ValueError), (dict(kv_len=lens.long()), TypeError),
                        (dict(block_tables=tab[0]), ValueError), (dict(lse=lse[0]), ValueError),
                        (dict(tree=torch.zeros((1, 2), dtype=torch.int64, **z)), ValueError),
                        (dict(block_lse=torch.zeros((1, N, 1, 3), **z)), ValueError),
                        (dict(q=q.expand(2, 1, 4, D)), ValueError), (dict(workspace=ws.cpu()), ValueError),
                        (dict(scale=math.nan), rk.PredError), (dict(block_tables=None, n_blocks=N + 1), rk.PredError),
                        (dict(q=torch.zeros((1, 65, 4, D), dtype=torch.bfloat16, **z),
                              out=torch.zeros((1, 65, 4, D), dtype=torch.bfloat16, **z)), rk.PredError),
                        (dict(q=torch.zeros((1, 0, 4, D), dtype=torch.bfloat16, **z),
                              out=torch.zeros((1, 0, 4, D), dtype=torch.bfloat16, **z)), rk.PredError)):
            with pytest.raises(err):
                attend(**kw)
        with pytest.raises(rk.PredError) as e:
            attend(q=torch.zeros((1 + q.numel(),), dtype=torch.bfloat16, **z)[1:].view(q.shape))
        assert e.value.code == rk.PRED_ERR_UNSUPPORTED
        big = rk.pred_attend_workspace_bytes(h, 1, 1, N)
        if big:
            with pytest.raises(rk.PredError) as e:
                attend(workspace=ws[:big - 1])
            assert e.value.code == rk.PRED_ERR_WORKSPACE
            with pytest.raises(rk.PredError) as e:
                attend(workspace=None)
            assert e.value.code == rk.PRED_ERR_WORKSPACE
        # caches
        for bad in ((k[:, :8], v[:, :8]), (k[:4], v[:4]), (k[..., :32], v[..., :32])):
            with pytest.raises(ValueError):
                attend(cache=rk.KVCache(*bad))
        with pytest.raises(ValueError):
            rk.KVCache(k, v.transpose(1, 2).contiguous().transpose(1, 2))
        with pytest.raises(ValueError):
            rk.KVCache(k, v.to(FP8))
        with pytest.raises(TypeError):
            rk.KVCache(k.float(), v.float())
        with pytest.raises(ValueError):
            rk.KVCache(k.transpose(2, 3), v.transpose(2, 3))
        for scales in ((2.0, 1.0), (1.0, 0.0), (1.0, math.inf), (1.0, math.nan), (-1.0, 1.0)):
            with pytest.raises(rk.PredError):
                attend(cache=rk.KVCache(k, v, *scales))
        base = torch.zeros((N * B * Hk * D * 2,), dtype=torch.bfloat16, **z)
        for strides in ((B * Hk * D, D, D, 1), (B * Hk * D, Hk * D, 32, 1), (B * D, Hk * D, D, 1),
                        (B * Hk * D + 4, Hk * D, D, 1), (B * Hk * D, 0, D, 1)):
            t = base.as_strided((N, B, Hk, D), strides)
            with pytest.raises(rk.PredError):
                attend(cache=rk.KVCache(t, t))
        # rotations
        x = torch.zeros((3, 4, D), dtype=torch.bfloat16, **z)
        pos = torch.zeros((3,), dtype=torch.int32, **z)
        kk = torch.zeros((3, Hk, D), dtype=torch.bfloat16, **z)
        slots = torch.full((3,), -1, dtype=torch.int64, **z)
        rk.pred_rotate_store(h, rope, x, kk, kk, pos, slots, kv, torch.empty_like(x))
        for args, err in (((x[..., :32], pos, x), ValueError), ((x, pos.long(), x), TypeError),
                          ((x, pos[:2], x), ValueError), ((x.transpose(0, 1), pos, x), ValueError),
                          ((x, pos, x.cpu()), ValueError)):
            with pytest.raises(err):
                rk.pred_rotate(h, rope, *args)
        wide, _, _ = _rope(128)
        back, _, _ = _rope(64, backward=True)
        for r in (wide, rk.Rope(rope.turns, 64, mscale=math.nan)):
            with pytest.raises(rk.PredError) as e:
                rk.pred_rotate(h, r, x, pos, x)
            assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE
        with pytest.raises(rk.PredError):
            rk.pred_rotate_store(h, back, x, kk, kk, pos, slots, kv, torch.empty_like(x))
        with pytest.raises(ValueError):
            rk.Rope(rope.turns, 62)
        with pytest.raises(TypeError):
            rk.Rope(rope.turns.cpu(), 64)
        with pytest.raises(ValueError):
            rk.pred_rotate_store(h, rope, x, kk[:2], kk, pos, slots, kv, torch.empty_like(x))
        strided = torch.zeros((3, 6, D), dtype=torch.bfloat16, **z)[:, :4]
        with pytest.raises(rk.PredError):       # in place with the tokens apart
            lib = rk.lib()
            rk.cache._check(lib.pred_rotate_store(h, rope._ref, strided.data_ptr(), 6 * D, kk.data_ptr(), Hk * D,
                                                  kk.data_ptr(), Hk * D, 3, pos.data_ptr(), slots.data_ptr(), kv._ref,
                                                  strided.data_ptr(), None))
        # eviction and weight
        mass = torch.zeros((1, N), **z)
        gone = torch.zeros_like(lens)
        for budget, first, last in ((-1, 0, 1), (1, -1, 1), (1, 0, 0)):
            with pytest.raises(rk.PredError) as e:
                rk.pred_evict_blocks(h, tab, mass, lens, budget, first, last, tab, mass, lens, gone)
            assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE
        with pytest.raises(rk.PredError):
            rk.pred_evict_blocks(h, tab, mass, None, 1, 0, 1, tab, mass, lens, gone)
        big = 32769
        t2, m2 = torch.zeros((1, big), dtype=torch.int32, **z), torch.zeros((1, big), **z)
        for w in (None, torch.empty((8 * big - 1,), dtype=torch.uint8, **z)):
            with pytest.raises(rk.PredError) as e:
                rk.pred_evict_blocks(h, t2, m2, lens, 1, 0, 1, t2, m2, lens, gone, w)
            assert e.value.code == rk.PRED_ERR_WORKSPACE
        blk = torch.zeros((1, N, 1, 4), **z)
        with pytest.raises(rk.PredError):
            rk.pred_accumulate_weight(h, lse, blk, None, lens, math.inf, mass)
        with pytest.raises(ValueError):
            rk.pred_accumulate_weight(h, lse, blk, None, lens, 1.0, mass[:, 1:])
        with pytest.raises(rk.PredError):
            rk.pred_accumulate_weight(h, None, blk, None, lens, 1.0, mass)
        rk.pred_device_error(h)
    with _handle(2, 1, 264, 16, 2) as p:
        k, v = _cache_tensors(2, 16, 1, 264, torch.bfloat16, "tokens", fill=0.0)
        q = torch.zeros((1, 1, 2, 264), dtype=torch.bfloat16, **z)
        with pytest.raises(rk.PredError) as e:
            rk.pred_attend(p.handle, rk.KVCache(k, v), q, None, None, None, None, 1.0, torch.empty_like(q))
        assert e.value.code == rk.PRED_ERR_UNSUPPORTED


def test_overlaps_are_refused():
    """An attention whose output lies on its queries, a store into a cache whose k and v are one."""
    D, B, Hk, N = 64, 16, 2, 8
    z = dict(device="cuda")
    with _handle(4, Hk, D, B, N) as p:
        k, v = _cache_tensors(N, B, Hk, D, torch.bfloat16, "tokens", fill=0.0)
        kv, lens = rk.KVCache(k, v), torch.ones((2,), dtype=torch.int32, **z)
        both = torch.zeros((3, 1, 4, D), dtype=torch.bfloat16, **z)
        ws = torch.empty((rk.pred_attend_workspace_bytes(p.handle, 2, 1, N) + 16,), dtype=torch.uint8, **z)

        def attend(q, out, table=None):
            rk.pred_attend(p.handle, kv, q, None, table, lens[:q.shape[0]], None, 1.0, out, workspace=ws)

        attend(both[:1], both[1:2])         # side by side
        for q, out in ((both[:2], both[:2]), (both[:2], both[1:]), (both[1:], both[:2])):
            with pytest.raises(rk.PredError) as e:
                attend(q, out)
            assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE and "overlaps" in str(e.value)
        with pytest.raises(TypeError):
            attend(both[:1], both[1:2], np.zeros((1, N), np.int32))
        rope, _, _ = _rope(64)
        x = torch.zeros((3, 4, D), dtype=torch.bfloat16, **z)
        kk = torch.zeros((3, Hk, D), dtype=torch.bfloat16, **z)
        slots, pos = torch.full((3,), -1, dtype=torch.int64, **z), torch.zeros((3,), dtype=torch.int32, **z)
        with pytest.raises(rk.PredError) as e:
            rk.pred_rotate_store(p.handle, rope, x, kk, kk, pos, slots, rk.KVCache(k, k), torch.empty_like(x))
        assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE
        rk.pred_device_error(p.handle)


def test_nothing_to_do():
    with _handle(4, 1, 64, 16, 4) as p:
        h = p.handle
        k, v = _cache_tensors(4, 16, 1, 64, torch.bfloat16, "tokens", fill=1.0)
        kv, z = rk.KVCache(k, v), dict(device="cuda")
        rope, _, _ = _rope(64)
        none = torch.empty((0, 4, 64), dtype=torch.bfloat16, **z)
        i0 = torch.empty((0,), dtype=torch.int32, **z)
        rk.pred_rotate(h, rope, none, i0, none)
        rk.pred_rotate_store(h, rope, none, none[:, :1], none[:, :1], i0, i0.long(), kv, none)
        q = torch.empty((0, 2, 4, 64), dtype=torch.bfloat16, **z)
        rk.pred_attend(h, kv, q, None, torch.empty((0, 3), dtype=torch.int32, **z), i0, None, 1.0, q)
        # no blocks: every row is empty
        q = torch.ones((2, 3, 4, 64), dtype=torch.bfloat16, **z)
        out, lse = torch.ones_like(q), torch.ones((2, 3, 4), **z)
        rk.pred_attend(h, kv, q, None, torch.empty((2, 0), dtype=torch.int32, **z), None, None, 1.0, out, lse)
        assert torch.all(out == 0) and torch.isneginf(lse).all()
        lens = torch.zeros((2,), dtype=torch.int32, **z)
        tab, mass = torch.empty((2, 0), dtype=torch.int32, **z), torch.empty((2, 0), **z)
        gone = torch.ones_like(lens)
        rk.pred_evict_blocks(h, tab, mass, lens, 1, 0, 1, tab, mass, lens, gone)
        assert gone.tolist() == [0, 0] and lens.tolist() == [0, 0]
        rk.pred_device_error(h)


# ---------------------------------------------------------------- together

class Serving:
    """A tiny serving loop over one cache: each step stores and attends a few drafted tokens of every sequence, accepts
    some of them, accumulates the weights and trims every sequence to its budget."""

    def __init__(self, dtype, S=3, M=4, Hq=8, Hk=2, D=64, B=16, budget=6):
        self.S, self.M, self.Hq, self.Hk, self.D, self.B, self.budget = S, M, Hq, Hk, D, B, budget
        self.n = budget + 3
        self.N = S * self.n
        self.k, self.v = _cache_tensors(self.N, B, Hk, D, dtype, "tokens", fill=0.0)
        self.scales = (0.0625, 0.0625) if dtype == FP8 else (1.0, 1.0)
        self.kv = rk.KVCache(self.k, self.v, *self.scales)
        self.rope, self.freq, _ = _rope(D, 10000.0)
        z = dict(device="cuda")
        self.p = _handle(Hq, Hk, D, B, self.N)
        self.tables = torch.randperm(self.N, generator=torch.Generator().manual_seed(5)).int().view(S, self.n).cuda()
        self.lens = torch.zeros((S,), dtype=torch.int32, **z)       # with the draft
        self.mass = torch.zeros((S, self.n), **z)
        self.qkv = torch.zeros((S * M, Hq + 2 * Hk, D), dtype=torch.bfloat16, **z)
        self.positions = torch.zeros((S * M,), dtype=torch.int32, **z)
        self.slots = torch.full((S * M,), -1, dtype=torch.int64, **z)
        self.q = torch.zeros((S * M, Hq, D), dtype=torch.bfloat16, **z)
        self.out = torch.zeros((S, M, Hq, D), dtype=torch.bfloat16, **z)
        self.lse = torch.zeros((S, M, Hq), **z)
        self.block_lse = torch.zeros((S, self.n, M, Hq), **z)
        self.drafts = torch.full((S,), M, dtype=torch.int32, **z)
        self.tree = torch.tensor([[1, 3, 5, 11][:M]] * S, **z)
        self.accepted = torch.full((S,), 0b1011, dtype=torch.int64, **z)
        self.gone = torch.zeros((S,), dtype=torch.int32, **z)
        self.ws = torch.empty((rk.pred_attend_workspace_bytes(self.p.handle, S, M, self.n) + 1,), dtype=torch.uint8, **z)

    def device_step(self):
        h, Hq, Hk = self.p.handle, self.Hq, self.Hk
        rk.pred_rotate_store(h, self.rope, self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hk], self.qkv[:, Hq + Hk:],
                             self.positions, self.slots, self.kv, self.q)
        rk.pred_attend(h, self.kv, self.q.view(self.S, self.M, Hq, self.D), self.tree, self.tables, self.lens,
                       self.drafts, 0.125, self.out, self.lse, self.block_lse, self.ws)
        rk.pred_accumulate_weight(h, self.lse, self.block_lse, self.accepted, self.lens, 0.9, self.mass)
        rk.pred_evict_blocks(h, self.tables, self.mass, self.lens, self.budget, 1, 2, self.tables, self.mass, self.lens,
                             self.gone)

    def feed(self, step):
        """The next draft's inputs, written into the buffers the step reads (the whole draft stays in the cache)."""
        g = torch.Generator().manual_seed(1000 + step)
        x = torch.randn(self.qkv.shape, generator=g).bfloat16()
        self.qkv.copy_(x)
        lens, tables = self.lens.cpu(), self.tables.cpu()
        slots = torch.empty((self.S, self.M), dtype=torch.int64)
        for s in range(self.S):
            for i in range(self.M):
                t = int(lens[s]) + i
                slots[s, i] = int(tables[s, t // self.B]) * self.B + t % self.B
        self.slots.copy_(slots.view(-1))
        self.positions.copy_(torch.arange(step * self.M, step * self.M + self.M).repeat(self.S).int())
        self.lens += self.M

    def state(self):
        return [t.clone() for t in (self.out, self.lse, self.tables, self.mass, self.lens, self.gone, self.k, self.v)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_serving_loop(dtype):
    """The operators together, step after step past several evictions, against the oracle run beside them."""
    w = Serving(dtype)
    S, M, B, g = w.S, w.M, w.B, w.Hq // w.Hk
    mass = np.zeros((S, w.n))
    evictions = 0
    for step in range(40):
        before_tables = w.tables.cpu().tolist()
        w.feed(step)
        lens = w.lens.tolist()
        w.device_step()
        rk.pred_device_error(w.p.handle)
        evictions += int(w.gone.sum())
        k, v = _f64(w.k) * w.scales[0], _f64(w.v) * w.scales[1]
        q = cache.rotate(_f64(w.qkv[:, :w.Hq]), w.positions.tolist(), w.freq)
        assert np.all(np.abs(_f64(w.q) - q) <= HALF_BF16 * np.abs(q) + 2.0 ** -18)
        q = _f64(w.q).reshape(S, M, w.Hq, w.D)
        for s in range(S):
            used = -(-lens[s] // B)
            pages = before_tables[s][:used]
            lse, blk = np.empty((M, w.Hq)), np.empty((used, M, w.Hq))
            seen = np.repeat(cache.seen_by(M, lens[s], M, w.tree[s].tolist()), g, axis=0)
            for h in range(w.Hk):
                kk, vv = (c[pages, :, h].reshape(-1, w.D)[:lens[s]] for c in (k, v))
                head = slice(h * g, h * g + g)
                want, want_lse, x, absolute = cache.attend_one(q[s, :, head].reshape(-1, w.D), kk, vv, seen, 0.125)
                got = _f64(w.out[s, :, head]).reshape(-1, w.D)
                assert np.all(np.abs(got - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -14 * absolute)
                lse[:, head] = want_lse.reshape(M, g)
                blk[:, :, head] = cache.block_lse_one(x, B).reshape(used, M, g)
            mass[s] = cache.accumulate(mass[s], lse, blk, used, 0.9, [0, 1, 3])
            table, new_mass, length, gone = cache.evict(before_tables[s], mass[s].tolist(), lens[s], B, w.budget, 1, 2)
            assert w.tables[s].tolist() == table and int(w.lens[s]) == length and int(w.gone[s]) == gone
            mass[s] = new_mass
            assert np.all(np.abs(_f64(w.mass[s]) - mass[s]) <= 2.0 ** -12 * mass[s])
    assert evictions >= 3 * S
    w.p.close()


def test_serving_step_in_a_graph():
    """The whole step captured once and replayed, each replay against the eager step on a twin; two graphs with
    workspaces of their own take turns."""
    a, b = Serving(torch.bfloat16), Serving(torch.bfloat16)
    for w in (a, b):        # warm: libraries, first launches
        w.feed(0)
        w.device_step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        state = [t.clone() for t in (b.tables, b.mass, b.lens)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.device_step()
        graphs.append(graph)
        for t, old in zip((b.tables, b.mass, b.lens), state):
            t.copy_(old)
        b.ws = torch.empty_like(b.ws)
    for step in range(1, 30):
        a.feed(step)
        a.device_step()
        b.feed(step)
        graphs[step % 2].replay()
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y), step
    a.p.close()
    b.p.close()


def test_other_streams():
    """Calls on a stream of the caller's, given or current, with the inputs made on it."""
    c = Case(2, 3, 16, 2, 128, 16, 40, tree="tree")
    with _handle(16, 2, 128, 16, c.N) as p:
        c.run(p)
        want = [t.clone() for t in (c.out, c.lse, c.block_lse)]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for given in (False, True):
            side.wait_stream(torch.cuda.current_stream())
            if given:       # the buffers' fill runs on the current stream, before the call on the other
                need = rk.pred_attend_workspace_bytes(p.handle, c.S, c.M, c.n)
                keep = torch.empty((max(need, 1),), dtype=torch.uint8, device="cuda")
                for t in (c.out, c.lse, c.block_lse):
                    t.fill_(9.0)
                side.wait_stream(torch.cuda.current_stream())
                rk.pred_attend(p.handle, c.kv, c.q, c.tree, c.tables, c.lens, c.drafts, c.scale, c.out, c.lse,
                               c.block_lse, keep, stream=side)
            else:
                with torch.cuda.stream(side):
                    keep = c.run(p)
            side.synchronize()
            del keep
            for x, y in zip((c.out, c.lse, c.block_lse), want):
                assert torch.equal(x, y)


def test_attend_over_the_kept_blocks():
    """Attention over the blocks that the predictor keeps: a table of the kept blocks alone gives the softmax over their
    tokens, here checked against masking the others out."""
    S, Hq, Hk, D, B, n = 1, 8, 2, 64, 16, 40
    c = Case(S, 1, Hq, Hk, D, B, n, ragged=False)
    with rk.Predictor(rk.dims(1, Hq, Hk, D, 16, B, c.N), seed=3) as p:
        rk.pred_project_kv_block(p.handle, 0, c.k[None].contiguous())
        q_proj = torch.empty((1, S, 1, Hq, 16), dtype=torch.bfloat16, device="cuda")
        rk.pred_project_q(p.handle, c.q, q_proj)
        scores = torch.empty((1, S, n), device="cuda")
        rk.pred_score_blocks(p.handle, 0, q_proj, c.tables, scores)
        mass, lens = scores[0], c.lens
        out_len, gone = torch.empty_like(lens), torch.empty_like(lens)
        rk.pred_evict_blocks(p.handle, c.tables, mass, lens, 10, 1, 1, c.tables, mass, out_len, gone)
        assert gone.tolist() == [30] and out_len.tolist() == [160]
        c.lens = out_len
        c.run(p)
        rk.pred_device_error(p.handle)
        c.check()
