"""GPU tests of the norms of queries and keys with the rotation and the store, their gradient, and the plain store and
load, against the float64 oracle (oracle/cache.py).

Tolerances, fixed before the first run, u = 2^-24:
* a normed value x r (o + w): a float32 sum of D squares is off by (D + 4) u relative, its root by half of that, and the
  reciprocal root, two products and offset + weight by a few u: ULPS(D) = (D / 2 + 12) u relative.
* a rotation: 2^-20 mscale (|a| + |b|) of the pair it turns (tests/test_gpu_cache.py).
* bf16 results: half a step, 2^-8 relative, more; e4m3 2^-4 relative or 2^-10 in the subnormals.
* a gradient dx = r (u - h m): the errors of u, h and m = mean(u h), the latter a float32 sum of D products.
* dweight: each summand's error, and N u sum |g h| for N summands added in any order.
"""

import math

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import cache
from tests.test_gpu_cache import FP8, HALF_BF16, _cache_tensors, _f64, _handle, _rope, _rotation_tolerance, _say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


def ulps(D):
    return (D / 2 + 12) * U


def _weight(g, D, kind):
    if kind is None:
        return None
    return (torch.randn((D,), generator=g) * 0.3 + (0.0 if kind else 1.0)).bfloat16().cuda()


def _w64(weight):
    return None if weight is None else _f64(weight)


def cache4(N, B, Hk, D, layout="heads"):
    """Bytes and scales of k and v of a 4-bit cache filled with a pattern, views [N, B, Hk, ..]."""
    def make(width, fill):
        if layout == "tokens":
            return [torch.full((N, B, Hk, width), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
        if layout == "heads":
            return [torch.full((N, Hk, B, width), fill, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
        pad = width * 32 // D           # 32 values of padding
        both = torch.full((N, 2, B, Hk, width + pad), fill, dtype=torch.uint8, device="cuda")[..., :width]
        return [both[:, 0], both[:, 1]]
    (k, v), (ks, vs) = make(D // 2, 0x21), make(D // 32, 125)
    return k, v, ks, vs


def values4(bits, scales):
    return cache.dequantise(cache.unpacked(bits.cpu().numpy()), scales.cpu().numpy())


NORMS = [
    # n, heads, D, rot (0: none), interleaved, kind, scaling arguments, first position, weight offset (None: no weight)
    (1, 4, 64, 64, False, "none", (), 0, 0.0),
    (5, 3, 64, 32, True, "linear", (4.0,), 77, 1.0),
    (67, 8, 128, 128, False, "llama3", (8.0, 1.0, 4.0, 8192.0), 131000, 0.0),
    (33, 5, 128, 64, True, "yarn", (16.0, 1.0, 32.0, 4096.0), 999000, None),
    (33, 17, 128, 32, False, "none", (), -40, 1.0),
    (9, 2, 80, 80, False, "ntk", (8.0,), 2 ** 31 - 10, 0.0),
    (9, 1, 80, 20, False, "none", (), 31, 0.0),         # pairs that straddle a lane's piece
    (4, 7, 96, 6, True, "none", (), 5, 1.0),
    (3, 70, 8, 2, False, "none", (), 5, 0.0),
    (3, 9, 16, 10, False, "none", (), 5, 0.0),
    (2, 3, 512, 512, True, "none", (), 4000, 0.0),
    (2, 3, 512, 256, False, "none", (), 4000, None),
    (5, 3, 256, 256, False, "none", (), 4000, 0.0),
    (300, 40, 128, 128, True, "none", (), -150, 0.0),
    (7, 6, 128, 0, False, "none", (), 0, 1.0),
    (2, 5, 24, 0, False, "none", (), 0, None),
    # tokens enough for a wave to take several heads of each place
    (1100, 13, 128, 128, False, "none", (), -7, 1.0),
    (1500, 17, 64, 32, True, "none", (), 100000, 0.0),
    (2300, 3, 256, 0, False, "none", (), 0, 0.0),
    (1200, 5, 80, 20, False, "none", (), 31, None),
]


def _inputs(n, heads, D, rot, inter, kind, args, first, offset):
    g = torch.Generator().manual_seed(n * 1000 + D + rot)
    rope, freq, mscale = _rope(rot, 500000.0, kind, args, inter) if rot else (None, None, 1.0)
    x = torch.randn((n, heads, D), generator=g) * torch.exp(2 * torch.randn((n, heads, 1), generator=g))
    x[0, 0] = 0                                     # a head of zeros
    pos = torch.arange(first, first + n, dtype=torch.int64)
    positions = ((pos + 2 ** 31) % 2 ** 32 - 2 ** 31).to(torch.int32).cuda()    # int32, wrapping at its end
    weight = _weight(g, D, offset)
    norm = rk.Norm(weight, 1e-5, offset or 0.0)
    return g, rope, freq, mscale, x.bfloat16(), positions, weight, norm


@pytest.mark.parametrize("n,heads,D,rot,inter,kind,args,first,offset", NORMS)
def test_norm_rotate(n, heads, D, rot, inter, kind, args, first, offset):
    _say("norm", n, heads, D, rot, inter, kind, first, offset)
    g, rope, freq, mscale, x0, positions, weight, norm = _inputs(n, heads, D, rot, inter, kind, args, first, offset)
    store = torch.full((n, heads + 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    x = store[:, 1:heads + 1]                       # tokens apart
    x.copy_(x0)
    with _handle(8, 2, D, 16, 4) as p:
        out = torch.full((n, heads + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
        rk.pred_norm_rotate(p.handle, norm, rope, x, positions if rot else None, out[:, :heads])
        normed = cache.norm(_f64(x), _w64(weight), 1e-5, offset or 0.0)
        want = normed if not rot else cache.rotate(normed, positions.cpu().numpy(), freq, mscale, inter)
        tol = HALF_BF16 * np.abs(want) + ulps(D) * np.abs(normed)
        if rot:     # an error of the pair's other value comes along
            tol = tol + (1 + ulps(D) * 2 ** 20) * _rotation_tolerance(normed, want, rot, inter, mscale)
        err = np.abs(_f64(out[:, :heads]) - want)
        assert np.all(err <= tol), (err - tol).max()
        assert torch.all(out[:, heads:] == 7)                                   # the row's rest stays
        rk.pred_norm_rotate(p.handle, norm, rope, x, positions if rot else None, x)     # in place
        assert torch.equal(x, out[:, :heads])
        assert torch.all(store[:, 0] == 5) and torch.all(store[:, -1] == 5)


def _gradient_bounds(x, dy, freq, positions, weight, offset, mscale, inter, rot, eps):
    """The oracle's gradients and how far float32 ones may be off."""
    D = x.shape[-1]
    g = dy if freq is None else cache.rotate(dy, positions, freq, mscale, inter, backward=True)
    eg = 4 * U * np.abs(g) + (0 if freq is None else _rotation_tolerance(dy, g, rot, inter, mscale))
    factor = np.ones(D) if weight is None else offset + weight
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h, u = x * r, g * factor
    eu, eh = eg * np.abs(factor) + 3 * U * np.abs(u), ulps(D) * np.abs(h)
    em = (eu * np.abs(h) + np.abs(u) * eh).mean(-1, keepdims=True) + (D + 8) * U * (np.abs(u * h)).mean(-1, keepdims=True)
    m = (u * h).mean(-1, keepdims=True)
    dx, dw = cache.norm_rotate_gradient(x, dy, positions, freq, weight, eps, offset, mscale, inter)
    tol = HALF_BF16 * np.abs(dx) + r * (eu + np.abs(h) * em + (eh + 4 * U * np.abs(h)) * np.abs(m)) + ulps(D) * r * (
        np.abs(u) + np.abs(h * m))
    N = x.shape[0] * x.shape[1]
    tol_w = (eg * np.abs(h) + np.abs(g) * eh).sum((0, 1)) + (N + 8) * U * np.abs(g * h).sum((0, 1))
    return dx, dw, tol, tol_w


@pytest.mark.parametrize("n,heads,D,rot,inter,kind,args,first,offset", [c for c in NORMS if c[0] < 300])
def test_gradient(n, heads, D, rot, inter, kind, args, first, offset):
    _say("gradient", n, heads, D, rot, inter, kind, first, offset)
    g, rope, freq, mscale, x0, positions, weight, norm = _inputs(n, heads, D, rot, inter, kind, args, first, offset)
    x = x0.cuda()
    wide = torch.randn((n, heads + 1, D), generator=g).bfloat16().cuda()
    dy = wide[:, 1:]
    with _handle(8, 2, D, 16, 4) as p:
        need = rk.pred_norm_rotate_workspace_bytes(p.handle, n, heads)
        ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")
        dx, dw = torch.full_like(x, 9.0), torch.full((D,), 9.0, device="cuda")
        pos = positions if rot else None
        rk.pred_norm_rotate_backward(p.handle, norm, rope, x, pos, dy, dx, dw, ws)
        want, want_w, tol, tol_w = _gradient_bounds(_f64(x), _f64(dy), freq, positions.cpu().numpy(), _w64(weight),
                                                    offset or 0.0, mscale, inter, rot, 1e-5)
        err = np.abs(_f64(dx) - want)
        assert np.all(err <= tol), (err - tol).max()
        err = np.abs(_f64(dw) - want_w)
        assert np.all(err <= tol_w), (err - tol_w).max()
        # without the weight's, into dy and into x
        alone = torch.empty_like(dx)
        rk.pred_norm_rotate_backward(p.handle, norm, rope, x, pos, dy, alone)
        assert torch.equal(alone, dx)
        rk.pred_norm_rotate_backward(p.handle, norm, rope, x, pos, dy, dy)
        assert torch.equal(dy, dx)
        wide.copy_(torch.randn((n, heads + 1, D), generator=g))
        again = torch.empty_like(dw)
        rk.pred_norm_rotate_backward(p.handle, norm, rope, x, pos, dy, dx, dw, ws)
        rk.pred_norm_rotate_backward(p.handle, norm, rope, x, pos, dy, x, again, ws)
        assert torch.equal(x, dx) and torch.equal(again, dw)


def test_gradient_is_the_difference():
    """dx against central differences of the oracle's forward, steps of 2^-10: a third derivative of order 10 times
    2^-20 / 6, and dx's own bf16 step."""
    r = np.random.default_rng(3)
    D, pos = 16, [3, -11]
    rope, freq, _ = _rope(16, 100.0)
    x, dy = (torch.from_numpy(r.standard_normal((2, 2, D))).bfloat16().cuda() for _ in range(2))
    w = torch.from_numpy(1 + 0.3 * r.standard_normal(D)).bfloat16().cuda()
    with _handle(2, 1, D, 16, 4) as p:
        dx, dw = torch.empty_like(x), torch.empty((D,), device="cuda")
        ws = torch.empty((rk.pred_norm_rotate_workspace_bytes(p.handle, 2, 2),), dtype=torch.uint8, device="cuda")
        rk.pred_norm_rotate_backward(p.handle, rk.Norm(w, 1e-2), rope, x, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                                     dy, dx, dw, ws)
    x, dy, w = _f64(x), _f64(dy), _f64(w)

    def value(x, w):
        return (cache.rotate(cache.norm(x, w, 1e-2), pos, freq) * dy).sum()

    step = 2.0 ** -10
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = step
        slope = (value(x + e, w) - value(x - e, w)) / (2 * step)
        assert abs(_f64(dx)[at] - slope) <= HALF_BF16 * abs(slope) + 1e-5
    for j in range(D):
        e = np.zeros(D)
        e[j] = step
        assert abs(_f64(dw)[j] - (value(x, w + e) - value(x, w - e)) / (2 * step)) <= 1e-5


@pytest.mark.parametrize("n,heads,D", [(9000, 5, 128), (2500, 64, 64), (700, 3, 96)])
def test_gradient_of_many_tokens(n, heads, D):
    """More units than workgroups: against torch's differentiation in 64 bits, and twice the same bits."""
    _say("gradient many", n, heads, D)
    g = torch.Generator().manual_seed(n)
    x, dy = (torch.randn((n, heads, D), generator=g).bfloat16().cuda() for _ in range(2))
    w = (1 + 0.2 * torch.randn((D,), generator=g)).bfloat16().cuda()
    rope, freq, _ = _rope(D, 500000.0)
    positions = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32).cuda()
    with _handle(8, 2, D, 16, 4) as p:
        ws = torch.empty((rk.pred_norm_rotate_workspace_bytes(p.handle, n, heads),), dtype=torch.uint8, device="cuda")
        got = []
        for _ in range(2):
            dx, dw = torch.empty_like(x), torch.empty((D,), device="cuda")
            rk.pred_norm_rotate_backward(p.handle, rk.Norm(w, 1e-6), rope, x, positions, dy, dx, dw, ws)
            got.append((dx, dw))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    x64, w64 = x.cpu().double().requires_grad_(), w.cpu().double().requires_grad_()
    y = x64 / (x64.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w64
    angle = (positions.cpu().double()[:, None] * torch.from_numpy(freq))[:, None]
    a, b = y.chunk(2, -1)
    d = dy.cpu().double()
    (torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1) * d).sum().backward()
    # |u|, |h|, |g| and r are under 16 here; the rotation's 2^-20 (|a| + |b|) is then the largest term by far
    err = (got[0][0].cpu().double() - x64.grad).abs()
    assert torch.all(err <= HALF_BF16 * x64.grad.abs() + 2.0 ** -20 * 16 * 4)
    err = (got[0][1].cpu().double() - w64.grad).abs()
    # N summands: each off by 2^-20 (|a| + |b|) |h|, of mean under 2 here, and the sum by N u of the summands' sizes
    N = n * heads
    assert torch.all(err <= N * (2.0 ** -20 * 2 + N * U))


STORES = [
    # n, Hq, Hk, D, B, rot, interleaved, kind, layout, fused
    (1, 4, 1, 64, 16, 64, False, "bf16", "tokens", True),
    (37, 8, 2, 64, 16, 32, True, "bf16", "heads", False),
    (37, 8, 2, 128, 16, 128, False, "fp8", "tokens", True),
    (130, 32, 8, 128, 32, 64, True, "fp4", "heads", True),
    (130, 32, 8, 128, 32, 64, False, "fp4", "tokens", True),
    (20, 5, 1, 80, 7, 20, False, "bf16", "padded", False),
    (20, 10, 2, 96, 1, 96, True, "fp8", "padded", False),
    (33, 3, 3, 96, 5, 22, False, "fp4", "padded", False),
    (65, 64, 8, 128, 8, 128, False, "fp4", "padded", True),
    (9, 4, 1, 64, 16, 64, False, "fp4", "heads", False),
    (9, 4, 2, 256, 16, 0, False, "fp4", "heads", False),
    (9, 4, 2, 32, 16, 32, False, "fp4", "tokens", False),
    (2300, 8, 2, 64, 16, 64, True, "fp4", "heads", True),
    (700, 40, 8, 128, 16, 128, False, "bf16", "tokens", True),
    (1100, 3, 3, 96, 5, 22, False, "fp8", "padded", False),
    (1100, 7, 7, 32, 16, 0, False, "fp4", "padded", True),
]


def _held(kind, N, B, Hk, D, layout):
    """(KVCache, the values of k and v as it holds them, a function)."""
    if kind == "fp4":
        k, v, ks, vs = cache4(N, B, Hk, D, layout)
        return rk.KVCache(k, v, 1.0, 1.0, ks, vs), lambda: (values4(k, ks), values4(v, vs))
    k, v = _cache_tensors(N, B, Hk, D, FP8 if kind == "fp8" else torch.bfloat16, layout, fill=3.0)
    scales = (0.0625, 0.37) if kind == "fp8" else (1.0, 1.0)
    return rk.KVCache(k, v, *scales), lambda: (_f64(k) * scales[0], _f64(v) * scales[1])


def _close4(got, want, slack, what):
    """What a 4-bit cache holds for values `want`, known to within `slack`: each of the values and scales that some
    value in that range would give.  Where no rounding is in doubt, exactly one."""
    codes, scales = cache.quantise(want)
    one = cache.dequantise(codes, scales)
    sure = got == one
    if sure.all():
        return
    # the same with every value at either end of its range, and the scale either end's largest gives
    flat, lo, g = np.abs(want).reshape(-1, 32), slack.reshape(-1, 32), np.abs(got).reshape(-1, 32)
    for i in np.unique(np.argwhere(~sure.reshape(-1, 32))[:, 0]):
        fits = False
        for top in (flat[i] - lo[i], flat[i] + lo[i]):
            _, sc = cache.quantise(np.full((1, 32), max(top.max(), 0.0)))
            e = 2.0 ** (float(sc[0, 0]) - 127)
            near = [np.abs(np.clip(flat[i] + d * lo[i], 0, None)[:, None] / e - cache.E2M1) for d in (-1, 0, 1)]
            allowed = np.any([n <= n.min(1, keepdims=True) + 1e-12 for n in near], 0)
            fits |= bool(np.all(np.any(allowed & (g[i][:, None] == e * cache.E2M1), 1)))
        assert fits, (what, i)


@pytest.mark.parametrize("norms", ["both", "k", "none"])
@pytest.mark.parametrize("n,Hq,Hk,D,B,rot,inter,kind,layout,fused", STORES)
def test_norm_rotate_store(n, Hq, Hk, D, B, rot, inter, kind, layout, fused, norms):
    _say("norm store", n, Hq, Hk, D, B, rot, inter, kind, layout, fused, norms)
    g = torch.Generator().manual_seed(n + D)
    N = n // B + 4
    rope, freq, _ = _rope(rot, 10000.0, interleaved=inter) if rot else (None, None, 1.0)
    kv, held = _held(kind, N, B, Hk, D, layout)
    qkv = torch.randn((n, Hq + 2 * Hk, D), generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = torch.randperm(N * B, generator=g)[:n]
    if n > 4:
        slots[1] = -1
    positions = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32).cuda()
    qw, kw = _weight(g, D, 0.0), _weight(g, D, 1.0)
    q_norm = rk.Norm(qw, 1e-6) if norms == "both" else None
    k_norm = rk.Norm(kw, 1e-3, 1.0) if norms != "none" else None
    with _handle(Hq, Hk, D, B, N) as p:
        q_out = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
        before = held()
        rk.pred_norm_rotate_store(p.handle, q_norm, k_norm, rope, q, k, v, positions if rot else None, slots.cuda(), kv,
                                  q_out)
        rk.pred_device_error(p.handle)
        pos = positions.cpu().numpy()

        def turned(x, norm, w, eps, offset):
            y = _f64(x) if norm is None else cache.norm(_f64(x), _f64(w), eps, offset)
            z = cache.rotate(y, pos, freq, 1.0, inter) if rot else y
            slack = (0 if norm is None else ulps(D)) * np.abs(y)
            if rot:
                slack = slack + (1 + ulps(D) * 2 ** 20) * _rotation_tolerance(y, z, rot, inter, 1.0)
            return z, slack

        want, slack = turned(q, q_norm, qw, 1e-6, 0.0)
        assert np.all(np.abs(_f64(q_out) - want) <= HALF_BF16 * np.abs(want) + slack)
        scales = (0.0625, 0.37) if kind == "fp8" else (1.0, 1.0)
        for got, old, (want, slack), scale in zip(held(), before, (turned(k, k_norm, kw, 1e-3, 1.0), (_f64(v), 0 * _f64(v))),
                                                  scales):
            got, old = got.reshape(N * B, Hk, D), old.reshape(N * B, Hk, D)
            if kind == "fp8":
                tol = 2.0 ** -4 * np.abs(want) + scale * 2.0 ** -10 + slack + 2.0 ** -22 * np.abs(want)
            else:
                tol = HALF_BF16 * np.abs(want) + slack
            hit = np.zeros(N * B, bool)
            for t, slot in enumerate(slots.tolist()):
                if slot < 0:
                    continue
                hit[slot] = True
                if kind == "fp4":       # rounded to bf16 before
                    _close4(got[slot], want[t], HALF_BF16 * np.abs(want[t]) * bool(slack.any()) + slack[t], (t, slot))
                else:
                    assert np.all(np.abs(got[slot] - want[t]) <= tol[t]), (t, slot)
            assert np.array_equal(got[~hit], old[~hit])
        # the same in steps: normed, turned, then stored
        if norms == "both" and kind == "fp4":
            kv2, held2 = _held(kind, N, B, Hk, D, layout)
            kk = torch.empty((n, Hk, D), dtype=torch.bfloat16, device="cuda")
            rk.pred_norm_rotate(p.handle, k_norm, rope, k, positions if rot else None, kk)
            rk.pred_store(p.handle, kk, v, slots.cuda(), kv2)
            for a, b in zip(held(), held2()):
                assert np.array_equal(a, b)
        if not fused:       # in place
            rk.pred_norm_rotate_store(p.handle, q_norm, k_norm, rope, q, k, v, positions if rot else None, slots.cuda(), kv, q)
            assert torch.equal(q, q_out)


@pytest.mark.parametrize("D,rot,inter,layout", [(128, 128, False, "heads"), (64, 20, False, "tokens"), (96, 96, True, "padded")])
def test_rotate_store_into_4_bits(D, rot, inter, layout):
    """pred_rotate_store takes a 4-bit cache: queries within a rotation's rounding of pred_rotate's, keys as turned."""
    n, Hq, Hk, B, N = 21, 6, 2, 8, 5
    g = torch.Generator().manual_seed(D)
    rope, freq, _ = _rope(rot, interleaved=inter)
    kv, held = _held("fp4", N, B, Hk, D, layout)
    q, k, v = (torch.randn((n, h, D), generator=g).bfloat16().cuda() for h in (Hq, Hk, Hk))
    slots = torch.randperm(N * B, generator=g)[:n]
    positions = torch.randint(0, 9999, (n,), generator=g, dtype=torch.int32).cuda()
    with _handle(Hq, Hk, D, B, N) as p:
        q_out = torch.empty_like(q)
        rk.pred_rotate_store(p.handle, rope, q, k, v, positions, slots.cuda(), kv, q_out)
        want = cache.rotate(_f64(q), positions.cpu().numpy(), freq, 1.0, inter)
        assert np.all(np.abs(_f64(q_out) - want) <= HALF_BF16 * np.abs(want) + _rotation_tolerance(_f64(q), want, rot, inter, 1.0))
        want = cache.rotate(_f64(k), positions.cpu().numpy(), freq, 1.0, inter)
        slack = HALF_BF16 * np.abs(want) + _rotation_tolerance(_f64(k), want, rot, inter, 1.0)
        got_k, got_v = (x.reshape(N * B, Hk, D)[slots.numpy()] for x in held())
        for t in range(n):
            _close4(got_k[t], want[t], slack[t], t)
        assert np.array_equal(got_v, cache.dequantise(*cache.quantise(_f64(v))))


@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
@pytest.mark.parametrize("n,Hk,D,B", [(1, 1, 64, 16), (50, 8, 128, 16), (33, 3, 96, 7), (20, 2, 32, 1), (9, 1, 512, 8), (9, 40, 64, 8),
                                       (2100, 3, 64, 16), (2050, 2, 128, 16)])
def test_store_and_load_4_bits(n, Hk, D, B, layout):
    """Bit for bit: values of every size, ties, zeros of both signs, groups that are all zero, tiny or not finite."""
    _say("store 4", n, Hk, D, B, layout)
    g = torch.Generator().manual_seed(n + D)
    N = n // B + 3
    x = torch.randn((2, n, Hk, D), generator=g) * torch.exp2(torch.randint(-30, 30, (2, n, Hk, 1), generator=g).float())
    grid = torch.tensor([0, 0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.0, -0.25, -5, -6, 6.03125, 4])
    x[0, 0, 0, :16], x[1, 0, 0, :16] = grid, -grid * 4096
    x[0, -1, -1], x[1, -1, -1] = 0.0, -0.0
    if n > 4:
        x[0, 2, 0, :32] = 2.0 ** -126 * grid.repeat(2)
        x[0, 3, 0, 31], x[1, 3, 0, 7], x[1, 4, 0, 3] = float("nan"), float("inf"), -float("inf")
        x[0, 4, 0, :32] = 3.3e38
    x = x.bfloat16().cuda()
    slots = torch.randperm(N * B, generator=g)[:n]
    k, v, ks, vs = cache4(N, B, Hk, D, layout)
    kv = rk.KVCache(k, v, 1.0, 1.0, ks, vs)
    with _handle(2 * Hk, Hk, D, B, N) as p:
        old = [t.clone() for t in (k, v, ks, vs)]
        rk.pred_store(p.handle, x[0], x[1], slots.cuda(), kv)
        back = torch.full_like(x, 7.0)
        rk.pred_load(p.handle, kv, slots.cuda(), back[0], back[1])
        rk.pred_device_error(p.handle)
        untouched = torch.ones((N * B,), dtype=torch.bool)
        untouched[slots] = False
        for bits, scales, old_bits, old_scales, want, got in ((k, ks, old[0], old[2], x[0], back[0]),
                                                              (v, vs, old[1], old[3], x[1], back[1])):
            codes, sc = cache.quantise(_f64(want))
            got_codes = cache.unpacked(bits.cpu().numpy()).reshape(N * B, Hk, D)[slots.numpy()]
            got_sc = scales.cpu().numpy().reshape(N * B, Hk, D // 32)[slots.numpy()]
            assert np.array_equal(got_sc, sc)
            assert np.array_equal(np.where(np.repeat(sc == 255, 32, -1), 0, codes), got_codes)
            assert np.array_equal(_f64(got), cache.dequantise(codes, sc), equal_nan=True)
            for a, b in ((bits, old_bits), (scales, old_scales)):
                a, b = (t.cpu().reshape(N * B, Hk, -1)[untouched] for t in (a, b))
                assert torch.equal(a, b)
        # a padding token and bad slots: their rows stay
        bad = slots.clone()
        bad[0] = -1
        back.fill_(7.0)
        rk.pred_load(p.handle, kv, bad.cuda(), back[0], back[1])
        rk.pred_device_error(p.handle)
        assert torch.all(back[:, 0] == 7)
        for slot in (N * B, -2, 2 ** 40, -2 ** 40):
            bad[0] = slot
            rk.pred_load(p.handle, kv, bad.cuda(), back[0], back[1])
            with pytest.raises(rk.PredError) as e:
                rk.pred_device_error(p.handle)
            assert "slot" in str(e.value) and torch.all(back[:, 0] == 7)
            rk.pred_store(p.handle, x[0][:1], x[1][:1], bad[:1].cuda(), kv)
            with pytest.raises(rk.PredError):
                rk.pred_device_error(p.handle)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("n,Hk,D,B,layout", [(1, 1, 64, 16, "tokens"), (45, 8, 128, 16, "heads"), (45, 3, 80, 7, "padded"),
                                              (2077, 5, 64, 16, "heads")])
def test_store_and_load(n, Hk, D, B, layout, dtype):
    g = torch.Generator().manual_seed(n + D)
    N = n // B + 3
    x = torch.randn((2, n, Hk, D), generator=g).bfloat16().cuda()
    slots = torch.randperm(N * B, generator=g)[:n]
    k, v = _cache_tensors(N, B, Hk, D, dtype, layout, fill=3.0)
    scales = (0.0625, 0.37) if dtype == FP8 else (1.0, 1.0)
    kv = rk.KVCache(k, v, *scales)
    with _handle(2 * Hk, Hk, D, B, N) as p:
        rk.pred_store(p.handle, x[0], x[1], slots.cuda(), kv)
        back = torch.full_like(x, 7.0)
        rk.pred_load(p.handle, kv, slots.cuda(), back[0], back[1])
        rk.pred_device_error(p.handle)
        if dtype == torch.bfloat16:
            assert torch.equal(back, x)
        for got, held, want, scale in ((back[0], k, x[0], scales[0]), (back[1], v, x[1], scales[1])):
            at = torch.from_numpy(_f64(held).reshape(N * B, Hk, D))[slots].numpy() * scale
            assert np.all(np.abs(_f64(got) - at) <= HALF_BF16 * np.abs(at))
            if dtype == FP8:
                w = _f64(want)
                assert np.all(np.abs(at - w) <= 2.0 ** -4 * np.abs(w) + scale * 2.0 ** -10 + 2.0 ** -22 * np.abs(w))


def test_gradient_and_stores_in_graphs():
    """A step (norm, rotation, store, read back) and a gradient, captured with workspaces of their own, replayed with
    eager work between."""
    n, Hq, Hk, D, B, N = 40, 8, 2, 128, 16, 6
    g = torch.Generator().manual_seed(1)
    rope, _, _ = _rope(128)
    q, k, v = (torch.randn((n, h, D), generator=g).bfloat16().cuda() for h in (Hq, Hk, Hk))
    dy = torch.randn((n, Hq, D), generator=g).bfloat16().cuda()
    slots = torch.randperm(N * B, generator=g)[:n].cuda()
    positions = torch.arange(n, dtype=torch.int32).cuda()
    w = torch.randn((D,), generator=g).bfloat16().cuda()
    norm = rk.Norm(w, 1e-6)
    kv, held = _held("fp4", N, B, Hk, D, "heads")
    with _handle(Hq, Hk, D, B, N) as p:
        ws = [torch.empty((rk.pred_norm_rotate_workspace_bytes(p.handle, n, Hq),), dtype=torch.uint8, device="cuda")
              for _ in range(2)]
        q_out, back, dx, dw = torch.empty_like(q), [torch.empty_like(k), torch.empty_like(v)], torch.empty_like(q), torch.empty((D,), device="cuda")

        def step(ws):
            rk.pred_norm_rotate_store(p.handle, norm, norm, rope, q, k, v, positions, slots, kv, q_out)
            rk.pred_load(p.handle, kv, slots, *back)
            rk.pred_norm_rotate_backward(p.handle, norm, rope, q, positions, dy, dx, dw, ws)

        step(ws[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(ws[0])
        for i in range(4):
            for t in (q, k, v, dy):
                t.copy_(torch.randn(t.shape, generator=g))
            step(ws[1])
            want = [t.clone() for t in (q_out, *back, dx, dw)]
            for t in (q_out, *back, dx, dw):
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((q_out, *back, dx, dw), want):
                assert torch.equal(a, b), i


def test_other_stream_and_nothing_to_do():
    D, B, Hk, N = 64, 16, 2, 8
    z = dict(device="cuda")
    with _handle(4, Hk, D, B, N) as p:
        h = p.handle
        kv, held = _held("fp4", N, B, Hk, D, "tokens")
        before = held()
        x0, k0 = torch.zeros((0, 4, D), dtype=torch.bfloat16, **z), torch.zeros((0, Hk, D), dtype=torch.bfloat16, **z)
        none32, none64 = torch.zeros((0,), dtype=torch.int32, **z), torch.zeros((0,), dtype=torch.int64, **z)
        norm = rk.Norm(None, 1e-6)
        dw = torch.full((D,), 5.0, **z)
        rk.pred_norm_rotate(h, norm, None, x0, None, x0)
        rk.pred_norm_rotate_backward(h, norm, None, x0, None, x0, x0, dw)
        assert torch.all(dw == 0)
        rk.pred_norm_rotate_store(h, norm, norm, None, x0, k0, k0, none32, none64, kv, x0)
        rk.pred_store(h, k0, k0, none64, kv)
        rk.pred_load(h, kv, none64, k0, k0)
        assert rk.pred_norm_rotate_workspace_bytes(h, 0, 4) == 0
        for a, b in zip(before, held()):
            assert np.array_equal(a, b)
        x = torch.randn((5, 4, D), **z).bfloat16()
        want, out = torch.empty_like(x), torch.zeros_like(x)
        rk.pred_norm_rotate(h, norm, None, x, None, want)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        rk.pred_norm_rotate(h, norm, None, x, None, out, stream=s)
        s.synchronize()
        assert torch.equal(out, want)


def test_as_many_tokens_as_a_launch_has_waves():
    """A wave a token: 2^26 - 32 of them run, one more is refused and nothing is written."""
    n = 2 ** 26 - 32
    x = torch.ones((n + 1, 1, 8), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 9.0)
    slots = torch.zeros((n + 1,), dtype=torch.int64, device="cuda")
    k, v = (torch.full((1, 1, 1, 8), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with _handle(1, 1, 8, 1, 1) as p:
        norm, kv = rk.Norm(None, 1e-6), rk.KVCache(k, v)
        for call in (lambda n: rk.pred_norm_rotate(p.handle, norm, None, x[:n], None, out[:n]),
                     lambda n: rk.pred_load(p.handle, kv, slots[:n], out[:n], x[:n])):
            out.fill_(9.0)
            with pytest.raises(rk.PredError):
                call(n + 1)
            assert torch.all(out == 9.0) and torch.all(x == 1.0)
            call(n)
            rk.pred_device_error(p.handle)
            assert torch.all(out[n:] == 9.0) and (out[:n] - out[0]).abs().max() == 0 and out[0, 0, 0] in (1.0, 3.0)


def test_refusals():
    D, B, Hk, N = 64, 16, 2, 8
    z = dict(device="cuda")
    with _handle(4, Hk, D, B, N) as p:
        h = p.handle
        kv, _ = _held("fp4", N, B, Hk, D, "tokens")
        rope, _, _ = _rope(64)
        back, _, _ = _rope(64, backward=True)
        wide, _, _ = _rope(128)
        w = torch.ones((D,), dtype=torch.bfloat16, **z)
        norm = rk.Norm(w, 1e-6)
        x, k = torch.zeros((3, 4, D), dtype=torch.bfloat16, **z), torch.zeros((3, Hk, D), dtype=torch.bfloat16, **z)
        pos, slots = torch.zeros((3,), dtype=torch.int32, **z), torch.full((3,), -1, dtype=torch.int64, **z)
        dw = torch.zeros((D,), **z)
        ws = torch.empty((rk.pred_norm_rotate_workspace_bytes(h, 3, 4) + 16,), dtype=torch.uint8, **z)
        rk.pred_norm_rotate(h, norm, rope, x, pos, x)
        for args, err in (((norm, rope, x[..., :32], pos, x), ValueError), ((norm, rope, x, pos.long(), x), TypeError),
                          ((norm, rope, x, pos[:2], x), ValueError), ((norm, rope, x.transpose(0, 1), pos, x), ValueError),
                          ((norm, rope, x, pos, x.cpu()), ValueError), ((norm, rope, x, None, x), rk.PredError),
                          ((norm, back, x, pos, x), rk.PredError), ((norm, wide, x, pos, x), rk.PredError),
                          ((rk.Norm(w[:32].clone(), 1e-6), rope, x, pos, x), ValueError),
                          ((rk.Norm(w, 0.0), rope, x, pos, x), rk.PredError), ((rk.Norm(w, -1.0), rope, x, pos, x), rk.PredError),
                          ((rk.Norm(w, math.nan), rope, x, pos, x), rk.PredError),
                          ((rk.Norm(w, 1e-6, math.inf), rope, x, pos, x), rk.PredError)):
            with pytest.raises(err):
                rk.pred_norm_rotate(h, *args)
        for args in ((w.float(), 1e-6), (w.cpu(), 1e-6), ([1.0], 1e-6)):
            with pytest.raises(TypeError):
                rk.Norm(*args)
        with pytest.raises(ValueError):
            rk.Norm(torch.ones((2 * D,), dtype=torch.bfloat16, **z)[::2], 1e-6)
        off = torch.ones((D + 1,), dtype=torch.bfloat16, **z)[1:]
        with pytest.raises(rk.PredError) as e:
            rk.pred_norm_rotate(h, rk.Norm(off, 1e-6), rope, x, pos, x)
        assert e.value.code == rk.PRED_ERR_UNSUPPORTED
        with pytest.raises(rk.PredError) as e:
            rk.cache._check(rk.lib().pred_norm_rotate(h, None, None, x.data_ptr(), 4 * D, 3, 4, None, x.data_ptr(), 4 * D, None))
        assert e.value.code == rk.PRED_ERR_NULL_ARG
        # the gradient
        rk.pred_norm_rotate_backward(h, norm, rope, x, pos, x, torch.empty_like(x), dw, ws)
        for w_, err in ((None, rk.PRED_ERR_WORKSPACE), (ws[:16], rk.PRED_ERR_WORKSPACE), (ws[1:], rk.PRED_ERR_WORKSPACE)):
            with pytest.raises(rk.PredError) as e:
                rk.pred_norm_rotate_backward(h, norm, rope, x, pos, x, torch.empty_like(x), dw, w_)
            assert e.value.code == err
        for kw, err in ((dict(dy=x[:2]), ValueError), (dict(dx=x.float()), TypeError), (dict(dweight=dw[:32]), ValueError),
                        (dict(dweight=dw.double()), TypeError), (dict(positions=None), rk.PredError)):
            a = dict(x=x, positions=pos, dy=x, dx=torch.empty_like(x), dweight=dw, workspace=ws)
            a.update(kw)
            with pytest.raises(err):
                rk.pred_norm_rotate_backward(h, norm, rope, **a)
        apart = torch.zeros((3, 6, D), dtype=torch.bfloat16, **z)
        with pytest.raises(rk.PredError) as e:      # in place with another stride
            rk.cache._check(rk.lib().pred_norm_rotate_backward(h, norm._ref, None, x.data_ptr(), 4 * D, 3, 4, None, apart.data_ptr(),
                                                               6 * D, apart.data_ptr(), 4 * D, None, None, 0, None))
        assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE
        # stores and loads
        rk.pred_norm_rotate_store(h, norm, norm, rope, x, k, k, pos, slots, kv, x)
        with pytest.raises(rk.PredError):
            rk.pred_norm_rotate_store(h, norm, norm, back, x, k, k, pos, slots, kv, x)
        with pytest.raises(rk.PredError):
            rk.pred_norm_rotate_store(h, norm, norm, rope, x, k, k, None, slots, kv, x)
        with pytest.raises(ValueError):
            rk.pred_store(h, k, k[:2], slots, kv)
        with pytest.raises(TypeError):
            rk.pred_store(h, k.float(), k, slots, kv)
        with pytest.raises(TypeError):
            rk.pred_load(h, kv, slots.int(), k, k)
        with pytest.raises(ValueError):
            rk.pred_load(h, kv, slots, k, k[:, :, :32])
        with pytest.raises(rk.PredError):
            rk.pred_load(h, kv, slots, None, k)
        # 4-bit caches
        kb, vb, ks, vs = cache4(N, B, Hk, D, "tokens")
        for args, err in (((kb, vb, 1.0, 1.0, ks, None), ValueError), ((kb, vb, 1.0, 1.0, ks[..., :1], vs[..., :1]), ValueError),
                          ((kb.view(FP8), vb.view(FP8), 1.0, 1.0, ks, vs), TypeError),
                          ((kb, vb, 1.0, 1.0, ks.int(), vs.int()), TypeError), ((kb, vb, 1.0, 1.0, ks.cpu(), vs), ValueError),
                          ((kb, vb, 1.0, 1.0, cache4(N, B, Hk, D, "heads")[2], vs), ValueError)):
            with pytest.raises(err):
                rk.KVCache(*args)
        for bad in (rk.KVCache(kb, vb, 2.0, 1.0, ks, vs), rk.KVCache(kb, kb, 1.0, 1.0, ks, vs), rk.KVCache(kb, vb, 1.0, 1.0, ks, ks)):
            with pytest.raises(rk.PredError):
                rk.pred_store(h, k, k, slots, bad)
        short = rk.KVCache(kb, vb, 1.0, 1.0, ks, vs)
        short._struct.k_scales = None
        with pytest.raises(rk.PredError) as e:
            rk.pred_load(h, short, slots, k, torch.empty_like(k))
        assert e.value.code == rk.PRED_ERR_NULL_ARG
        odd = rk.KVCache(kb, vb, 1.0, 1.0, ks, vs)
        odd._struct.head_stride += 16
        with pytest.raises(rk.PredError) as e:
            rk.pred_load(h, odd, slots, k, torch.empty_like(k))
        assert e.value.code == rk.PRED_ERR_UNSUPPORTED
        rk.pred_device_error(h)
    with _handle(2, 1, 520, 16, 2) as p:
        x = torch.zeros((1, 2, 520), dtype=torch.bfloat16, **z)
        with pytest.raises(rk.PredError) as e:
            rk.pred_norm_rotate(p.handle, rk.Norm(None, 1e-6), None, x, None, x)
        assert e.value.code == rk.PRED_ERR_UNSUPPORTED
    with _handle(2, 1, 48, 16, 2) as p:     # no whole groups of 32
        x = torch.zeros((1, 1, 48), dtype=torch.bfloat16, **z)
        kv = rk._lib.PredKvCache(1 << 20, 1 << 21, 16 * 64, 64, 64, rk.PRED_KV_FP4, 1.0, 1.0, 1 << 22, 1 << 23)
        import ctypes
        rc = rk.lib().pred_store(p.handle, x.data_ptr(), 48, x.data_ptr(), 48, 1, torch.zeros((1,), dtype=torch.int64, **z).data_ptr(),
                                 ctypes.byref(kv), None)
        assert rc == rk.PRED_ERR_UNSUPPORTED
