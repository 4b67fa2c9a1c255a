"""GPU tests of the edges of the cache's stores and read back: outputs that overlap, tokens too wide to count,
signs of what a 4-bit cache holds.  Tolerances: those of tests/test_gpu_norm.py."""

import ctypes

import numpy as np
import pytest

import rank_kv_block_amd as rk
from oracle import cache
from tests.close4 import close4
from tests.test_gpu_cache import HALF_BF16, _f64, _handle, _rope, _rotation_tolerance
from tests.test_gpu_norm import STORES, _held, _weight, ulps

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_load_refuses_outputs_that_overlap(kind):
    n, Hk, D, B, N = 5, 2, 64, 16, 3
    kv, _ = _held(kind, N, B, Hk, D, "tokens")
    both = torch.full((2 * n, Hk, D), 9.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(n, device="cuda")
    with _handle(4, Hk, D, B, N) as p:
        for at in (0, 1, n - 1):
            for k, v in ((both[:n], both[at:at + n]), (both[at:at + n], both[:n])):
                with pytest.raises(rk.PredError) as e:
                    rk.pred_load(p.handle, kv, slots, k, v)
                assert e.value.code == rk.PRED_ERR_OUT_OF_RANGE and torch.all(both == 9.0)
        apart = torch.empty_like(both)
        for k, v in ((both[:n], both[n:]), (both[n:], both[:n])):       # side by side
            rk.pred_load(p.handle, kv, slots, k, v)
            rk.pred_load(p.handle, kv, slots, apart[:n], apart[n:])
            assert torch.equal(k, apart[:n]) and torch.equal(v, apart[n:])
        rk.pred_load(p.handle, kv, slots[:0], both[:0], both[:0])
        rk.pred_device_error(p.handle)


def test_load_refuses_tokens_too_wide_to_count():
    """2^31 values of a token: refused by the dims, so the addresses are never read."""
    Hk, D = 1 << 15, 1 << 16
    with _handle(Hk, Hk, D, 1, 1) as p:
        kv = rk._lib.PredKvCache(1 << 20, 1 << 21, Hk * D, Hk * D, D, rk.PRED_KV_BF16, 1.0, 1.0, None, None)
        slots = torch.full((1,), -1, dtype=torch.int64, device="cuda")
        rc = rk.lib().pred_load(p.handle, ctypes.byref(kv), 1, slots.data_ptr(), 1 << 22, 1 << 40, None)
        assert rc == rk.PRED_ERR_UNSUPPORTED, rk.pred_last_error()
        rk.pred_device_error(p.handle)


@pytest.mark.parametrize("norms", ["k", "none"])
@pytest.mark.parametrize("n,Hq,Hk,D,B,rot,inter,kind,layout,fused", [c for c in STORES if c[7] == "fp4" and c[5]])
def test_signs_of_stored_keys(n, Hq, Hk, D, B, rot, inter, kind, layout, fused, norms):
    """Keys normed and turned, or turned alone, into a 4-bit cache: within the roundings of the oracle's, signs included;
    with a norm bit for bit those stored after the steps; without one those of pred_rotate_store."""
    g = torch.Generator().manual_seed(n + D + 1)
    N = n // B + 4
    rope, freq, _ = _rope(rot, 10000.0, interleaved=inter)
    (kv, held), (other, other_held) = (_held(kind, N, B, Hk, D, layout) for _ in range(2))
    q, k, v = (torch.randn((n, h, D), generator=g).bfloat16().cuda() for h in (Hq, Hk, Hk))
    slots = torch.randperm(N * B, generator=g)[:n]
    positions = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32).cuda()
    w = _weight(g, D, 1.0)
    norm = rk.Norm(w, 1e-3, 1.0) if norms == "k" else None
    with _handle(Hq, Hk, D, B, N) as p:
        q_out = torch.empty_like(q)
        rk.pred_norm_rotate_store(p.handle, None, norm, rope, q, k, v, positions, slots.cuda(), kv, q_out)
        if norm:
            turned = torch.empty_like(k)
            rk.pred_norm_rotate(p.handle, norm, rope, k, positions, turned)
            rk.pred_store(p.handle, turned, v, slots.cuda(), other)
        else:
            rk.pred_rotate_store(p.handle, rope, q, k, v, positions, slots.cuda(), other, q_out)
        rk.pred_device_error(p.handle)
        for a, b in zip(held(), other_held()):
            assert np.array_equal(a, b)
        y = cache.norm(_f64(k), _f64(w), 1e-3, 1.0) if norm else _f64(k)
        want = cache.rotate(y, positions.cpu().numpy(), freq, 1.0, inter)
        slack = (ulps(D) if norm else 0) * np.abs(y) + (1 + ulps(D) * 2 ** 20) * _rotation_tolerance(y, want, rot, inter, 1.0)
        got_k, got_v = (x.reshape(N * B, Hk, D)[slots.numpy()] for x in held())
        for t in range(n):
            close4(got_k[t], want[t], HALF_BF16 * np.abs(want[t]) + slack[t], t)
        assert np.array_equal(got_v, cache.dequantise(*cache.quantise(_f64(v))))
