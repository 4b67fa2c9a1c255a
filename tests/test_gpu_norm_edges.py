"""GPU tests of the edges of the cache's stores and read back: outputs that overlap, tokens too wide to count."""

import ctypes

import pytest

import rank_kv_block_amd as rk
from tests.test_gpu_cache import _handle
from tests.test_gpu_norm import _held

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
