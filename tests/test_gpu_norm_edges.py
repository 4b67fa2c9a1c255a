"""GPU tests of the edges of the cache's stores and read back: tokens too wide to count."""

import ctypes

import pytest

import rank_kv_block_amd as rk
from tests.test_gpu_cache import _handle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


def test_load_refuses_tokens_too_wide_to_count():
    """2^31 values of a token: refused by the dims, so the addresses are never read."""
    Hk, D = 1 << 15, 1 << 16
    with _handle(Hk, Hk, D, 1, 1) as p:
        kv = rk._lib.PredKvCache(1 << 20, 1 << 21, Hk * D, Hk * D, D, rk.PRED_KV_BF16, 1.0, 1.0, None, None)
        slots = torch.full((1,), -1, dtype=torch.int64, device="cuda")
        rc = rk.lib().pred_load(p.handle, ctypes.byref(kv), 1, slots.data_ptr(), 1 << 22, 1 << 40, None)
        assert rc == rk.PRED_ERR_UNSUPPORTED, rk.pred_last_error()
        rk.pred_device_error(p.handle)
