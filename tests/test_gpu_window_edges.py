"""GPU tests of windowed attention where its kernels, its tables and its plans meet: sequences without a row, the bits of a
weight, few live rows of many.  Tolerances: those of tests/test_gpu_window.py."""

import pytest

import rank_kv_block_amd as rk
from tests.test_gpu_cache import _handle, _say
from tests.test_gpu_window import ALL, make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rk.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("Hq,Hk,D,B,kind,name", [(6, 2, 80, 16, "bf16", "plain"), (4, 2, 96, 16, "fp4", "plain"),
                                                 (2, 1, 256, 7, "fp8", "plain"), (8, 2, 128, 16, "bf16", "stream"),
                                                 (4, 1, 64, 16, "fp4", "chunk")])
def test_a_sequence_without_a_row_needs_no_entries(Hq, Hk, D, B, kind, name, M):
    """Sequences that hold tokens but have no row in this call, their blocks given back: zeros, -inf and no error, beside
    one that has rows."""
    n, S = 12, 3
    c = make(kind, S, M, Hq, Hk, D, B, n, lens=[n * B - 3, n * B, 5], drafts=[0, min(M, n * B), 0])
    with _handle(Hq, Hk, D, B, c.N) as p:
        assert rk.pred_attend_window_kernel_name(p.handle, c.kv, M) == f"attend_{name if M == 1 or name == 'plain' else 'chunk'}_kernel"
        for bad in (-1, c.N, 2 ** 31 - 1):
            c.tables[0], c.tables[2] = bad, bad
            for window, sinks in ((30, 4), (ALL, 0), (1, 0)):
                c.run(p, window, sinks)
                rk.pred_device_error(p.handle)
                for s in (0, 2):
                    assert torch.all(c.out[s] == 0) and torch.all(torch.isneginf(c.lse[s]))
                c.check(p, window, sinks)


@pytest.mark.parametrize("S,M,Hq,Hk,D,B,n,kind,layout,window,sinks", [
    (2, 1, 8, 2, 64, 16, 40, "fp4", "heads", 100, 4), (3, 1, 16, 1, 64, 32, 30, "fp4", "tokens", ALL, 0),
    (2, 4, 8, 2, 64, 16, 200, "fp4", "padded", 1500, 4), (2, 3, 8, 2, 128, 7, 99, "fp8", "padded", 100, 9),
    (2, 2, 8, 1, 128, 1, 400, "bf16", "tokens", 300, 4), (1, 1, 32, 8, 128, 8, 300, "fp4", "heads", ALL, 0),
    (2, 16, 3, 3, 128, 12, 80, "fp8", "heads", 500, 4)])
def test_two_terms_a_weight_up_to_16_queries(monkeypatch, S, M, Hq, Hk, D, B, n, kind, layout, window, sinks):
    """Up to 16 queries per kv head a weight keeps 16 bits whichever kernel the cache's layout takes them to: the bounds are
    those of the stream kernel (check() asks for the kernel's name to know them)."""
    _say("window two terms", S, M, Hq, Hk, D, B, n, kind, layout, window, sinks)
    c = make(kind, S, M, Hq, Hk, D, B, n, layout)
    with _handle(Hq, Hk, D, B, c.N) as p:
        assert rk.pred_attend_window_kernel_name(p.handle, c.kv, M) == "attend_chunk_kernel"
        c.run(p, window, sinks)
        rk.pred_device_error(p.handle)
        monkeypatch.setattr(rk, "pred_attend_window_kernel_name", lambda *a: "attend_stream_kernel")
        c.check(p, window, sinks)
