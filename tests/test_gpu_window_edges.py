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


def _time(f, calls=10):
    """us a call, the best of three."""
    best = float("inf")
    for _ in range(3):
        f()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(calls):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best


def test_few_live_rows_of_many():
    """A captured step of 2048 rows whose last chunk has 16 of them, on a long context: the work is split as it is for a call
    of 16 rows, which takes a thirtieth of one group's whole walk (3281 and 120 us when walks were left whole by n_rows); a
    call in which all rows live keeps its walks whole.  Each against the oracle."""
    Hq, Hk, D, B, n = 32, 8, 128, 16, 8192
    few = make("bf16", 1, 16, Hq, Hk, D, B, n, lens=[n * B - 5], drafts=[16])
    with _handle(Hq, Hk, D, B, few.N) as p:
        few.run(p, ALL, 0)
        q = torch.zeros((1, 2048, Hq, D), dtype=torch.bfloat16, device="cuda")
        q[:, :16] = few.q
        q[:, 16:] = float("nan")
        out, lse = torch.full_like(q, 9.0), torch.full((1, 2048, Hq), 9.0, device="cuda")

        def call(M, q, out, lse, ws):
            rk.pred_attend_window(p.handle, few.kv, q, few.tables, few.lens, few.drafts, ALL, 0, few.scale, out, lse, ws)

        ws = [torch.empty((max(1, rk.pred_attend_window_workspace_bytes(p.handle, 1, M, n, ALL, 0)),), dtype=torch.uint8, device="cuda")
              for M in (16, 2048)]
        call(2048, q, out, lse, ws[1])
        rk.pred_device_error(p.handle)
        few.check(p, ALL, 0)
        few.out.copy_(out[:, :16])
        few.lse.copy_(lse[:, :16])
        few.check(p, ALL, 0)
        assert torch.all(out[:, 16:] == 0) and torch.all(torch.isneginf(lse[:, 16:]))
        alone = _time(lambda: call(16, few.q, few.out, few.lse, ws[0]))
        among = _time(lambda: call(2048, q, out, lse, ws[1]))
        print("16 rows", alone, "us, 16 of 2048", among, "us", flush=True)
        assert among < 4 * alone


@pytest.mark.parametrize("live", [1, 20, 33, 300, 1400, 1535, 1536, 1600, 2048])
def test_rows_of_one_long_sequence(live):
    """Live rows to either side of where the walks of one long sequence stay whole (384 groups of 512 places: 1536 rows)."""
    Hq, Hk, D, B, n, M = 8, 8, 64, 16, 520, 2048 * 4
    live *= 4
    c = make("bf16", 1, M, Hq, Hk, D, B, n + 100, lens=[n * B + (live > n * B) * 100], drafts=[live])
    with _handle(Hq, Hk, D, B, c.N) as p:
        need = rk.pred_attend_window_workspace_bytes(p.handle, 1, M, c.n, ALL, 0)
        assert 0 < need < 100 << 20
        c.run(p, ALL, 0)
        rk.pred_device_error(p.handle)
        c.check(p, ALL, 0)


def test_no_live_row_of_many():
    """A step made for many rows of one long sequence in which it has none, then some: the join finds what this call left."""
    Hq, Hk, D, B, n, M = 8, 8, 64, 16, 620, 2048 * 4
    c = make("bf16", 1, M, Hq, Hk, D, B, n, lens=[n * B - 7], drafts=[0])
    with _handle(Hq, Hk, D, B, c.N) as p:
        ws = torch.full((rk.pred_attend_window_workspace_bytes(p.handle, 1, M, n, ALL, 0),), 0x7F, dtype=torch.uint8, device="cuda")
        for live in (0, 40, M, 0, 200):
            c.drafts.fill_(live)
            c.out.fill_(9.0)
            c.lse.fill_(9.0)
            rk.pred_attend_window(p.handle, c.kv, c.q, c.tables, c.lens, c.drafts, ALL, 0, c.scale, c.out, c.lse, ws)
            rk.pred_device_error(p.handle)
            c.check(p, ALL, 0)


def test_workspace_of_long_prompts():
    """The partial results of one sequence are those of calls that can be split: no more for 2^20 rows than for 2^13."""
    with _handle(32, 8, 128, 16, 4) as p:
        sizes = [rk.pred_attend_window_workspace_bytes(p.handle, 1, M, 1 << 21, ALL, 0) for M in (1 << 11, 1 << 13, 1 << 20)]
        assert 0 < sizes[0] <= sizes[1] == sizes[2] < 100 << 20
