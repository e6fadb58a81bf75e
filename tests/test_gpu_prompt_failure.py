"""Failure detection of the prompt operators, made on the host: a workspace whose words are preset so that a wait
runs out or a meeting finds words that no call left. No kernel faults; each call returns, reports and stays in its
buffers."""

import time

import pytest
import torch

from synth import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SYNC = 64  # byte of the arrival word in moe_route's workspace, the count of CTAs past the wait behind it


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _preset(ws, word):
    ws.buf[SYNC:SYNC + 4].view(torch.int32).fill_(word)


def test_route_wait_that_runs_out(fme, monkeypatch):
    T, E, k = 3000, 64, 4
    logits, bias = torch.randn(T, E, device=DEV), torch.zeros(E, device=DEV)
    want = fme.moe_route(logits, bias, k)
    ws = fme.Workspace(fme.moe_route_workspace(T, E, k), DEV)
    monkeypatch.setenv("FME_WAIT_TIMEOUT_MS", "20")
    _preset(ws, -1)  # the count of arrivals ends one short
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    got = fme.moe_route(logits, bias, k, workspace=ws)
    assert ws.error() == 2 and time.perf_counter() - t0 < 2.0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not got[2].any()  # groups without rows
    assert ws.error() == 0  # read and cleared, but the workspace is not clean:
    for _ in range(3):
        got = fme.moe_route(logits, bias, k, workspace=ws)
        assert ws.error() == 2 and not got[2].any()
    ws.clear()
    got = fme.moe_route(logits, bias, k, workspace=ws)
    assert ws.error() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("preset", [1, 5, 100, 151, 152, 153, 1 << 20])
def test_route_stale_words_write_nothing_outside(fme, monkeypatch, preset):
    """Arrivals that no call left, and counts far above the routes there are."""
    T, E, k = 3000, 64, 4
    logits, bias = torch.randn(T, E, device=DEV), torch.zeros(E, device=DEV)
    ws = fme.Workspace(fme.moe_route_workspace(T, E, k), DEV)
    monkeypatch.setenv("FME_WAIT_TIMEOUT_MS", "20")
    n, guard = T * k, 1 << 16
    bufs = [torch.full((n + 2 * guard,), -7, dtype=torch.int32, device=DEV) for _ in range(2)]
    rows, tokens = (b[guard:guard + n] for b in bufs)
    for _ in range(5):
        ws.clear()
        ws.buf[256:].fill_(0xFF)
        _preset(ws, preset)
        fme.moe_route(logits, bias, k, rows=rows, tokens=tokens, workspace=ws)
        assert ws.error() == 2
        for b in bufs:
            assert (b[:guard] == -7).all() and (b[guard + n:] == -7).all()
            assert int(b.max()) < n


@pytest.mark.parametrize("R,E,N", [(1000, 8, 256), (1 << 25, 1024, 16384)])
def test_grouped_offsets_that_overlap(fme, R, E, N):
    """Groups that hold every row again and again (at the larger size their tiles are more than 32 bits count): nothing
    is computed, the error is reported, and ascending offsets run as before."""
    K = 128
    a = torch.full((1, K), 0x38, dtype=torch.uint8, device=DEV)  # ones
    sa = torch.ones(1, 1, device=DEV)
    w = torch.full((E, N, K), 0x38, dtype=torch.uint8, device=DEV)
    sw = torch.ones(E, N // 128, 1, device=DEV)
    rows = torch.zeros(R, dtype=torch.int32, device=DEV)
    out = torch.full((1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = fme.Workspace(fme.moe_grouped_fp8_workspace(R, K, N, E), DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1::2] = R
    fme.moe_grouped_gemm_fp8(a, sa, w, sw, off, in_rows=rows, out_rows=rows, out=out, workspace=ws)
    assert ws.error() == 8 and (out == 7).all()
    off[:] = 3
    off[-1] = 4
    fme.moe_grouped_gemm_fp8(a, sa, w, sw, off, in_rows=rows, out_rows=rows, out=out, workspace=ws)
    assert ws.error() == 0 and (out == K).all()


def _prompt(T):
    cfg = W.RAGGED
    w13h, w2h = W.fp8_weights_host(cfg, 61)
    s13, s2 = W.fp8_weight_scales(cfg, 61)
    weights = [torch.from_numpy(v).to(DEV) for v in (w13h.full(), s13, w2h.full(), s2)]
    q = torch.randint(0, 0x7F, (T, cfg.H), dtype=torch.uint8, device=DEV)
    s = torch.rand(T, cfg.H // 128, device=DEV) * 2.0 ** -8
    logits, bias = torch.randn(T, cfg.E, device=DEV), torch.zeros(cfg.E, device=DEV)
    return cfg, (q, s, logits, bias, *weights, cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0)


def test_prompt_errors_are_read_and_cleared_on_the_default_path(fme, monkeypatch):
    cfg, args = _prompt(200)
    want = fme.moe_prompt_fp8(*args)
    assert fme.kept_workspace_error() == 0 and fme.kept_workspace_error(DEV) == 0
    kept = fme._stream_workspace(fme.moe_route_workspace(200, cfg.E, cfg.top_k), torch.device(DEV), None)
    monkeypatch.setenv("FME_WAIT_TIMEOUT_MS", "20")
    _preset(kept, -1)
    fme.moe_prompt_fp8(*args)
    fme.moe_prompt_fp8(*args)
    assert fme.kept_workspace_error() == 2
    assert not kept.buf[:256].any() and fme.kept_workspace_error() == 0
    got = fme.moe_prompt_fp8(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and fme.kept_workspace_error() == 0


def test_prompt_with_the_callers_workspaces(fme, monkeypatch):
    cfg, args = _prompt(200)
    want = fme.moe_prompt_fp8(*args)
    ws = fme.moe_prompt_workspaces(300, cfg.H, cfg.I, cfg.E, cfg.top_k, DEV)  # they serve fewer tokens, too
    kept = dict(fme._ws_cache)
    got = fme.moe_prompt_fp8(*args, workspaces=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and [w.error() for w in ws] == [0, 0, 0]
    monkeypatch.setenv("FME_WAIT_TIMEOUT_MS", "20")
    _preset(ws[0], -1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _, _ = fme.moe_prompt_fp8(*args, workspaces=ws)
    assert set(fme._ws_cache) == set(kept)
    g.replay()
    assert [w.error() for w in ws] == [2, 0, 0]
    ws[0].clear()
    g.replay()
    assert [w.error() for w in ws] == [0, 0, 0] and torch.equal(y, want[0])
    assert fme.kept_workspace_error() == 0


def test_every_form_of_the_bounded_wait_runs_out(fme):
    """The flag's wait and the mbarrier waits of the decode and the grouped kernels (one barrier, two), one after another."""
    ws = fme.Workspace(512, DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert fme.lib.fme_selftest_wait_timeout(ws.ptr(), 512, 50, stream) == 0
    ws.error(), ws.clear()  # loaded
    t0 = time.perf_counter()
    assert fme.lib.fme_selftest_wait_timeout(ws.ptr(), 512, 50, stream) == 0
    assert ws.error() == 3
    assert 0.2 <= time.perf_counter() - t0 < 5.0
