"""Failure detection of the prompt operators, made on the host: a workspace whose words are preset so that a wait runs
out or a meeting finds words that no call left. No kernel faults; each call returns, reports and stays in its buffers."""

import time

import pytest
import torch

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
