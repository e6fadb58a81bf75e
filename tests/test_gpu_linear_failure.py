"""Failure detection of the dense product, made on the host: counts that no call left, and what a call that gave up leaves, are
planted in its workspace. Each call returns, reports, and stays in its buffers."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
COUNTS = 256             # byte of the counts of a cut product's units, up to 4096
REFUSED = -(1 << 31)     # in each of them after a call that gave up


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _words(ws, at, end):
    return ws.buf[at:end].view(torch.int32)


@pytest.fixture(params=[(64, 256, 7168, False), (128, 256, 7168, True), (20, 16, 3584, False), (300, 500, 2000, True)],
                ids=lambda p: "x".join(map(str, p)))
def product(request, fme):
    M, N, K, f32 = request.param
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
    ws = fme.Workspace(fme.linear_bf16_workspace(M, N, K), DEV)
    assert ws.nbytes > 4096  # K is cut: units count in the workspace

    def call():
        out = torch.full((M, N), 7.0, dtype=torch.float32 if f32 else BF, device=DEV)
        return fme.linear_bf16(x, w, out=out, workspace=ws)

    want = call()
    assert ws.error() == 0
    return call, ws, want


# Counts from one up to the most units that a tile has, and of sixteen units begun that none of this call did.
@pytest.mark.parametrize("word", [*range(1, 16), *((16 << 16) + n for n in range(16)), 0x7F7F7F7F, -1])
def test_counts_that_no_call_left_are_reported(product, word):
    call, ws, want = product
    _words(ws, COUNTS, 4096).fill_(word)
    call()
    assert ws.error() == 2
    assert ws.error() == 0  # read and cleared, but the workspace is not clean:
    for _ in range(3):
        assert (call() == 7).all() and ws.error() == 2
    ws.clear()
    assert torch.equal(call(), want) and ws.error() == 0


def test_one_count_that_no_call_left_is_reported(product):
    call, ws, want = product
    _words(ws, COUNTS, 4096)[0] = 1  # of the first tile's first rows alone
    call()
    assert ws.error() == 2
    ws.clear()
    assert torch.equal(call(), want) and ws.error() == 0


def test_after_a_call_that_gave_up_nothing_is_written_until_the_workspace_is_cleared(fme, product):
    call, ws, want = product
    for left in (0, 2, 3 << 16 | 2, 16 << 16 | 15):  # the units that had begun and arrived
        ws.clear()
        _words(ws, COUNTS, 4096).fill_(REFUSED + left)
        for _ in range(3):
            assert (call() == 7).all() and ws.error() == 2
    # Products that do not cut K have no counts and run as ever.
    x, w = torch.randn(700, 128, device=DEV).to(BF), torch.randn(640, 128, device=DEV).to(BF)
    for rows in (1, 8, 700):
        assert fme.linear_bf16_workspace(rows, 640, 128) == 4096
        assert torch.equal(fme.linear_bf16(x[:rows], w, workspace=ws), fme.linear_bf16(x[:rows], w))
        assert ws.error() == 0
    ws.clear()
    for _ in range(3):
        assert torch.equal(call(), want) and ws.error() == 0


def test_kept_workspaces_of_products_are_cleared_with_their_error(fme):
    M, N, K = 64, 256, 7168
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
    want = fme.linear_bf16(x, w)
    assert fme.kept_workspace_error() == 0
    kept = fme._stream_workspace(fme.linear_bf16_workspace(M, N, K), torch.device(DEV), None)
    _words(kept, COUNTS, 4096).fill_(REFUSED)
    fme.linear_bf16(x, w)
    assert fme.kept_workspace_error() == 2
    assert torch.equal(fme.linear_bf16(x, w), want) and fme.kept_workspace_error() == 0
