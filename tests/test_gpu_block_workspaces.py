"""A routed block of a prompt with the caller's workspaces: eager and in a graph, its errors all in their words."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def test_block_with_the_callers_workspaces(fme):
    T, H, I, E, k = 50, 3584, 128, 24, 3
    assert fme.linear_bf16_workspace(T, E, H) > 4096  # the router's product cuts K: it has counts to be wrong about
    codes = [torch.randint(0, 0x7F, s, dtype=torch.uint8, device=DEV) for s in ((E, 2 * I, H), (E, H, I))]
    scales = [torch.rand(s, device=DEV) * 2.0 ** -8 for s in ((E, 2 * I // 128, H // 128), (E, H // 128, I // 128))]
    experts = (codes[0], scales[0], codes[1], scales[1])
    x = torch.randn(T, H, device=DEV).to(BF)
    gamma = torch.ones(H, dtype=BF, device=DEV)
    router = (torch.randn(E, H, device=DEV) / 32).to(BF)
    bias = torch.zeros(E, device=DEV)
    xq, sx, h, normed = fme.block_norm(x, gamma, x, quant="fp8", want_normed=True)

    def block(ws, n=T):
        return fme.moe_prompt_block_fp8(xq[:n], sx[:n], normed[:n], h[:n], router, bias, *experts, k, 7.0, 1.0, False,
                                        next_gamma=gamma, quant="fp8", groups=4, top_groups=2, workspaces=ws)

    want = {n: block(None, n) for n in (1, 33, T)}
    torch.cuda.synchronize()
    ws = fme.moe_prompt_workspaces(T, H, I, E, k, DEV, router=True)
    kept = dict(fme._ws_cache)
    fme._ws_cache.clear()  # a step that took a kept workspace would make one
    try:
        for n, ref in want.items():
            assert all(torch.equal(a, b) for a, b in zip(block(ws, n), ref))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = block(ws)
        assert not fme._ws_cache
    finally:
        fme._ws_cache.update(kept)
    g.replay()
    assert [w.error() for w in ws] == [0, 0, 0, 0]
    assert all(torch.equal(a, b) for a, b in zip(got, want[T]))
    ws[3].buf[256:4096].view(torch.int32).fill_(1)  # counts that no call left
    g.replay()
    assert [w.error() for w in ws] == [0, 0, 0, 2]
    ws[3].clear()
    g.replay()
    assert [w.error() for w in ws] == [0, 0, 0, 0]
    assert all(torch.equal(a, b) for a, b in zip(got, want[T]))
    # Three of them: the router's product has a kept one.
    assert all(torch.equal(a, b) for a, b in zip(block(ws[:3]), want[T]))
    assert fme.kept_workspace_error() == 0
