"""One workspace for routing, the grouped products and the dense product in turn, kept by the binding or the caller's: what
one of them leaves behind is no count of another's."""

import pytest
import torch

from synth import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


# Products whose K is cut, after routings of as many bytes of workspace and of other sizes.
@pytest.mark.parametrize("T,E,k,M,N,K", [(1350, 384, 6, 20, 16, 3584), (1270, 384, 6, 20, 16, 3584),
                                         (1160, 896, 16, 64, 40, 2048), (16384, 1024, 8, 64, 256, 7168)])
@pytest.mark.parametrize("kept", [True, False])
def test_routing_and_cut_products_in_turn(fme, T, E, k, M, N, K, kept):
    need = fme.moe_route_workspace(T, E, k), fme.linear_bf16_workspace(M, N, K)
    assert need[1] > 4096  # K is cut
    logits, bias = torch.randn(T, E, device=DEV), 0.1 * torch.randn(E, device=DEV)
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
    route = fme.moe_route(logits, bias, k, workspace=fme.Workspace(need[0], DEV))
    product = fme.linear_bf16(x, w, workspace=fme.Workspace(need[1], DEV))
    ws = None if kept else fme.Workspace(max(need), DEV)
    for _ in range(3):
        got = fme.moe_route(logits, bias, k, workspace=ws)
        out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
        fme.linear_bf16(x, w, out=out, workspace=ws)
        assert torch.equal(out, product)
        assert all(torch.equal(a, b) for a, b in zip(got, route))
    assert (fme.kept_workspace_error() if kept else ws.error()) == 0


def test_a_prompt_of_one_workspace(fme):
    cfg, T = W.RAGGED, 700
    w13h, w2h = W.fp8_weights_host(cfg, 61)
    s13, s2 = W.fp8_weight_scales(cfg, 61)
    experts = [torch.from_numpy(v).to(DEV) for v in (w13h.full(), s13, w2h.full(), s2)]
    x = torch.randn(T, cfg.H, device=DEV).to(BF)
    gamma = torch.ones(cfg.H, dtype=BF, device=DEV)
    router = (torch.randn(cfg.E, cfg.H, device=DEV) / 32).to(BF)
    bias = torch.zeros(cfg.E, device=DEV)
    xq, sx, h, normed = fme.block_norm(x, gamma, x, quant="fp8", want_normed=True)

    def layer(own, ws):
        logits = fme.linear_bf16(normed, router, out_dtype=torch.float32, workspace=own)
        cut = fme.linear_bf16(normed[:20], router, workspace=own)
        return (*fme.moe_prompt_fp8(xq, sx, logits, bias, *experts, cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0,
                                    workspaces=ws), logits, cut)

    want = layer(None, None)
    one = fme.Workspace(1 << 23, DEV)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(layer(one, (one, one, one)), want))
    assert one.error() == 0


def test_graphs_and_streams_of_cut_products_share_nothing(fme):
    """Two graphs of routing and a cut product, replayed side by side on two streams beside calls on a third."""
    T, E, k, (M, N, K) = 1350, 384, 6, (20, 16, 3584)
    logits, bias = torch.randn(T, E, device=DEV), 0.1 * torch.randn(E, device=DEV)
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)

    def step():
        return [*fme.moe_route(logits, bias, k), fme.linear_bf16(x, w), fme.linear_bf16(x, w, out_dtype=torch.float32)]

    want = step()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step())
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = step()
    torch.cuda.synchronize()
    for got in (*outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fme.kept_workspace_error() == 0
