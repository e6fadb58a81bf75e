"""Routing over few experts costs no more than over many: what every CTA adds up is as little as there is."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _us(fme, T, E, k, reps=10, runs=30):
    """The least time of a call in a graph, of many replays."""
    logits, bias = torch.randn(T, E, device=DEV), torch.zeros(E, device=DEV)
    ws = fme.Workspace(fme.moe_route_workspace(T, E, k), DEV)
    out = dict(zip(("ids", "weights", "offsets", "rows", "tokens"), fme.moe_route(logits, bias, k, workspace=ws)))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(reps):
            fme.moe_route(logits, bias, k, workspace=ws, **out)
    times = []
    for _ in range(runs):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1000 / reps)
    assert ws.error() == 0
    return min(times)


@pytest.mark.parametrize("T", [17, 300, 1533])
def test_eight_experts_cost_no_more_than_sixty_four(fme, T):
    """(Every thread of a CTA adding to eight experts' words, most of them nothing, took half as long again.)"""
    assert _us(fme, T, 8, 2) < 1.25 * _us(fme, T, 64, 2)
