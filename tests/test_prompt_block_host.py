"""CPU checks of what the binding's prompt calls hand to their steps."""

import pytest

from tests.test_prompt_host import _Operand


@pytest.fixture(scope="module")
def fme():
    import __graft_entry__
    __graft_entry__.build()
    import fp4_moe_expert_gb300 as m
    return m


class _Reached(Exception):
    pass


def _stop(given):
    def step(*args, **kw):
        given.append((args, kw))
        raise _Reached
    return step


def _operands(T=4, H=256, E=6, I=128):
    import torch
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    return dict(xq=_Operand(u8, T, H), sx=_Operand(f32, T, H // 128), logits=_Operand(f32, T, E), bias=_Operand(f32, E),
                w13=_Operand(u8, E, 2 * I, H), s13=_Operand(f32, E, 2 * I // 128, H // 128), w2=_Operand(u8, E, H, I),
                s2=_Operand(f32, E, H // 128, I // 128), top_k=2, limit=7.0, scale=1.0, ue8m0=False), \
        dict(normed=_Operand(bf, T, H), residual=_Operand(bf, T, H), router=_Operand(bf, E, H))


@pytest.mark.parametrize("given,want", [(None, None), ((1, 2, 3), None), ((1, 2, 3, 4), 4)])
def test_the_blocks_router_product_takes_the_fourth_workspace(fme, monkeypatch, given, want):
    args, more = _operands()
    del args["logits"]
    seen = []
    monkeypatch.setattr(fme, "linear_bf16", _stop(seen))
    with pytest.raises(_Reached):
        fme.moe_prompt_block_fp8(**args, **more, workspaces=given)
    assert seen[0][1].get("workspace") == want


def test_workspaces_of_a_block_serve_every_fewer_tokens(fme):
    H, I, E, k = 7168, 2048, 256, 8
    assert len(fme.moe_prompt_workspaces(300, H, I, E, k, "cpu")) == 3
    for T in (1, 70, 700):
        ws = fme.moe_prompt_workspaces(T, H, I, E, k, "cpu", router=True)
        assert len(ws) == 4
        for t in range(1, T + 1):
            assert fme.moe_route_workspace(t, E, k) <= ws[0].nbytes and fme.linear_bf16_workspace(t, E, H) <= ws[3].nbytes
    # A product of more tokens than any that cuts K needs no more.
    assert fme.moe_prompt_workspaces(1 << 20, 256, 128, 8, 2, "cpu", router=True)[3].nbytes <= 1 << 25


def test_rows_pass_every_option_of_the_routing_on(fme, monkeypatch):
    """moe_route knows no groups: whatever is asked of them goes to the call that checks it."""
    args, _ = _operands()
    plain, scored = [], []
    monkeypatch.setattr(fme, "moe_route", _stop(plain))
    monkeypatch.setattr(fme, "moe_route_groups", _stop(scored))

    def call(**kw):
        for fn in (fme.moe_prompt_rows_fp8, fme.moe_prompt_fp8):
            with pytest.raises(_Reached):
                fn(**{**args, **kw})

    call(), call(top_groups=1)
    assert len(plain) == 4 and not scored
    call(group_top=2)
    assert len(plain) == 4 and len(scored) == 2 and all(2 in a for a, _ in scored)
    call(group_top=7), call(group_top=1, top_groups=1), call(renormalise=False), call(score="softmax"), call(bias=None)
    assert len(plain) == 4 and len(scored) == 12
    with pytest.raises(ValueError, match="top_groups"):
        fme.moe_prompt_fp8(**args, top_groups=2)


def test_prompt_operands_are_checked_once(fme, monkeypatch):
    args, _ = _operands()
    checks, seen = [], []
    need = fme._need_prompt
    monkeypatch.setattr(fme, "_need_prompt", lambda *a, **kw: checks.append(need(*a, **kw)))
    monkeypatch.setattr(fme, "moe_route", _stop(seen))
    for fn in (fme.moe_prompt_fp8, fme.moe_prompt_rows_fp8):
        checks.clear()
        with pytest.raises(_Reached):
            fn(**args)
        assert len(checks) == 1
