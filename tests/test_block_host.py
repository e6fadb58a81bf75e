"""CPU checks of the argument handling of the operators around a routed block: rejected before any launch."""

import ctypes

import pytest

from tests.test_prompt_host import _Operand

vp = ctypes.c_void_p
EINVAL, EUNSUPPORTED, EALIGN, EWORKSPACE = -1, -2, -3, -6


@pytest.fixture(scope="module")
def fme():
    import __graft_entry__
    __graft_entry__.build()
    import fp4_moe_expert_gb300 as m
    return m


def _call(fn, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return fn(*args.values())


def test_route_groups_refusals(fme):
    d = dict(lg=vp(16), dt=0, bias=vp(16), T=4, E=40, k=3, score=0, groups=5, top=2, each=2, renorm=1, scale=1.0,
             ids=vp(16), w=vp(16), off=vp(16), rows=vp(16), tok=vp(16), ws=vp(16), wsb=1 << 20, st=None)

    def call(**kw):
        return _call(fme.lib.fme_moe_route_groups, d, **kw)

    assert call(lg=None) == EINVAL and call(tok=None) == EINVAL
    assert call(dt=2) == EINVAL and call(T=-1) == EINVAL and call(T=(1 << 20) + 1) == EINVAL
    assert call(E=1025) == EUNSUPPORTED and call(k=0) == EINVAL and call(k=33) == EINVAL
    assert call(score=2) == EINVAL and call(score=-1) == EINVAL
    assert call(groups=0) == EINVAL and call(groups=3) == EINVAL and call(groups=40) == EINVAL  # 40 > 32
    assert call(top=0) == EINVAL and call(top=6) == EINVAL
    assert call(k=17) == EINVAL and call(k=16, top=1) == EINVAL  # two groups of 8 hold 16
    assert call(each=0) == EINVAL and call(each=3) == EINVAL and call(E=32, groups=32, top=32, each=2) == EINVAL
    assert call(scale=float("nan")) == EINVAL and call(rows=vp(20)) == EALIGN and call(bias=vp(8)) == EALIGN
    assert call(ws=None) == EWORKSPACE and call(wsb=16) == EWORKSPACE


def test_block_norm_refusals(fme):
    far = [vp(1 << 30 | i << 24) for i in range(12)]
    d = dict(x=far[0], ldx=256, rw=far[1], k=2, shared=far[2], post=far[3], gate=far[4], ldg=256, res=far[5], ldr=256,
             alpha=1.0, gamma=far[6], T=4, H=256, eps=1e-5, quant=1, ue=0, q=far[7], s=far[8], normed=far[9],
             res_out=far[10], st=None)

    def call(**kw):
        return _call(fme.lib.fme_block_norm, d, **kw)

    assert call(T=0) == 0
    assert call(x=None) == EINVAL and call(res_out=None) == EINVAL
    assert call(q=None) == EINVAL and call(s=None) == EINVAL and call(quant=3) == EINVAL and call(quant=-1) == EINVAL
    assert call(quant=0) == EINVAL  # q and scales without quant
    assert call(gamma=None) == EINVAL  # normed and q need it
    assert call(gamma=None, quant=0, q=None, s=None, normed=None, T=0) == 0
    assert call(k=0) == EINVAL and call(rw=None) == EINVAL and call(k=33) == EINVAL and call(k=-1) == EINVAL
    assert call(k=0, rw=None) == EINVAL  # a shared expert's rows without routes
    assert call(T=-1) == EINVAL and call(T=(1 << 20) + 1) == EINVAL and call(T=1 << 20, k=33) == EINVAL
    assert call(H=192, ldx=192, ldg=192, ldr=192) == EINVAL and call(H=16512) == EINVAL
    assert call(ldx=248) == EINVAL and call(ldx=260) == EINVAL and call(ldr=0) == EINVAL and call(ldg=8) == EINVAL
    assert call(ldx=(1 << 34) + 8) == EINVAL
    assert call(alpha=float("inf")) == EINVAL and call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL
    assert call(x=vp(24)) == EALIGN and call(s=vp((1 << 30) + 4)) == EALIGN and call(rw=vp((1 << 30) + 2)) == EALIGN
    # Outputs over inputs and over one another.
    assert call(res_out=far[0]) == EINVAL and call(normed=far[10]) == EINVAL and call(q=far[5]) == EINVAL
    assert call(res_out=far[5], ldr=512) == EINVAL  # in place needs dense rows
    assert call(res_out=vp(far[5].value + 512)) == EINVAL
    assert call(s=vp(far[6].value)) == EINVAL and call(normed=vp(far[4].value + 16)) == EINVAL


def test_linear_refusals(fme):
    far = [vp(1 << 30 | i << 24) for i in range(6)]
    d = dict(x=far[0], ldx=256, w=far[1], ldw=256, bias=far[2], act=0, res=far[3], ldr=100, M=40, N=100, K=250,
             out=far[4], dt=1, ldo=100, ws=far[5], wsb=1 << 24, st=None)

    def call(**kw):
        return _call(fme.lib.fme_linear_bf16, d, **kw)

    assert call(M=0) == 0
    assert call(x=None) == EINVAL and call(w=None) == EINVAL and call(out=None) == EINVAL
    assert call(M=-1) == EINVAL and call(M=(1 << 20) + 1) == EINVAL and call(N=0) == EINVAL and call(K=0) == EINVAL
    assert call(N=(1 << 17) + 1) == EINVAL and call(K=(1 << 17) + 1) == EINVAL
    assert call(ldx=248) == EINVAL and call(ldw=250) == EINVAL and call(ldx=(1 << 34) + 8) == EINVAL
    assert call(ldo=99) == EINVAL and call(ldr=99) == EINVAL
    assert call(act=5) == EINVAL and call(act=-1) == EINVAL and call(dt=2) == EINVAL
    assert call(x=vp(24)) == EALIGN and call(out=vp((1 << 30) + 1)) == EALIGN and call(bias=vp((1 << 30) + 2)) == EALIGN
    assert call(dt=0, res=vp((1 << 30) + 2)) == EALIGN
    assert call(ws=None) == EWORKSPACE and call(wsb=64) == EWORKSPACE
    assert call(out=far[0]) == EINVAL and call(out=far[1]) == EINVAL and call(out=far[2]) == EINVAL
    assert call(out=vp(far[3].value + 2)) == EINVAL and call(out=far[3], ldo=101) == EINVAL
    # Columns of one buffer: those beside each other are fine, those that meet are not.
    assert call(out=vp(far[0].value + 512), ldx=400, ldo=400, ws=None) == EWORKSPACE
    assert call(out=vp(far[0].value + 496), ldx=400, ldo=400, ws=None) == EINVAL
    assert call(out=vp(far[0].value + 608), ldx=400, ldo=400, ws=None) == EINVAL  # its ends reach the next row of x
    assert fme.linear_bf16_workspace(-1, 8, 8) == 0 and fme.linear_bf16_workspace(8, 0, 8) == 0
    for M, N, K in ((0, 8, 8), (1, 256, 7168), (64, 256, 7168), (1533, 896, 3584), (1 << 20, 1 << 17, 8)):
        assert 0 < fme.linear_bf16_workspace(M, N, K) <= 1 << 25


def test_binding_refuses_what_it_cannot_pass_on(fme):
    import torch

    bf = torch.bfloat16
    x, g = torch.zeros(2, 256, dtype=bf), torch.zeros(256, dtype=bf)
    with pytest.raises(ValueError):
        fme.block_norm(x, g)  # not on a GPU
    with pytest.raises(ValueError):
        fme.linear_bf16(x, torch.zeros(8, 256, dtype=bf))
    with pytest.raises(ValueError):
        fme.moe_route_groups(torch.zeros(2, 8, dtype=torch.float16), None, 2)
    with pytest.raises(ValueError, match="score"):
        fme.moe_route_groups(torch.zeros(2, 8), None, 2, score="tanh")


def test_binding_refuses_operands_that_disagree(fme, monkeypatch):
    import torch

    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    T, H, E, k = 4, 256, 6, 2
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ws, far = fme.Workspace.__new__(fme.Workspace), fme.Workspace.__new__(fme.Workspace)
    ws.nbytes, ws.buf = 1 << 20, _Operand(u8, 1 << 20)
    far.nbytes, far.buf = 1 << 20, _Operand(u8, 1 << 20, gpu=1)
    calls = {
        fme.moe_route_groups: (dict(logits=(f32, T, E), bias=(f32, E), ids=(i32, T, k), weights=(f32, T, k),
                                    offsets=(i32, E + 1), rows=(i32, T * k), tokens=(i32, T * k)),
                               dict(top_k=k, workspace=ws)),
        fme.block_norm: (dict(x=(bf, T * k, H), gamma=(bf, H), residual=(bf, T, H), route_weights=(f32, T, k),
                              shared_out=(bf, T, H), post_gamma=(bf, H), gate=(bf, T, H), q=(u8, T, H),
                              scales=(f32, T, 2), normed=(bf, T, H), residual_out=(bf, T, H)), dict(quant="fp8")),
        fme.linear_bf16: (dict(x=(bf, T, H), w=(bf, E, H), bias=(f32, E), residual=(bf, T, E), out=(bf, T, E)),
                          dict(workspace=ws)),
    }
    for fn, (spec, rest) in calls.items():
        elsewhere = {**rest, "workspace": far} if "workspace" in rest else rest
        with pytest.raises(ValueError, match="current device"):  # everything on one device, but not the current one
            fn(**{n: _Operand(*v, gpu=1) for n, v in spec.items()}, **elsewhere)
        if "workspace" in rest:
            with pytest.raises(ValueError, match="workspace"):
                fn(**{n: _Operand(*v) for n, v in spec.items()}, **elsewhere)
        for name in spec:
            with pytest.raises(ValueError, match="cuda:1"):
                fn(**{n: _Operand(*v, gpu=int(n == name)) for n, v in spec.items()}, **rest)
        for name, (dtype, *shape) in spec.items():  # one more column (or value) than the others agree on
            if name == "x" and fn is fme.linear_bf16 or name == "logits":
                continue
            with pytest.raises(ValueError):
                fn(**{n: _Operand(*v) for n, v in {**spec, name: (dtype, *shape[:-1], shape[-1] + 1)}.items()}, **rest)
    x = _Operand(bf, T, H)
    with pytest.raises(ValueError, match="quant"):
        fme.block_norm(x, _Operand(bf, H), quant="int8")
    with pytest.raises(ValueError, match="without quant"):
        fme.block_norm(x, _Operand(bf, H), q=_Operand(u8, T, H))
    with pytest.raises(ValueError, match="without gamma"):
        fme.block_norm(x, None, want_normed=True)
    with pytest.raises(ValueError, match="without route_weights"):
        fme.block_norm(x, _Operand(bf, H), shared_out=_Operand(bf, T, H))
    with pytest.raises(ValueError, match="activation"):
        fme.linear_bf16(x, _Operand(bf, E, H), activation="tanh")
    with pytest.raises(ValueError, match="out_dtype"):
        fme.linear_bf16(x, _Operand(bf, E, H), out_dtype=torch.float16)
    with pytest.raises(ValueError, match="expected a CUDA"):
        fme.linear_bf16(x, _Operand(bf, E, H), residual=_Operand(f32, T, E))
