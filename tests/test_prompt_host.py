"""CPU checks of the prompt operators' argument handling: rejected before any launch, so no GPU is needed."""

import ctypes

import pytest

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


def test_norm_refusals(fme):
    d = dict(x=vp(16), ldx=256, res=vp(32), ldr=256, gamma=vp(16), T=4, H=256, eps=1e-5, ue=0, q=vp(16), s=vp(16),
             normed=None, res_out=vp(64), st=None)

    def call(**kw):
        return _call(fme.lib.fme_add_rmsnorm_fp8, d, **kw)

    assert call(x=None) == EINVAL and call(q=None) == EINVAL and call(s=None) == EINVAL
    assert call(res=None) == EINVAL and call(res_out=None) == EINVAL  # residual and residual_out come together
    assert call(T=-1) == EINVAL and call(T=(1 << 20) + 1) == EINVAL
    assert call(H=192, ldx=192) == EINVAL and call(H=0) == EINVAL and call(H=16512, ldx=16512, ldr=16512) == EINVAL
    assert call(ldx=248) == EINVAL and call(ldx=260) == EINVAL and call(ldr=0) == EINVAL
    assert call(res_out=vp(32), ldr=512) == EINVAL  # in place needs dense rows
    assert call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL
    assert call(x=vp(24)) == EALIGN and call(normed=vp(20)) == EALIGN and call(s=vp(4)) == EALIGN
    assert call(T=0) == 0
    del d["ue"]

    def mx(**kw):
        return _call(fme.lib.fme_add_rmsnorm_mxfp8, d, **kw)

    assert mx(H=240, ldx=240, ldr=240) == EINVAL and mx(T=0, H=96, s=vp(3)) == 0


def test_route_refusals(fme):
    d = dict(lg=vp(16), dt=0, bias=vp(16), T=4, E=40, k=3, scale=1.0, ids=vp(16), w=vp(16), off=vp(16), rows=vp(16),
             tok=vp(16), ws=vp(16), wsb=1 << 20, st=None)

    def call(**kw):
        return _call(fme.lib.fme_moe_route, d, **kw)

    assert call(lg=None) == EINVAL and call(tok=None) == EINVAL
    assert call(dt=2) == EINVAL and call(T=-1) == EINVAL and call(T=(1 << 20) + 1) == EINVAL
    assert call(E=1025) == EUNSUPPORTED and call(E=0) == EUNSUPPORTED
    assert call(k=0) == EINVAL and call(k=33) == EINVAL and call(E=2) == EINVAL
    assert call(scale=float("inf")) == EINVAL and call(rows=vp(20)) == EALIGN
    assert call(ws=None) == EWORKSPACE and call(wsb=16) == EWORKSPACE
    assert fme.moe_route_workspace(4, 40, 41) == 0
    sizes = [fme.moe_route_workspace(T, 256, 8) for T in (0, 1, 17, 300, 5000, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0  # a workspace for T serves every smaller T


def test_grouped_refusals(fme):
    d = dict(a=vp(16), sa=vp(16), a_rows=64, w=vp(16), sw=vp(16), off=vp(4), rows=vp(4), R=64, H=256, I=128, E=4,
             limit=7.0, ue=0, gf=0, q=vp(16), s=vp(16), ws=vp(16), wsb=256, st=None)

    def swiglu(**kw):
        return _call(fme.lib.fme_moe_grouped_swiglu_fp8, d, **kw)

    assert swiglu(a=None) == EINVAL and swiglu(off=None) == EINVAL and swiglu(s=None) == EINVAL
    assert swiglu(R=-1) == EINVAL and swiglu(R=(1 << 25) + 1) == EINVAL
    assert swiglu(H=200) == EINVAL and swiglu(I=192) == EINVAL and swiglu(I=8320) == EINVAL
    assert swiglu(H=16512) == EUNSUPPORTED and swiglu(E=1025) == EUNSUPPORTED
    assert swiglu(rows=None, a_rows=63) == EINVAL and swiglu(a_rows=0) == EINVAL
    assert swiglu(limit=0.0) == EINVAL and swiglu(limit=float("nan")) == EINVAL
    assert swiglu(w=vp(8)) == EALIGN and swiglu(off=vp(2)) == EALIGN and swiglu(rows=vp(6)) == EALIGN
    assert swiglu(ws=None) == EWORKSPACE and swiglu(wsb=255) == EWORKSPACE and swiglu(R=0) == 0

    g = dict(a=vp(16), sa=vp(16), a_rows=64, w=vp(16), sw=vp(16), off=vp(4), rows=vp(4), out_rows=vp(4), R=64, K=128,
             N=256, E=4, out=vp(16), out_n=64, ws=vp(16), wsb=256, st=None)

    def gemm(**kw):
        return _call(fme.lib.fme_moe_grouped_gemm_fp8, g, **kw)

    assert gemm(out=None) == EINVAL and gemm(N=64) == EINVAL and gemm(K=0) == EINVAL
    assert gemm(out_rows=None, out_n=63) == EINVAL and gemm(out_n=0) == EINVAL
    assert gemm(out=vp(8)) == EALIGN and gemm(out_rows=vp(7)) == EALIGN and gemm(R=0) == 0
    assert fme.moe_grouped_fp8_workspace(64, 200, 256, 4) == 0
    assert fme.moe_grouped_fp8_workspace(64, 256, 256, 4) >= 256


def test_binding_refuses_what_it_cannot_pass_on(fme):
    import torch

    x, g = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fme.add_rmsnorm_fp8(x, g)  # not on a GPU
    with pytest.raises(ValueError):
        fme.add_rmsnorm_fp8(x.float(), g)
    with pytest.raises(ValueError):
        fme.moe_route(torch.zeros(2, 8, dtype=torch.float16), torch.zeros(8), 2)
    a, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        fme.moe_grouped_gemm_fp8(a, s, torch.zeros(1, 128, 256, dtype=torch.uint8), torch.zeros(1, 1, 2),
                                 torch.zeros(2, dtype=torch.int32))


class _Operand:
    """What the binding asks of a tensor before it launches: enough to stand for one on a GPU that is not there."""

    def __init__(self, dtype, *shape, gpu=0):
        import torch
        self.dtype, self.shape, self.device, self.is_cuda = dtype, torch.Size(shape), torch.device("cuda", gpu), True

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = [self.shape[j + 1:].numel() for j in range(len(self.shape))]
        return tuple(s) if i is None else s[i]

    def data_ptr(self):
        return 16


def test_binding_refuses_operands_of_two_devices(fme, monkeypatch):
    import torch

    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    T, H, E, I, k = 4, 256, 3, 128, 2
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ws, far = fme.Workspace.__new__(fme.Workspace), fme.Workspace.__new__(fme.Workspace)
    ws.nbytes, ws.buf = 1 << 20, _Operand(u8, 1 << 20)
    far.nbytes, far.buf = 1 << 20, _Operand(u8, 1 << 20, gpu=1)
    calls = {
        fme.add_rmsnorm_fp8: dict(x=(bf, T, H), gamma=(bf, H), residual=(bf, T, H), q=(u8, T, H), scales=(f32, T, 2),
                                  normed=(bf, T, H), residual_out=(bf, T, H)),
        fme.add_rmsnorm_mxfp8: dict(x=(bf, T, H), gamma=(bf, H), residual=(bf, T, H), q=(u8, T, H),
                                    scales=(u8, T, 8), normed=(bf, T, H), residual_out=(bf, T, H)),
        fme.moe_route: dict(logits=(f32, T, E), bias=(f32, E), ids=(i32, T, k), weights=(f32, T, k),
                            offsets=(i32, E + 1), rows=(i32, T * k), tokens=(i32, T * k)),
        fme.moe_grouped_swiglu_fp8: dict(a=(u8, T, H), sa=(f32, T, 2), w13=(u8, E, 2 * I, H), s13=(f32, E, 2, 2),
                                         offsets=(i32, E + 1), in_rows=(i32, 8), q=(u8, 8, I), scales=(f32, 8, 1)),
        fme.moe_grouped_gemm_fp8: dict(a=(u8, T, H), sa=(f32, T, 2), w=(u8, E, I, H), sw=(f32, E, 1, 2),
                                       offsets=(i32, E + 1), in_rows=(i32, 8), out_rows=(i32, 8), out=(bf, 8, I)),
        fme.moe_prompt_fp8: dict(xq=(u8, T, H), sx=(f32, T, 2), logits=(f32, T, E), bias=(f32, E),
                                 w13=(u8, E, 2 * I, H), s13=(f32, E, 2, 2), w2=(u8, E, H, I), s2=(f32, E, 2, 1),
                                 shared_out=(bf, T, H)),
    }
    more = {fme.moe_route: dict(top_k=k, workspace=ws), fme.moe_grouped_swiglu_fp8: dict(workspace=ws),
            fme.moe_grouped_gemm_fp8: dict(workspace=ws),
            fme.moe_prompt_fp8: dict(top_k=k, limit=7.0, scale=1.0, ue8m0=False)}
    for fn, spec in calls.items():
        rest = more.get(fn, {})
        if fn is not fme.moe_prompt_fp8:  # everything on one device, but not the current one
            elsewhere = {**rest, "workspace": far} if "workspace" in rest else rest
            with pytest.raises(ValueError, match="current device"):
                fn(**{n: _Operand(*v, gpu=1) for n, v in spec.items()}, **elsewhere)
            if "workspace" in rest:
                with pytest.raises(ValueError, match="workspace"):
                    fn(**{n: _Operand(*v) for n, v in spec.items()}, **elsewhere)
        for name in spec:
            if fn is fme.moe_prompt_fp8 and name in ("s13", "s2"):
                continue  # the products refuse those
            with pytest.raises(ValueError, match="cuda:1"):
                fn(**{n: _Operand(*v, gpu=int(n == name)) for n, v in spec.items()}, **rest)
