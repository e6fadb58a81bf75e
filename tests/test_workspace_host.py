"""CPU checks of the workspaces that the binding keeps for calls that are given none: which calls get the same one."""

import pytest

from tests.test_prompt_host import _Operand


@pytest.fixture
def calls(monkeypatch):
    """Decode calls by name, each returning the address of the workspace it was given; nothing is launched."""
    import __graft_entry__
    __graft_entry__.build()
    import torch

    import fp4_moe_expert_gb300 as fme

    class Kept:
        made = 0

        def __init__(self, nbytes, device):
            Kept.made += 1
            self.nbytes, self.buf, self.at = int(nbytes), _Operand(torch.uint8, int(nbytes)), Kept.made

        def ptr(self):
            return self.at

    monkeypatch.setattr(fme, "Workspace", Kept)
    monkeypatch.setattr(fme, "_ws_cache", {})
    monkeypatch.setattr(fme, "_stream", lambda device: 0)
    given = []
    for name, n in (("moe_routed_fp8", -3), ("moe_routed_fp8_mx", -3), ("moe_layer_fp8", -3), ("shared_expert_fp8", -3),
                    ("moe_routed_nvfp4", -3), ("moe_layer_nvfp4", -3)):
        monkeypatch.setattr(fme.lib, "fme_" + name, lambda *a, n=n: given.append(a[n]) or 0)
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None: _Operand(dtype, *shape))
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32

    def expert(*lead, H, I):
        return (_Operand(u8, *lead, 2 * I, H), _Operand(f32, *lead, 2 * I // 128, H // 128), _Operand(u8, *lead, H, I),
                _Operand(f32, *lead, H // 128, I // 128))

    def routed(M, H, I, E, k):
        fme.moe_routed_fp8(_Operand(bf, M, H), _Operand(f32, M, E), _Operand(f32, E), *expert(E, H=H, I=I), k, 7.0, 1.0, 0)
        return given[-1]

    def routed_mx(M, H, I, E, k):
        fme.moe_routed_fp8_mx(_Operand(u8, M, H), _Operand(u8, M, H // 32), _Operand(f32, M, E), _Operand(f32, E),
                              *expert(E, H=H, I=I), k, 7.0, 1.0, 0)
        return given[-1]

    def layer(M, H, I, E, k):
        fme.moe_layer_fp8(_Operand(bf, M, H), _Operand(f32, M, E), _Operand(f32, E), *expert(E, H=H, I=I), k, 7.0, 1.0, 0,
                          *expert(H=H, I=I), 7.0, 0)
        return given[-1]

    def shared(M, H, I):
        fme.shared_expert_fp8(_Operand(bf, M, H), *expert(H=H, I=I), 7.0, 0)
        return given[-1]

    def fp4(L, H, N):
        return (_Operand(u8, L, 2 * N, H // 2), _Operand(u8, L, 2 * N, H // 16), _Operand(u8, L, H, N // 2),
                _Operand(u8, L, H, N // 16))

    def nvfp4(M, H, N, L, k):
        fme.moe_routed_nvfp4(_Operand(bf, M, H), _Operand(i32, M, k), _Operand(f32, M, k), *fp4(L, H, N), 0)
        return given[-1]

    def nvfp4_layer(M, H, N, L, k):
        fme.moe_layer_nvfp4(_Operand(bf, M, H), _Operand(f32, M, 2 * L), _Operand(f32, 2 * L), *fp4(L, H, N), 0, k)
        return given[-1]

    return fme, dict(routed=routed, routed_mx=routed_mx, layer=layer, shared=shared, nvfp4=nvfp4, nvfp4_layer=nvfp4_layer)


def test_kept_workspaces_of_one_size_but_other_layouts_are_apart(calls):
    """Calls of two kinds, or of other sizes than M, place their counters differently, whatever their bytes."""
    fme, c = calls
    assert fme.moe_routed_fp8_workspace(1, 256, 128, 8, 2) == fme.shared_expert_fp8_workspace(1, 256, 256)
    assert fme.moe_routed_fp8_workspace(1, 1024, 128, 8, 2) == fme.moe_routed_fp8_workspace(1, 256, 256, 8, 2)
    assert fme.moe_routed_nvfp4_workspace(1, 256, 128, 8, 2) == fme.moe_routed_nvfp4_workspace(1, 256, 256, 8, 2)
    apart = [c["routed"](1, 256, 128, 8, 2), c["shared"](1, 256, 256), c["routed"](1, 1024, 128, 8, 2),
             c["routed"](1, 256, 256, 8, 2), c["nvfp4"](1, 256, 128, 8, 2), c["nvfp4"](1, 256, 256, 8, 2),
             c["shared"](1, 256, 128)]
    assert len(set(apart)) == len(apart)


def test_kept_workspaces_serve_again(calls):
    _, c = calls
    for name, sizes in (("routed", (4, 512, 256, 16, 4)), ("layer", (4, 512, 256, 16, 4)), ("shared", (4, 512, 256)),
                        ("nvfp4", (4, 512, 256, 16, 4))):
        first = c[name](*sizes)
        assert c[name](*sizes) == first
    # Entry points that share a layout share the workspace.
    assert c["routed"](4, 512, 256, 16, 4) == c["routed_mx"](4, 512, 256, 16, 4)
    assert c["nvfp4"](4, 512, 256, 16, 4) == c["nvfp4_layer"](4, 512, 256, 16, 4)
