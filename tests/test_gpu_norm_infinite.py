"""A normed value that is infinite: the block norm's scales and codes are add_rmsnorm's."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


@pytest.mark.parametrize("H", [256, 1024, 7168])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("quant,ue8m0", [("fp8", False), ("fp8", True), ("mxfp8", False)])
def test_infinite_values_of_a_block(fme, H, value, quant, ue8m0):
    """Its block's scale is infinite (MXFP8: the largest), its code NaN (MXFP8: the largest), the block's others 0."""
    x, gamma = torch.ones(3, H, dtype=BF, device=DEV), torch.ones(H, dtype=BF, device=DEV)
    gamma[133] = value
    x[:, 133] = 4.0  # 4 / sqrt(1 + 15 / H) of 3e38 overflows
    q, s, _, normed = fme.block_norm(x, gamma, quant=quant, ue8m0=ue8m0, want_normed=True)
    assert torch.isinf(normed[:, 133]).all()
    if quant == "fp8":
        rq, rs, _, _ = fme.add_rmsnorm_fp8(x, gamma, ue8m0=ue8m0)
        assert torch.isinf(s[:, 1]).all() and torch.isfinite(s[:, 0]).all()
        assert (q[:, 133] & 0x7F == 0x7F).all()
        assert (q[:, 128:133] == 0).all() and (q[:, 134:256] == 0).all()
    else:
        rq, rs, _, _ = fme.add_rmsnorm_mxfp8(x, gamma)
    block = slice(128, 256) if quant == "fp8" else slice(128, 160)
    assert torch.equal(q[:, block], rq[:, block])
    assert torch.equal(s[:, 1 if quant == "fp8" else 4], rs[:, 1 if quant == "fp8" else 4])
