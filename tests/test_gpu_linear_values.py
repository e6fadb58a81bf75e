"""The dense product's activations over the whole range of their argument, from one token to many, against the 64-bit
oracle."""

import numpy as np
import pytest
import torch

from oracle import linear as oracle_linear

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _arguments():
    """To where each activation ends: past the arguments whose exponential overflows or is below the normal numbers."""
    near = [s * (v + d) for s in (-1.0, 1.0) for v in (0.0, 20.0, 87.336, 88.376, 88.722, 92.0, 103.9, 126.0)
            for d in np.linspace(-0.3, 0.3, 61)]
    far = [s * v for s in (-1.0, 1.0) for v in (150.0, 1e3, 1e10, 1e30, 3e38)]
    return np.concatenate([np.linspace(-130, 130, 2086), near, far, [0.0, 1e-3, -1e-3, 1e-30, -1e-30]]).astype(np.float32)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("M,f32", [(1, False), (1, True), (8, False), (16, True), (17, False), (70, False), (70, True),
                                   (300, False), (20000, False), (20000, True)])
def test_activations_over_their_whole_range(fme, act, M, f32):
    b = _arguments()
    N, K = len(b), 64
    x = torch.zeros(M, K, dtype=BF, device=DEV)  # sums of zeros: the argument is the bias
    w = torch.randn(N, K, device=DEV).to(BF)
    got = fme.linear_bf16(x, w, torch.from_numpy(b).to(DEV), act, out_dtype=torch.float32 if f32 else BF)
    assert torch.equal(got, got[:1].expand(M, N))
    y, _ = oracle_linear.linear(np.zeros((1, K)), np.zeros((N, K)), b, act)
    # The argument is exact, so that the activation's own errors are left: 16 u as the oracle takes them, of GELU's tail 4 z^2 u
    # more (past z = 20 it is the argument or nothing), and 2^-126 for what is below the normal numbers. Then the output's
    # rounding. BF16 outputs may take the hardware's exp, off by 2 + 1.173 |z| units of 2^-23 as documented.
    z = np.minimum(np.abs(b.astype(np.float64)), 130)
    rel = {"relu": 0.0, "gelu": 16 + 4 * np.minimum(z, 20) ** 2}.get(act, 16.0) * 2.0 ** -24
    tol = np.abs(y) * (rel + (2.0 ** -24 if f32 else 2.0 ** -8 + (2 + 1.173 * z) * 2.0 ** -23)) + 2.0 ** -126
    got = got[:1].double().cpu().numpy()
    over = np.abs(y) > 3.38e38  # beyond BF16's largest: infinite is right, too
    ok = (np.abs(got - y) <= tol) | (over & (np.isinf(got)))
    assert ok.all(), [(b[i], got[0, i], y[0, i]) for i in np.nonzero(~ok[0])[0][:5]]


@pytest.mark.parametrize("act,want", [("relu", (0.0, np.inf)), ("sigmoid", (0.0, 1.0)), (None, (-np.inf, np.inf))])
@pytest.mark.parametrize("M", [1, 8, 70])
def test_infinite_arguments(fme, act, want, M):
    x, w = torch.zeros(M, 64, dtype=BF, device=DEV), torch.zeros(3, 64, dtype=BF, device=DEV)
    b = torch.tensor([-np.inf, np.inf, np.nan], device=DEV)
    for dt in (torch.float32, BF):
        got = fme.linear_bf16(x, w, b, act, out_dtype=dt)
        assert (got[:, 0] == want[0]).all() and (got[:, 1] == want[1]).all() and torch.isnan(got[:, 2]).all()
