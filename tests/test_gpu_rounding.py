"""The kernels' short arithmetic forms against the general operations, bit for bit: reciprocals and SiLU over every float
of their ranges, quotients over 2^32 pairs; and a gate far below zero through the operator itself."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _bits(v):
    return int(np.float32(v).view(np.uint32))


def _mismatches(fme, what, first, count):
    n = torch.zeros(1, dtype=torch.int64, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert fme.lib.fme_selftest_rounding(what, first, count, n.data_ptr(), stream) == 0
    return int(n.item())


def test_reciprocals(fme):
    first, last = _bits(2.0 ** -4), _bits(2.0 ** 125)
    assert _mismatches(fme, 0, first, last - first + 1) == 0


def test_silu_of_every_float(fme):
    assert _mismatches(fme, 1, 0, 1 << 32) == 0


def test_quotients(fme):
    assert _mismatches(fme, 2, 0, 1 << 32) == 0


def test_selftest_arguments(fme):
    n = torch.zeros(2, dtype=torch.int64, device=DEV)
    call = fme.lib.fme_selftest_rounding
    assert call(3, 0, 1, n.data_ptr(), None) == -1 and call(0, 0, 0, n.data_ptr(), None) == -1
    assert call(0, 0, (1 << 32) + 1, n.data_ptr(), None) == -1 and call(0, 0, 1, None, None) == -1
    assert call(0, 0, 1, n.data_ptr() + 4, None) == -3


@pytest.mark.parametrize("gate", [-50.0, -85.0, -88.0, -100.0, -1e9, -1e25, -3e38])
def test_swiglu_of_a_gate_far_below_zero(fme, gate):
    """One gate value, the rest zero: the hidden value is silu(gate) * limit, which is zero for every code from -60 down.
    The scale is then the least one, max(0, 1e-10) / 448."""
    H, I = 128, 128
    a = torch.zeros(1, H, dtype=torch.uint8, device=DEV)
    a[0, 0] = 0x38  # one
    sa = torch.ones(1, 1, device=DEV)
    w = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device=DEV)
    w[0, 5, 0], w[0, I + 5, 0] = 0x78, 0xB8  # up 256 (clamped to the limit), gate -1
    sw = torch.tensor([[[1.0], [-gate]]], device=DEV)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    q, s = fme.moe_grouped_swiglu_fp8(a, sa, w, sw, off, limit=7.0)
    g = np.float64(np.float32(gate))
    h = g * np.exp(g) * 7.0  # 1 + exp(g) is one
    want = max(abs(h), 1e-10) / 448
    assert abs(float(s) - want) <= 8 * 2.0 ** -24 * want
    assert q[0, 5].item() & 0x7F == 0 and not q[0, :5].any() and not q[0, 6:].any()
