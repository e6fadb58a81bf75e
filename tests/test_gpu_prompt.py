"""GPU checks of the prompt operators against the 64-bit oracle.

Tolerances, from the arithmetic (u = 2^-24, the FP32 rounding):
* norm: a thread sums at most 64 squares, 13 additions join them, so the mean is within 80 u and 1 / sqrt within
  half that plus three roundings; with the two products y is within 64 u of the exact norm.
* a product: a block's partial sum is an FP32 accumulation of exact products and the scaled partials are added one
  after another: within (K/128 + 8) * 2 u of the sum of the terms' magnitudes.
* SwiGLU: |silu'| <= 1.1 and |silu(g)| <= |g|; expf, the division and the products add at most 16 u of the result.
* E4M3 holds a value within 2^-4 of it (2^-10 of the scale below 2^-6 of it), BF16 within 2^-8.
"""

import numpy as np
import pytest
import torch

from oracle import codecs, prompt, quant, routing
from oracle.ep_local import mx_exponent
from oracle.finalize import finalize as oracle_finalize
from oracle.moe_fp8 import clamped_swiglu
from synth import workloads as W
from tests.parity import assert_outputs, assert_routing

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


# --------------------------------------------------------------------------- norm
def _norm_inputs(T, H, seed, residual):
    rng = np.random.default_rng(seed)
    x = codecs.bf16_round((rng.normal(size=(T, H)) * np.exp2(rng.integers(-3, 4, size=(T, 1)))).astype(np.float32))
    r = codecs.bf16_round((5 * rng.normal(size=(T, H))).astype(np.float32)) if residual else None
    g = codecs.bf16_round(rng.uniform(-1.5, 1.5, size=H).astype(np.float32))
    if T > 2:
        x[1] = 0
        if residual:
            r[1] = 0
    return x, r, g


def _check_codes(codes, scale, y, err):
    """Each code's value times its scale is y, saturated at 448 scales, rounded to E4M3 (err: how far the kernel's y
    may be off). MXFP8's exponent leaves values between 448 and 512 scales to the saturation."""
    v = codecs.e4m3_decode(codes) * scale
    y = np.clip(y, -448 * scale, 448 * scale)
    assert np.all(np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) * 1.001 + err)


@pytest.mark.parametrize("T,H,residual,ue8m0", [(1, 128, False, False), (1, 7168, True, False), (5, 1024, True, True),
                                                (3, 1152, False, False), (67, 3584, True, False), (2, 8192, True, False),
                                                (9, 16384, True, True), (300, 256, False, False)])
def test_add_rmsnorm_fp8(fme, T, H, residual, ue8m0):
    x, r, g = _norm_inputs(T, H, T + H, residual)
    z, y = prompt.add_rmsnorm(x, r, g, 1e-5)
    bf = torch.bfloat16
    q, s, res, normed = fme.add_rmsnorm_fp8(_dev(x, bf), _dev(g, bf), None if r is None else _dev(r, bf), 1e-5, ue8m0,
                                            want_normed=True)
    assert (res is None) == (r is None)
    if res is not None:
        assert np.array_equal(_np(res), z)
    assert np.all(np.abs(_np(normed) - y) <= np.abs(y) * 2.0 ** -8 * 1.001)
    s = _np(s).astype(np.float64)
    amax = np.abs(y).reshape(T, H // 128, 128).max(-1)
    base = np.maximum(amax, 1e-10) / 448
    if ue8m0:
        base = np.maximum(base, 1e-10)
        assert np.array_equal(s, np.exp2(np.round(np.log2(s))))
        assert np.all(s >= base * (1 - 80 * U)) and np.all(s < 2 * base * (1 + 80 * U))
    else:
        assert np.all(np.abs(s - base) <= 70 * U * base)
    _check_codes(_np(q), np.repeat(s, 128, axis=1), y, 70 * U * np.abs(y))


@pytest.mark.parametrize("T,H,residual", [(1, 32, False), (4, 96, True), (33, 3584, True), (2, 7168, False),
                                          (3, 8224, True)])
def test_add_rmsnorm_mxfp8(fme, T, H, residual):
    x, r, g = _norm_inputs(T, H, 3 * T + H, residual)
    z, y = prompt.add_rmsnorm(x, r, g, 1e-5)
    bf = torch.bfloat16
    q, s, res, normed = fme.add_rmsnorm_mxfp8(_dev(x, bf), _dev(g, bf), None if r is None else _dev(r, bf), 1e-5)
    assert normed is None
    if r is not None:
        assert np.array_equal(_np(res), z)
    e = _np(s).astype(np.int64) - 127
    amax = np.abs(y).reshape(T, H // 32, 32).max(-1)
    low, high = (np.vectorize(mx_exponent)(amax * f) for f in (1 - 70 * U, 1 + 70 * U))
    assert np.all((e >= low) & (e <= high))
    _check_codes(_np(q), np.repeat(np.exp2(e.astype(np.float64)), 32, axis=1), y, 70 * U * np.abs(y))


def test_norm_strides_in_place_and_streams(fme):
    T, H = 37, 640
    x, r, g = _norm_inputs(T, H, 5, True)
    bf = torch.bfloat16
    dx, dr, dg = _dev(x, bf), _dev(r, bf), _dev(g, bf)
    ref = fme.add_rmsnorm_fp8(dx, dg, dr, want_normed=True)
    wide = torch.full((T, H + 24), float("nan"), dtype=bf, device=DEV)
    wide[:, 8:H + 8] = dx
    rwide = torch.full((T, 2 * H), float("nan"), dtype=bf, device=DEV)
    rwide[:, :H] = dr
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fme.add_rmsnorm_fp8(wide[:, 8:H + 8], dg, rwide[:, :H], want_normed=True)
        same = fme.add_rmsnorm_fp8(dx, dg, dr, want_normed=True, residual_out=dr)  # the residual updated in place
    side.synchronize()
    assert same[2] is dr
    for a, b, c in zip(ref, got, same):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_norm_bad_values_stay_in_their_row(fme):
    x, _, g = _norm_inputs(4, 512, 8, False)
    bf = torch.bfloat16
    dx, dg = _dev(x, bf), _dev(g, bf)
    ref = fme.add_rmsnorm_fp8(dx, dg, want_normed=True)
    bad = dx.clone()
    bad[0, 5] = float("nan")
    bad[2, 7] = float("inf")
    got = fme.add_rmsnorm_fp8(bad, dg, want_normed=True)
    for a, b in ((ref[0], got[0]), (ref[1], got[1]), (ref[3], got[3])):
        assert torch.equal(a[1::2], b[1::2])
    assert torch.isnan(got[3][0]).all()


def test_norm_offsets_past_32_bits(fme):
    H, ld, T = 256, 1 << 28, 10  # the last row starts 2.4e9 elements in
    g = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    buf = torch.zeros((T - 1) * ld + H, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((T, H), (ld, 1))
    x.copy_(torch.randn(T, H, device=DEV))
    a = fme.add_rmsnorm_fp8(x, g)
    b = fme.add_rmsnorm_fp8(x.contiguous(), g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --------------------------------------------------------------------------- route
@pytest.mark.parametrize("T,E,k,bf16,spread", [(1, 256, 8, True, 0.05), (1, 8, 8, False, 0.1), (65, 40, 3, True, 0.1),
                                               (333, 896, 16, False, 0.5), (2500, 256, 8, True, 0.05),
                                               (200, 1024, 32, False, 0.1), (9, 1, 1, False, 0.1)])
def test_route(fme, T, E, k, bf16, spread):
    rng = np.random.default_rng(T + E)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    if bf16:
        logits = codecs.bf16_round(logits)
    bias = rng.normal(size=E).astype(np.float32) * np.float32(spread)
    dl = _dev(logits, torch.bfloat16 if bf16 else None)
    ids, w, off, rows, tok = (_np(t) for t in fme.moe_route(dl, _dev(bias), k, 2.5))
    rid, rw, keys = routing.route(logits, bias, k, 2.5)
    assert_routing(ids, w, rid, rw, keys)
    for got, ref in zip((off, rows, tok), prompt.group_routes(ids, E)):
        assert np.array_equal(got, ref)


def test_route_ties_go_to_the_lower_expert(fme):
    T, E, k = 70, 48, 5
    logits = torch.zeros(T, E, device=DEV)
    logits[1::2, 40:43] = 1.0
    ids, w, off, rows, _ = fme.moe_route(logits, torch.zeros(E, device=DEV), k)
    assert ids[0].tolist() == [0, 1, 2, 3, 4] and ids[1].tolist() == [40, 41, 42, 0, 1]
    assert np.array_equal(_np(rows), prompt.group_routes(_np(ids), E)[1])
    assert torch.allclose(w.sum(1), torch.ones(T, device=DEV), atol=1e-6)


def test_route_picks_match_the_decode_kernel(fme):
    cfg, M = W.RAGGED, 33
    w13h, w2h = W.fp8_weights_host(cfg, 3)
    s13, s2 = W.fp8_weight_scales(cfg, 3)
    x, logits, bias = W.fp8_activations(cfg, M, 4)
    _, ids, w = fme.moe_routed_fp8(_dev(x, torch.bfloat16), _dev(logits), _dev(bias), _dev(w13h.full()), _dev(s13),
                                   _dev(w2h.full()), _dev(s2), cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0)
    got = fme.moe_route(_dev(logits), _dev(bias), cfg.top_k, cfg.scale)
    assert torch.equal(got[0], ids) and torch.equal(got[1], w)


def test_route_of_bad_logits_and_of_no_tokens(fme):
    T, E, k = 20, 40, 6
    logits = torch.randn(T, E, device=DEV)
    logits[3] = float("nan")
    logits[4] = -float("nan")
    logits[5] = -float("inf")
    logits[6, ::2] = float("inf")
    ids, _, off, rows, _ = fme.moe_route(logits, torch.zeros(E, device=DEV), k)
    a = _np(ids)
    assert a.min() >= 0 and a.max() < E and all(len(set(r)) == k for r in a.tolist())
    assert np.array_equal(_np(rows), prompt.group_routes(a, E)[1])
    assert a[6].tolist() == [0, 2, 4, 6, 8, 10]
    ids, w, off, rows, tok = fme.moe_route(logits[:0], torch.zeros(E, device=DEV), k)
    assert ids.shape == (0, k) and rows.numel() == 0 and not off.any()


def test_route_beside_other_streams_of_other_priorities(fme):
    """Launches whose CTAs meet, beside each other and beside work that holds SMs for a while: all meet."""
    T, E, k = 3000, 64, 4
    lg = [torch.randn(T, E, device=DEV) for _ in range(2)]
    bias = torch.zeros(E, device=DEV)
    x, gamma = torch.randn(8192, 4096, device=DEV).bfloat16(), torch.ones(4096, device=DEV).bfloat16()
    want = [fme.moe_route(t, bias, k) for t in lg]
    ws = [fme.Workspace(fme.moe_route_workspace(T, E, k), DEV) for _ in lg]
    low, high, busy = torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        with torch.cuda.stream(busy):
            fme.add_rmsnorm_fp8(x, gamma)
        for i, s in enumerate((low, high)):
            with torch.cuda.stream(s):
                got[i].append(fme.moe_route(lg[i], bias, k, workspace=ws[i]))
    torch.cuda.synchronize()
    assert [w.error() for w in ws] == [0, 0]
    for ref, runs in zip(want, got):
        assert all(torch.equal(a, b) for run in runs for a, b in zip(run, ref))


# --------------------------------------------------------------------------- grouped products
def _grouped_inputs(counts, H, N, a_rows, seed, gather, ue8m0=False):
    rng = np.random.default_rng(seed)
    E, R = len(counts), int(sum(counts))
    a, sa = quant.fp8_quant_mul(rng.normal(size=(a_rows, H)).astype(np.float32), ue8m0)
    w = codecs.e4m3_encode(rng.normal(size=(E, N, H)).astype(np.float32))
    sw = np.exp2(rng.uniform(-7, -3, size=(E, N // 128, H // 128))).astype(np.float32)
    off = np.cumsum([0] + list(counts)).astype(np.int32)
    idx = rng.integers(0, a_rows, size=R).astype(np.int32) if gather else None
    return a, sa, w, sw, off, idx


COUNTS = [([1], 1), ([3, 0, 1, 5], 2), ([128, 129, 0, 127], 3), ([0, 0, 300, 7, 0], 4), ([31, 33, 64, 2, 16, 17], 5),
          ([513], 6)]


@pytest.mark.parametrize("counts,seed", COUNTS)
@pytest.mark.parametrize("K,N", [(128, 128), (384, 384), (1024, 512)])
def test_grouped_gemm(fme, counts, seed, K, N):
    R = sum(counts)
    gather = seed % 2 == 0
    a, sa, w, sw, off, idx = _grouped_inputs(counts, K, N, max(R, 1) if not gather else 50, seed * 100 + K, gather)
    y, size = prompt.grouped_product(a, sa, w, sw, off, idx)
    tol = (K // 128 + 8) * 2 * U * size
    perm = np.random.default_rng(seed).permutation(R).astype(np.int32)
    out = fme.moe_grouped_gemm_fp8(_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off),
                                   in_rows=None if idx is None else _dev(idx), out_rows=_dev(perm))
    got = _np(out)[perm]
    assert np.all(np.abs(got - y) <= tol + np.abs(y) * 2.0 ** -8 * 1.001)
    again = fme.moe_grouped_gemm_fp8(_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off),
                                     in_rows=None if idx is None else _dev(idx))
    assert np.array_equal(_np(again), got)


@pytest.mark.parametrize("counts,seed", COUNTS)
@pytest.mark.parametrize("H,I,limit,ue8m0,gate_first", [(128, 128, 7.0, False, False), (512, 384, 0.5, True, False),
                                                        (1024, 256, float("inf"), False, True)])
def test_grouped_swiglu(fme, counts, seed, H, I, limit, ue8m0, gate_first):
    R = sum(counts)
    gather = seed % 2 == 1
    a, sa, w, sw, off, idx = _grouped_inputs(counts, H, 2 * I, max(R, 1) if not gather else 70, seed * 10 + H, gather)
    y, size = prompt.grouped_product(a, sa, w, sw, off, idx)
    up, gate = (y[:, I:], y[:, :I]) if gate_first else (y[:, :I], y[:, I:])
    su, sg = (size[:, I:], size[:, :I]) if gate_first else (size[:, :I], size[:, I:])
    h = clamped_swiglu(gate, up, limit)
    du, dg = ((H // 128 + 8) * 2 * U * v for v in (su, sg))
    g, u = np.minimum(gate, limit), np.clip(up, -limit, limit)
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 16 * U * np.abs(h)
    q, s = fme.moe_grouped_swiglu_fp8(_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off),
                                      in_rows=None if idx is None else _dev(idx), limit=limit, ue8m0=ue8m0,
                                      gate_first=gate_first)
    q, s = _np(q), _np(s).astype(np.float64)
    hb, db = (v.reshape(R, I // 128, 128) for v in (h, dh))
    base = np.maximum(np.abs(hb).max(-1), 1e-10) / 448
    slack = db.max(-1) / 448 + 4 * U * base
    if ue8m0:
        base = np.maximum(base, 1e-10)
        assert np.array_equal(s, np.exp2(np.round(np.log2(s))))
        assert np.all(s >= base - slack) and np.all(s < 2 * (base + slack))
    else:
        assert np.all(np.abs(s - base) <= slack)
    _check_codes(q, np.repeat(s, 128, axis=1), h, dh + 4 * U * np.abs(h))


def test_grouped_gemm_wide_tiles(fme):
    """Enough tiles for 256 output columns each, the last of them half a tile."""
    K, N = 128, 2176
    counts = [4100, 0, 1, 2500, 3399]
    a, sa, w, sw, off, _ = _grouped_inputs(counts, K, N, 10000, 77, False)
    y, size = prompt.grouped_product(a, sa, w, sw, off)
    got = _np(fme.moe_grouped_gemm_fp8(_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off)))
    assert np.all(np.abs(got - y) <= (K // 128 + 8) * 2 * U * size + np.abs(y) * 2.0 ** -8 * 1.001)


def test_grouped_long_launches(fme):
    """Enough tiles for CTAs in pairs: odd and even counts of row tiles, an odd count of weight tiles, the last of them
    half. The rows come from 50, so every expected row is one of 50 an expert."""
    counts = [7001, 0, 12999, 64]
    E, K, N, I, rows = len(counts), 128, 4224, 2048, 50
    off = np.cumsum([0] + counts).astype(np.int32)
    idx = np.random.default_rng(81).integers(0, rows, size=off[-1]).astype(np.int32)
    which = np.repeat(np.arange(E), counts) * rows + idx
    every = np.arange(E + 1, dtype=np.int32) * rows
    a, sa, w, sw, _, _ = _grouped_inputs([1] * E, K, N, rows, 82, False)
    y, size = prompt.grouped_product(a, sa, w, sw, every, np.tile(np.arange(rows), E))
    got = _np(fme.moe_grouped_gemm_fp8(_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off), in_rows=_dev(idx)))
    tol = (K // 128 + 8) * 2 * U * size + np.abs(y) * 2.0 ** -8 * 1.001
    first = np.array([np.flatnonzero(which == k)[0] if (which == k).any() else -1 for k in range(E * rows)])
    for k in np.flatnonzero(first >= 0):
        assert np.all(np.abs(got[first[k]] - y[k]) <= tol[k])
    assert np.array_equal(got, got[first[which]])  # equal rows give equal rows, wherever their tile ran

    w13, s13 = w[:, :2 * I], sw[:, :2 * I // 128]
    q, s = fme.moe_grouped_swiglu_fp8(_dev(a), _dev(sa), _dev(w13), _dev(s13), _dev(off), in_rows=_dev(idx), limit=7.0)
    q, s = _np(q), _np(s).astype(np.float64)
    up, gate, su, sg = y[:, :I], y[:, I:2 * I], size[:, :I], size[:, I:2 * I]
    h = clamped_swiglu(gate, up, 7.0)
    du, dg = ((K // 128 + 8) * 2 * U * v for v in (su, sg))
    g, u = np.minimum(gate, 7.0), np.clip(up, -7.0, 7.0)
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 16 * U * np.abs(h)
    for k in np.flatnonzero(first >= 0):
        base = np.maximum(np.abs(h[k]).reshape(-1, 128).max(-1), 1e-10) / 448
        assert np.all(np.abs(s[first[k]] - base) <= dh[k].reshape(-1, 128).max(-1) / 448 + 4 * U * base)
        _check_codes(q[first[k]], np.repeat(s[first[k]], 128), h[k], dh[k] + 4 * U * np.abs(h[k]))
    assert np.array_equal(q, q[first[which]]) and np.array_equal(s, s[first[which]])


@pytest.mark.parametrize("K", [640, 1024])
def test_grouped_long_launches_of_many_k_blocks(fme, K):
    """Hundreds of tiles a CTA, with and without four K blocks' scales in a 16-byte unit, rows by index and as whole
    boxes. The rows are 50, so every expected row is one of 50 an expert; the two forms of the input agree bit for bit."""
    counts = [7001, 0, 12999, 64]
    E, N, I, rows = len(counts), 4224, 2048, 50
    off = np.cumsum([0] + counts).astype(np.int32)
    idx = np.random.default_rng(83).integers(0, rows, size=off[-1]).astype(np.int32)
    which = np.repeat(np.arange(E), counts) * rows + idx
    a, sa, w, sw, _, _ = _grouped_inputs([1] * E, K, N, rows, 84, False)
    y, size = prompt.grouped_product(a, sa, w, sw, np.arange(E + 1, dtype=np.int32) * rows, np.tile(np.arange(rows), E))
    da, dsa, dw, dsw, doff, didx = _dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off), _dev(idx)
    got = fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, doff, in_rows=didx)
    boxes = fme.moe_grouped_gemm_fp8(da[didx.long()], dsa[didx.long()], dw, dsw, doff)
    assert torch.equal(got, boxes)
    got = _np(got)
    first = np.array([np.flatnonzero(which == k)[0] if (which == k).any() else -1 for k in range(E * rows)])
    tol = (K // 128 + 8) * 2 * U * size + np.abs(y) * 2.0 ** -8 * 1.001
    for k in np.flatnonzero(first >= 0):
        assert np.all(np.abs(got[first[k]] - y[k]) <= tol[k])
    assert np.array_equal(got, got[first[which]])

    w13, s13 = dw[:, :2 * I].contiguous(), dsw[:, :2 * I // 128].contiguous()
    q, s = fme.moe_grouped_swiglu_fp8(da, dsa, w13, s13, doff, in_rows=didx, limit=7.0)
    qb, sb = fme.moe_grouped_swiglu_fp8(da[didx.long()], dsa[didx.long()], w13, s13, doff, limit=7.0)
    assert torch.equal(q, qb) and torch.equal(s, sb)
    q, s = _np(q), _np(s).astype(np.float64)
    up, gate, su, sg = y[:, :I], y[:, I:2 * I], size[:, :I], size[:, I:2 * I]
    h = clamped_swiglu(gate, up, 7.0)
    du, dg = ((K // 128 + 8) * 2 * U * v for v in (su, sg))
    g, u = np.minimum(gate, 7.0), np.clip(up, -7.0, 7.0)
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 16 * U * np.abs(h)
    for k in np.flatnonzero(first >= 0):
        base = np.maximum(np.abs(h[k]).reshape(-1, 128).max(-1), 1e-10) / 448
        assert np.all(np.abs(s[first[k]] - base) <= dh[k].reshape(-1, 128).max(-1) / 448 + 4 * U * base)
        _check_codes(q[first[k]], np.repeat(s[first[k]], 128), h[k], dh[k] + 4 * U * np.abs(h[k]))
    assert np.array_equal(q, q[first[which]]) and np.array_equal(s, s[first[which]])


def test_grouped_outputs_at_any_16_bytes(fme):
    a, sa, w, sw, off, _ = _grouped_inputs([70, 60], 256, 384, 130, 78, False)
    args = (_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off))
    ref = fme.moe_grouped_gemm_fp8(*args)
    buf = torch.zeros(130 * 384 + 8, dtype=torch.bfloat16, device=DEV)
    out = buf[8:].view(130, 384)  # 16 bytes past an allocation's start
    assert out.data_ptr() % 32 == 16
    fme.moe_grouped_gemm_fp8(*args, out=out)
    assert torch.equal(out, ref) and not buf[:8].any()


def test_grouped_many_groups(fme):
    """1024 groups, most of them empty, K blocks that are no multiple of four."""
    E, K, N = 1024, 384, 128
    rng = np.random.default_rng(79)
    counts = np.zeros(E, int)
    counts[rng.choice(E, 40, replace=False)] = rng.integers(1, 140, size=40)
    counts[-1] = 5
    a, sa, w, sw, off, idx = _grouped_inputs(counts, K, N, 60, 80, True)
    y, size = prompt.grouped_product(a, sa, w, sw, off, idx)
    got = _np(fme.moe_grouped_gemm_fp8(_dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off), in_rows=_dev(idx)))
    assert np.all(np.abs(got - y) <= (K // 128 + 8) * 2 * U * size + np.abs(y) * 2.0 ** -8 * 1.001)


def test_grouped_offsets_rows_and_errors(fme):
    """Places outside every group stay as they are; offsets out of range are clamped; a bad index gives zeros or is
    skipped, and is reported; NaN codes stay in their row."""
    K, N = 256, 256
    a, sa, w, sw, _, _ = _grouped_inputs([40, 40], K, N, 90, 9, False)
    da, dsa, dw, dsw = _dev(a), _dev(sa), _dev(w), _dev(sw)
    ws = fme.Workspace(fme.moe_grouped_fp8_workspace(90, K, N, 2), DEV)

    def off(*v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    full = fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, off(0, 40, 80), workspace=ws)
    out = torch.full((90, N), 7.0, dtype=torch.bfloat16, device=DEV)
    fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, off(10, 40, 75), out=out, workspace=ws)
    assert torch.equal(out[10:75], full[10:75]) and (out[:10] == 7).all() and (out[75:] == 7).all()
    out.fill_(7.0)
    fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, off(-5, 40, 100000), out=out, workspace=ws)
    assert torch.equal(out[:80], full[:80])
    fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, off(60, 20, 10), out=out, workspace=ws)  # descending: nothing
    assert ws.error() == 0
    idx = torch.arange(90, dtype=torch.int32, device=DEV)
    idx[3], idx[50] = -1, 90
    got = fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, off(0, 40, 80), in_rows=idx, workspace=ws)
    assert ws.error() == 8
    keep = [i for i in range(80) if i not in (3, 50)]
    assert torch.equal(got[keep], full[keep]) and (got[3] == 0).all() and (got[50] == 0).all()
    out.fill_(7.0)
    fme.moe_grouped_gemm_fp8(da, dsa, dw, dsw, off(0, 40, 80), out_rows=idx, out=out, workspace=ws)
    assert ws.error() == 8
    assert torch.equal(out[keep], full[keep]) and (out[3] == 7).all() and (out[50] == 7).all()
    q, s = fme.moe_grouped_swiglu_fp8(da, dsa, dw, dsw, off(0, 40, 80), in_rows=idx, limit=7.0, workspace=ws)
    assert ws.error() == 8 and (q[3] == 0).all() and (s[3] > 0).all()
    bad = da.clone()
    bad[7] = 0x7F
    got = fme.moe_grouped_gemm_fp8(bad, dsa, dw, dsw, off(0, 40, 80), workspace=ws)
    keep = [i for i in range(80) if i != 7]
    assert torch.equal(got[keep], full[keep]) and torch.isnan(got[7]).all() and ws.error() == 0


def test_grouped_no_rows_and_far_output_rows(fme):
    K, N = 128, 7168
    a, sa, w, sw, off, _ = _grouped_inputs([3, 2], K, N, 5, 11, False)
    args = (_dev(a), _dev(sa), _dev(w), _dev(sw))
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert fme.moe_grouped_gemm_fp8(*args, torch.zeros(3, dtype=torch.int32, device=DEV), in_rows=none).shape == (0, N)
    ref = fme.moe_grouped_gemm_fp8(*args, _dev(off))
    far = torch.zeros(620000, N, dtype=torch.bfloat16, device=DEV)  # 4.4e9 elements
    rows = torch.tensor([619999, 0, 300000, 599999, 5], dtype=torch.int32, device=DEV)
    fme.moe_grouped_gemm_fp8(*args, _dev(off), out_rows=rows, out=far)
    assert torch.equal(far[rows.long()], ref)
    assert int((far != 0).any(1).sum()) == 5


# --------------------------------------------------------------------------- together
def _layer(cfg, seed):
    w13h, w2h = W.fp8_weights_host(cfg, seed)
    s13, s2 = W.fp8_weight_scales(cfg, seed)
    return [_dev(v) for v in (w13h.full(), s13, w2h.full(), s2)]


def test_prompt_layer_matches_the_decode_layer(fme):
    """The same tokens, quantised the same, through the decode kernel and the prompt operators: picks and weights bit
    for bit, combined rows within the decode kernel's own tolerance of each other."""
    cfg, M = W.RAGGED, 60
    weights = _layer(cfg, 21)
    x, logits, bias = W.fp8_activations(cfg, M, 22)
    codes, sx = quant.fp8_quant_mul(x, cfg.ue8m0)
    routed = (cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0)
    out, ids, wts = fme.moe_routed_fp8(_dev(x, torch.bfloat16), _dev(logits), _dev(bias), *weights, *routed)
    y, pid, pw = fme.moe_prompt_fp8(_dev(codes), _dev(sx), _dev(logits), _dev(bias), *weights, *routed)
    assert torch.equal(ids, pid) and torch.equal(wts, pw)
    assert_outputs(_np(y), _np(fme.moe_finalize(out, wts)), "prompt against decode")
    assert np.array_equal(_np(fme.moe_finalize(out, wts)), oracle_finalize(_np(out), _np(wts)))


def test_prompt_operators_in_a_graph(fme):
    cfg, T = W.RAGGED, 150
    w13, s13, w2, s2 = _layer(cfg, 31)
    gamma = torch.ones(cfg.H, dtype=torch.bfloat16, device=DEV)
    x = torch.randn(T, cfg.H, device=DEV).bfloat16()
    logits = torch.randn(T, cfg.E, device=DEV)
    bias = torch.zeros(cfg.E, device=DEV)
    y = torch.empty(T, cfg.H, dtype=torch.bfloat16, device=DEV)
    R = T * cfg.top_k
    ws = [fme.Workspace(n, DEV) for n in (fme.moe_route_workspace(T, cfg.E, cfg.top_k),
                                          fme.moe_grouped_fp8_workspace(R, cfg.H, 2 * cfg.I, cfg.E),
                                          fme.moe_grouped_fp8_workspace(R, cfg.I, cfg.H, cfg.E))]

    def step(y=None):
        q, s, _, _ = fme.add_rmsnorm_fp8(x, gamma)
        _, wt, off, rows, tok = fme.moe_route(logits, bias, cfg.top_k, cfg.scale, workspace=ws[0])
        hq, sh = fme.moe_grouped_swiglu_fp8(q, s, w13, s13, off, in_rows=tok, limit=cfg.limit, workspace=ws[1])
        out = fme.moe_grouped_gemm_fp8(hq, sh, w2, s2, off, out_rows=rows, workspace=ws[2])
        return fme.moe_finalize(out, wt, y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(y)
    for _ in range(3):
        x.normal_()
        logits.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step())
    assert [w.error() for w in ws] == [0, 0, 0]


def test_streams_have_workspaces_of_their_own(fme):
    """Calls of two streams that overlap share nothing the binding keeps."""
    lg = [torch.randn(3000, 256, device=DEV) for _ in range(2)]
    bias = torch.zeros(256, device=DEV)
    ref = [fme.moe_route(v, bias, 8) for v in lg]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lg]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fme.moe_route(lg[i], bias, 8))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, ref[i]))


def test_prompt_layer_example(fme):
    """The example's layer against the decode layer. They quantise norms that are one BF16 rounding apart (2^-9 of a
    value and of a block's scale): about one E4M3 code in fifty differs, a percent of the tokens' norm; the hidden
    values, 1.6 percent apart, differ in a code in six, which makes 3 to 4 percent of an output (an E4M3 rounding
    alone is 2.6). Unrelated outputs are more than 100 apart."""
    import importlib.util
    import os
    import sys

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prompt_layer.py")
    spec = importlib.util.spec_from_file_location("prompt_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    argv, sys.argv = sys.argv, [path, "--tokens", "333"]
    try:
        assert mod.main() < 0.05
    finally:
        sys.argv = argv


def test_prompt_layer_without_tokens_and_captured_without_workspaces(fme):
    cfg, T = W.RAGGED, 40
    weights = _layer(cfg, 41)
    routed = (cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0)
    q = torch.randint(0, 0x7F, (T, cfg.H), dtype=torch.uint8, device=DEV)
    s = torch.rand(T, cfg.H // 128, device=DEV) * 2.0 ** -8
    logits, bias = torch.randn(T, cfg.E, device=DEV), torch.zeros(cfg.E, device=DEV)
    y, ids, _ = fme.moe_prompt_fp8(q[:0], s[:0], logits[:0], bias, *weights, *routed)
    assert y.shape == (0, cfg.H) and y.dtype == torch.bfloat16 and ids.shape == (0, cfg.top_k)
    torch.cuda.synchronize()
    kept = dict(fme._ws_cache)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _, _ = fme.moe_prompt_fp8(q, s, logits, bias, *weights, *routed)
    assert set(fme._ws_cache) == set(kept)  # nothing of the graph's memory is kept for other calls
    for _ in range(3):
        logits.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, fme.moe_prompt_fp8(q, s, logits, bias, *weights, *routed)[0])


def test_prompt_layer_refuses_operands_that_disagree(fme):
    """Tokens and logits of different counts, and weights of another shape, are refused before anything runs."""
    cfg, T = W.RAGGED, 20
    w13, s13, w2, s2 = _layer(cfg, 51)
    q = torch.zeros(T, cfg.H, dtype=torch.uint8, device=DEV)
    s = torch.ones(T, cfg.H // 128, device=DEV)
    lg, bias = torch.randn(T, cfg.E, device=DEV), torch.zeros(cfg.E, device=DEV)
    shared = torch.zeros(T, cfg.H, dtype=torch.bfloat16, device=DEV)
    good = dict(xq=q, sx=s, logits=lg, bias=bias, w13=w13, s13=s13, w2=w2, s2=s2, top_k=cfg.top_k, limit=cfg.limit,
                scale=cfg.scale, ue8m0=cfg.ue8m0, shared_out=shared)
    fme.moe_prompt_fp8(**good)
    for name, t in (("logits", lg[:-1]), ("logits", torch.cat([lg, lg[:1]])), ("logits", lg[0]), ("sx", s[1:]),
                    ("bias", bias[1:]), ("w13", w13[1:]), ("w13", w13[:, :-256].contiguous()),
                    ("w2", w2[:, :-128].contiguous()), ("w2", w2[1:]), ("shared_out", shared[1:])):
        with pytest.raises(ValueError, match="expected"):
            fme.moe_prompt_fp8(**{**good, name: t})
    few = {**good, "xq": q[:-1], "sx": s[:-1]}
    with pytest.raises(ValueError, match="logits"):
        fme.moe_prompt_fp8(**few)


@pytest.mark.parametrize("limit", [7.0, float("inf")])
def test_grouped_swiglu_keeps_nan(fme, limit):
    """A NaN token, token scale, gate weight or up weight makes NaN codes where it enters, and nothing else changes."""
    H, I, R = 256, 256, 40
    a, sa, w, sw, off, _ = _grouped_inputs([25, 15], H, 2 * I, R, 91, False)
    da, dsa, dw, dsw, doff = _dev(a), _dev(sa), _dev(w), _dev(sw), _dev(off)
    q, s = fme.moe_grouped_swiglu_fp8(da, dsa, dw, dsw, doff, limit=limit)
    assert not ((q & 0x7F) == 0x7F).any()
    bad, bad_s = da.clone(), dsa.clone()
    bad[3, 17] = 0x7F
    bad_s[30, 1] = float("nan")
    qt, st = fme.moe_grouped_swiglu_fp8(bad, bad_s, dw, dsw, doff, limit=limit)
    keep = [i for i in range(R) if i not in (3, 30)]
    assert torch.equal(qt[keep], q[keep]) and torch.equal(st[keep], s[keep])
    assert ((qt[[3, 30]] & 0x7F) == 0x7F).all()
    wb = dw.clone()
    wb[0, 5, 100] = 0xFF       # up row 5 of the first expert
    wb[1, I + 140, 9] = 0x7F   # gate row 140 of the second
    qw, _ = fme.moe_grouped_swiglu_fp8(da, dsa, wb, dsw, doff, limit=limit)
    nan = (qw & 0x7F) == 0x7F
    assert nan[:25, 5].all() and nan[25:, 140].all() and int(nan.sum()) == R
    assert torch.equal(qw[:25, 128:], q[:25, 128:]) and torch.equal(qw[25:, :128], q[25:, :128])


def test_finalize_of_the_longest_prompt(fme):
    """2^20 tokens of 16384 values, more 16-byte items than 31 bits count: every row is combined."""
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("needs 70 GB")
    T, H = 1 << 20, 16384
    out = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    w = (torch.arange(T, device=DEV) % 251 + 1).float()[:, None]
    y = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    fme.moe_finalize(out, w, y=y)
    for part in range(0, T, 1 << 16):
        assert (y[part:part + (1 << 16)] == w[part:part + (1 << 16)].bfloat16()).all()
    del out, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 3), (64, 8), (65, 8), (200, 32), (256, 8), (257, 5), (512, 8), (513, 16),
                                 (896, 16), (1024, 32)])
def test_route_equals_the_decode_kernel_bit_for_bit(fme, E, k, bf16):
    """Picks and weights of one long call against the decode kernel's of 64 tokens each: ordinary logits, logits whose
    scores saturate or underflow, equal logits, and infinities."""
    H, I, T = 128, 128, 320
    g = torch.Generator(device=DEV).manual_seed(E + k)
    logits = torch.randn(T, E, generator=g, device=DEV)
    logits[64:128] *= 40.0
    logits[128:192] = logits[128:192].round()
    logits[192:200] = 0.25
    logits[200:208] -= 87.0
    logits[208:212, ::3] = float("inf")
    logits[212:216, ::2] = -float("inf")
    logits[216:220] = -200.0
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    if bf16:
        logits = logits.bfloat16()
    zeros = [torch.zeros(s, dtype=d, device=DEV) for s, d in (((E, 2 * I, H), torch.uint8), ((E, 2, 1), torch.float32),
                                                               ((E, H, I), torch.uint8), ((E, 1, 1), torch.float32))]
    x = torch.zeros(64, H, dtype=torch.bfloat16, device=DEV)
    ids, w = fme.moe_route(logits, bias, k, 2.5)[:2]
    for t in range(0, T, 64):
        _, di, dw = fme.moe_routed_fp8(x, logits[t:t + 64], bias, *zeros, k, 7.0, 2.5, False)
        assert torch.equal(ids[t:t + 64], di)
        assert torch.equal(w[t:t + 64].nan_to_num(-1.0).view(torch.int32), dw.nan_to_num(-1.0).view(torch.int32))
