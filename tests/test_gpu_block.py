"""GPU checks of the operators around a routed block (dense product, group-limited routing, the norms between blocks)
against the 64-bit oracle, whose functions give the bounds of FP32 arithmetic; an output's own rounding adds 2^-8 (BF16)
or 2^-24 (FP32) of it, an E4M3 code 2^-4 (2^-10 of the scale below 2^-6 of it).
"""

import numpy as np
import pytest
import torch

from oracle import codecs, linear as oracle_linear, prompt, routing
from oracle.ep_local import mx_exponent
from oracle.finalize import finalize as oracle_finalize
from oracle.routing import route_groups as routing_oracle
from synth import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.float().cpu().numpy() if t.dtype == BF else t.cpu().numpy()


def _bf(rng, *shape):
    return codecs.bf16_round(rng.normal(size=shape).astype(np.float32))


def _wide(a, pad, fill=float("nan")):
    """BF16 rows of a in a buffer of rows that are whole 16-byte units and `pad` values longer; the gaps hold `fill`."""
    n, k = a.shape
    buf = torch.full((n, (k + 7) // 8 * 8 + pad), fill, dtype=BF, device=DEV)
    buf[:, :k] = _dev(a, BF)
    return buf[:, :k]


# --------------------------------------------------------------------------- linear
def _check_linear(fme, M, N, K, bias, act, residual, f32, pad=0, seed=0, ws=None):
    rng = np.random.default_rng([M, N, K, seed])
    x, w = _bf(rng, M, K), _bf(rng, N, K) / np.float32(max(1, int(np.sqrt(K))))
    w = codecs.bf16_round(w.astype(np.float32))
    b = rng.normal(size=N).astype(np.float32) if bias else None
    r = None
    if residual:
        r = rng.normal(size=(M, N)).astype(np.float32)
        r = r if f32 else codecs.bf16_round(r)
    dt = torch.float32 if f32 else BF
    y, tol = oracle_linear.linear(x, w, b, act, r)
    out = fme.linear_bf16(_wide(x, pad), _wide(w, pad), None if b is None else _dev(b), act,
                          None if r is None else _dev(r, dt), out_dtype=dt, workspace=ws)
    assert out.dtype == dt and out.shape == (M, N)
    got = _np(out).astype(np.float64)
    tol = tol + np.abs(y) * (U if f32 else 2.0 ** -8) * 1.001
    assert np.all(np.abs(got - y) <= tol), float(np.max(np.abs(got - y) / tol))
    return out


ACTS = [None, "relu", "silu", "gelu", "sigmoid"]


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("N,K,pad", [(1, 1, 0), (256, 7168, 0), (7, 1003, 8), (515, 136, 0), (40, 1024, 16), (1, 4097, 0)])
def test_linear_of_few_tokens(fme, M, N, K, pad):
    i = M + N
    _check_linear(fme, M, N, K, i % 2 == 0, ACTS[i % 5], i % 3 == 0, i % 2 == 1, pad)


@pytest.mark.parametrize("M", [9, 16, 31, 64, 100, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K,pad", [(1, 8, 0), (16, 64, 0), (17, 63, 8), (255, 200, 0), (256, 1024, 0), (257, 65, 24),
                                     (640, 2048, 0), (1100, 129, 0)])
def test_linear(fme, M, N, K, pad):
    i = M + N
    _check_linear(fme, M, N, K, i % 2 == 0, ACTS[i % 5], i % 3 == 0, i % 4 == 1, pad)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,f32", [(3, False), (3, True), (50, False), (50, True), (2000, False), (2000, True)])
def test_linear_activations(fme, act, M, f32):
    _check_linear(fme, M, 272, 320, True, act, True, f32)


@pytest.mark.parametrize("M,N,K", [(64, 256, 7168), (1533, 895, 3581), (2500, 2048, 512), (64, 7168, 2048), (700, 8, 7168),
                                   (5000, 1280, 256)])
def test_linear_larger(fme, M, N, K):
    ws = fme.Workspace(fme.linear_bf16_workspace(M, N, K), DEV)
    first = _check_linear(fme, M, N, K, True, "silu", True, False, ws=ws)
    again = _check_linear(fme, M, N, K, True, "silu", True, False, ws=ws)  # the counters are back at zero
    assert torch.equal(first, again) and ws.error() == 0


def test_linear_is_the_same_bits_every_time(fme):
    for M, N, K in ((5, 300, 4000), (64, 256, 7168), (300, 500, 2000)):
        x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
        ref = fme.linear_bf16(x, w, out_dtype=torch.float32)
        for _ in range(20):
            assert torch.equal(ref, fme.linear_bf16(x, w, out_dtype=torch.float32))


def test_linear_cut_products_of_one_workspace(fme):
    """FP32 sums in one and several accumulations, K cut and not, ragged and residual, in turn on one workspace."""
    shapes = [(17, 256, 7168), (512, 256, 7168), (129, 250, 6999), (2048, 256, 7168), (70, 3000, 4096), (300, 896, 3584),
              (64, 48, 16384)]
    ws = fme.Workspace(max(fme.linear_bf16_workspace(*shape) for shape in shapes), DEV)
    first = {}
    for again in range(2):
        for i, (M, N, K) in enumerate(shapes):
            for f32 in (True, False):
                out = _check_linear(fme, M, N, K, i % 2 == 0, ACTS[i % 5], i % 3 != 0, f32, ws=ws) if not again else None
                x, w = (torch.ones(n, (K + 7) // 8 * 8, device=DEV, dtype=BF)[:, :K] for n in (M, N))
                x[::3] = 0.5
                y = fme.linear_bf16(x, w, out_dtype=torch.float32, workspace=ws)
                assert torch.equal(y, x[:, :1].float() * K * torch.ones(1, N, device=DEV))
                if out is not None:
                    first[M, N, K, f32] = out
                else:
                    out = _check_linear(fme, M, N, K, i % 2 == 0, ACTS[i % 5], i % 3 != 0, f32, ws=ws)
                    assert torch.equal(first[M, N, K, f32], out)
    assert ws.error() == 0


def test_linear_reports_a_workspace_that_was_not_cleared(fme):
    M, N, K = 64, 256, 7168  # K is cut: units count their arrivals in the workspace
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
    ws = fme.Workspace(fme.linear_bf16_workspace(M, N, K), DEV)
    assert ws.nbytes > 4096
    ref = fme.linear_bf16(x, w, workspace=ws)
    assert ws.error() == 0
    ws.buf[256:4096] = 0x7F
    fme.linear_bf16(x, w, workspace=ws)
    assert ws.error() == 2
    ws.clear()
    assert torch.equal(fme.linear_bf16(x, w, workspace=ws), ref) and ws.error() == 0


@pytest.mark.parametrize("M", [4, 70, 400])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_strided_outputs(fme, M, f32):
    """Output rows at any stride and alignment hold what dense ones do, and nothing beside them changes; out may be the
    residual, or columns of the buffer that x is columns of."""
    N, K, dt = 272, 192, torch.float32 if f32 else BF
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
    b, r = torch.randn(N, device=DEV), torch.randn(M, N, device=DEV).to(dt)
    ref = fme.linear_bf16(x, w, b, "silu", r, out_dtype=dt)
    for lead, extra in ((0, 16), (1, 3), (8, 8), (0, 1)):
        buf = torch.full((M, lead + N + extra), 7.0, dtype=dt, device=DEV)
        out = buf[:, lead:lead + N]
        assert fme.linear_bf16(x, w, b, "silu", r, out=out) is out
        assert torch.equal(out, ref) and (buf[:, :lead] == 7).all() and (buf[:, lead + N:] == 7).all()
        out.copy_(r)
        fme.linear_bf16(x, w, b, "silu", out, out=out)
        assert torch.equal(out, ref)
    if not f32:
        buf = torch.zeros(M, K + N, dtype=BF, device=DEV)
        buf[:, :K] = x
        fme.linear_bf16(buf[:, :K], w, b, "silu", r, out=buf[:, K:])
        assert torch.equal(buf[:, K:], ref) and torch.equal(buf[:, :K], x)


@pytest.mark.parametrize("M", [6, 90, 2100])
def test_linear_bad_values_stay_in_their_row_and_column(fme, M):
    N, K = 144, 200
    x, w = torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)
    for act in ACTS:
        ref = fme.linear_bf16(x, w, None, act)
        bx, bw = x.clone(), w.clone()
        bx[2, 5], bw[3, 7], bw[140, 1] = float("nan"), float("inf"), float("nan")
        got = fme.linear_bf16(bx, bw, None, act)
        rows = [i for i in range(M) if i != 2]
        cols = [i for i in range(N) if i not in (3, 140)]
        assert torch.equal(got[rows][:, cols], ref[rows][:, cols])
        assert torch.isnan(got[2]).all() and torch.isnan(got[:, 140]).all()


def test_linear_no_tokens_and_far_rows(fme):
    w = torch.randn(24, 64, device=DEV).to(BF)
    assert fme.linear_bf16(torch.empty(0, 64, dtype=BF, device=DEV), w).shape == (0, 24)
    for M in (6, 40):
        ld = (1 << 31) // (M - 1) + 8 & ~7  # the last row starts past 2^31 values
        buf = torch.zeros((M - 1) * ld + 64, dtype=BF, device=DEV)
        x = buf.as_strided((M, 64), (ld, 1))
        x.copy_(torch.randn(M, 64, device=DEV))
        far = torch.zeros((M - 1) * ld + 24, dtype=BF, device=DEV)
        out = far.as_strided((M, 24), (ld, 1))
        ref = fme.linear_bf16(x.contiguous(), w)
        assert torch.equal(fme.linear_bf16(x, w, out=out), ref)
        assert int(torch.count_nonzero(far)) == int(torch.count_nonzero(ref))
        del buf, x, far, out


def test_linear_many_tokens(fme):
    """2^20 rows, more than 2^31 output values; the rows come from 50."""
    M, N, K = 1 << 20, 2064, 24
    few = torch.randn(50, K, device=DEV).to(BF)
    w, b = torch.randn(N, K, device=DEV).to(BF), torch.randn(N, device=DEV)
    which = torch.randint(0, 50, (M,), device=DEV)
    got = fme.linear_bf16(few[which], w, b)
    ref = got[torch.stack([(which == i).nonzero()[0, 0] for i in range(50)])]
    y, tol = oracle_linear.linear(_np(few), _np(w), _np(b))
    assert np.all(np.abs(_np(ref) - y) <= tol + np.abs(y) * 2.0 ** -8 * 1.001)
    for i in range(0, M, 1 << 18):
        assert torch.equal(got[i:i + (1 << 18)], ref[which[i:i + (1 << 18)]])


# --------------------------------------------------------------------------- route
def _check_route(fme, T, E, k, bf16, seed, bias_spread, most_excused=0.05, **kw):
    rng = np.random.default_rng([T, E, seed])
    logits = (1.5 * rng.normal(size=(T, E))).astype(np.float32)
    if bf16:
        logits = codecs.bf16_round(logits)
    bias = None if bias_spread is None else (bias_spread * rng.normal(size=E)).astype(np.float32)
    ids, w, off, rows, tok = (_np(t) for t in fme.moe_route_groups(
        _dev(logits, BF if bf16 else None), None if bias is None else _dev(bias), k, scale=2.5, **kw))
    kw.setdefault("groups", 1)
    kw.setdefault("top_groups", kw["groups"])
    kw.setdefault("group_top", 2 if E >= 2 * kw["groups"] else 1)
    rid, rw, gaps = routing.route_groups(logits, bias, k, scale=2.5, **kw)
    # FP32 scores, sums of two and biased keys are within 16 u; a token whose deciding gap is below that may differ.
    sure = gaps > 32 * U
    assert sure.mean() >= 1 - most_excused
    assert np.array_equal(ids[sure], rid[sure])
    assert np.all((ids >= 0) & (ids < E)) and all(len(set(r)) == k for r in ids.tolist())
    # A weight: exp within 2 u and its argument's rounding (u of |l - max| <= 16), sums of 1024 terms in trees, k picks.
    assert np.all(np.abs(w - rw)[sure] <= (64 + k) * U * np.abs(rw)[sure])
    for got, ref in zip((off, rows, tok), prompt.group_routes(ids, E)):
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", [
    (1, 256, 8, 8, 4, 2), (300, 256, 8, 8, 4, 2), (65, 40, 3, 5, 2, 1), (33, 40, 3, 8, 5, 2), (70, 64, 6, 32, 9, 2),
    (40, 384, 6, 8, 3, 2), (50, 896, 16, 7, 2, 2), (21, 1024, 32, 16, 1, 1), (9, 6, 2, 6, 3, 1), (90, 256, 8, 1, 1, 1),
    (30, 510, 4, 17, 5, 2), (200, 256, 8, 16, 16, 2), (50, 896, 4, 8, 3, 2)])
def test_route_groups(fme, score, T, E, k, groups, top_groups, group_top):
    for i, (bias, bf16) in enumerate(((0.1, False), (None, False), (0.5, True))):
        _check_route(fme, T, E, k, bf16, i, bias, score=score, groups=groups, top_groups=top_groups, group_top=group_top,
                     renormalise=i != 1)


def test_route_groups_defaults_and_long(fme):
    _check_route(fme, 5000, 256, 8, True, 3, 0.05, score="sigmoid", groups=8, top_groups=4)
    _check_route(fme, 1533, 896, 16, False, 4, 0.5, score="softmax", renormalise=False)
    _check_route(fme, 7, 3, 2, False, 5, None)


def test_route_groups_equals_route_without_groups(fme):
    for T, E, k in ((1, 256, 8), (700, 256, 8), (333, 896, 16), (40, 40, 3)):
        logits, bias = torch.randn(T, E, device=DEV), 0.1 * torch.randn(E, device=DEV)
        for lg in (logits, logits.to(BF)):
            a, b = fme.moe_route(lg, bias, k, 2.5), fme.moe_route_groups(lg, bias, k, scale=2.5)
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", [
    (40, 896, 16, 8, 1, 2), (40, 896, 32, 8, 2, 1), (25, 500, 20, 10, 1, 2), (33, 1000, 32, 8, 1, 2), (31, 130, 8, 13, 4, 2),
    (20, 1022, 5, 14, 6, 2), (18, 257, 9, 1, 1, 1), (50, 258, 31, 6, 5, 2), (2000, 999, 7, 27, 9, 2)])
def test_route_groups_in_few_lanes_or_across_two(fme, T, E, k, groups, top_groups, group_top):
    for i, (score, bias, bf16) in enumerate((("softmax", 0.1, False), ("sigmoid", 0.3, True))):
        _check_route(fme, T, E, k, bf16, i, bias, score=score, groups=groups, top_groups=top_groups, group_top=group_top)


def test_route_groups_more_equal_keys_than_lanes(fme):
    for E, k in ((896, 16), (256, 8), (1000, 32), (64, 32)):
        top = list(range(5, E, max(1, E // 45)))[:40]
        logits = torch.zeros(3, E, device=DEV)
        logits[1, top] = 1.0
        logits[2, top[:3]] = 1.0
        rest = [e for e in range(E) if e not in top[:3]]
        for ids in (fme.moe_route_groups(logits, None, k)[0], fme.moe_route(logits, torch.zeros(E, device=DEV), k)[0]):
            assert ids[0].tolist() == list(range(k))
            assert ids[1].tolist() == top[:k]
            assert ids[2].tolist() == (top[:3] + rest)[:k]


def test_route_of_more_tokens_than_16_bits_count(fme):
    T, E = 66000, 24
    logits = torch.zeros(T, E, device=DEV)
    logits[:, 3] = 2.0
    second = torch.arange(T, device=DEV) * 7 % 20 + 4
    logits[torch.arange(T, device=DEV), second] = 1.0
    ids, _, off, rows, tok = (_np(t) for t in fme.moe_route(logits, torch.zeros(E, device=DEV), 2))
    assert np.all(ids[:, 0] == 3) and np.array_equal(ids[:, 1], _np(second))
    assert off[4] - off[3] == T
    for got, ref in zip((off, rows, tok), prompt.group_routes(ids, E)):
        assert np.array_equal(got, ref)


def test_route_groups_ties(fme):
    T, E, k = 70, 48, 5
    logits = torch.zeros(T, E, device=DEV)
    logits[1::2, 40:43] = 1.0
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.zeros(E, device=DEV)):
            ids = fme.moe_route_groups(logits, bias, k, score, groups=4, top_groups=2)[0]
            assert ids[0].tolist() == [0, 1, 2, 3, 4] and ids[1].tolist() == [40, 41, 42, 0, 1]
    # Without a bias saturated and underflowed scores still differ by their logits.
    lg = torch.zeros(2, 64, device=DEV)
    lg[0, 60], lg[0, 7], lg[0, 33] = 40.0, 30.0, 35.0
    lg[1] = -200 - torch.arange(64, device=DEV) % 7 * 1.0
    lg[1, 5] = 0
    ids = fme.moe_route_groups(lg, None, 3, "sigmoid")[0]
    assert ids[0].tolist() == [60, 33, 7]
    ids, w, _, _, _ = fme.moe_route_groups(lg, None, 3, "softmax")
    assert ids[1].tolist() == [5, 0, 7] and w[1].tolist() == [1.0, 0.0, 0.0]
    ids = fme.moe_route_groups(lg, None, 3, "sigmoid", groups=4, top_groups=1, group_top=1)[0]
    assert ids[0].tolist() == [60, 48, 49]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_groups_of_bad_logits(fme, score, bias):
    T, E, k = 40, 40, 6
    logits = torch.randn(T, E, device=DEV)
    logits[3] = float("nan")
    logits[4] = -float("nan")
    logits[5] = -float("inf")
    logits[6, ::2] = float("inf")
    logits[7, 5] = float("nan")
    logits[8] = torch.finfo(torch.float32).min
    logits[9, 1:] = -float("inf")
    b = torch.zeros(E, device=DEV)
    b[10:] = -float("inf") if bias else 0.0
    ids, w, off, rows, _ = fme.moe_route_groups(logits, b if bias else None, k, score, groups=5, top_groups=2)
    a = _np(ids)
    assert a.min() >= 0 and a.max() < E and all(len(set(r)) == k for r in a.tolist())
    assert all(len(set(e // 8 for e in r)) <= 2 for r in a.tolist())
    for got, ref in zip((off, rows), prompt.group_routes(a, E)):
        assert np.array_equal(_np(got), ref)
    good = [t for t in range(T) if t not in (3, 4, 6, 7)]
    assert torch.isfinite(w[good]).all()
    assert a[5].tolist() == [0, 1, 2, 3, 4, 5] and not w[5].any()
    if score == "softmax":
        assert w[9].tolist() == [1.0, 0, 0, 0, 0, 0]
    ids, w, off, rows, tok = fme.moe_route_groups(logits[:0], None, k, score, groups=5, top_groups=2)
    assert ids.shape == (0, k) and rows.numel() == 0 and not off.any()


# --------------------------------------------------------------------------- block norm
def _norm_inputs(T, H, top_k, seed, shared=False, post=False, gate=None, residual=True):
    rng = np.random.default_rng([T, H, top_k, seed])
    n = T * max(top_k, 1)
    d = {"x": codecs.bf16_round((rng.normal(size=(n, H)) * np.exp2(rng.integers(-3, 4, size=(n, 1)))).astype(np.float32))}
    if top_k:
        d["route_weights"] = rng.uniform(0.05, 1.0, size=(T, top_k)).astype(np.float32)
    if shared:
        d["shared_out"] = _bf(rng, T, H)
    if post:
        d["post_gamma"] = codecs.bf16_round(rng.uniform(-1.5, 1.5, size=H).astype(np.float32))
    if gate:
        d["gate"] = codecs.bf16_round(rng.uniform(-1, 1, size=(H,) if gate == "row" else (T, H)).astype(np.float32))
    if residual:
        d["residual"] = codecs.bf16_round((5 * rng.normal(size=(T, H))).astype(np.float32))
    if T > 2:
        d["x"][max(top_k, 1):2 * max(top_k, 1)] = 0
        for name in ("shared_out", "residual"):
            if name in d:
                d[name][1] = 0
    d["gamma"] = codecs.bf16_round(rng.uniform(-1.5, 1.5, size=H).astype(np.float32))
    return d


def _to_dev(d):
    return {k: _dev(v, None if k == "route_weights" else BF) for k, v in d.items()}


def _check_codes(codes, scale, y, err):
    v = codecs.e4m3_decode(codes) * scale
    y = np.clip(y, -448 * scale, 448 * scale)
    assert np.all(np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) * 1.001 + err)


def _check_norm(fme, d, quant, alpha, ue8m0=False, dev=None, **kw):
    T = len(d["x"]) // (d["route_weights"].shape[1] if "route_weights" in d else 1)
    H = d["x"].shape[1]
    h, y, dh, dy = prompt.block_norm(**d, residual_scale=alpha)
    q, s, res, normed = fme.block_norm(**(dev or _to_dev(d)), residual_scale=alpha, quant=quant, ue8m0=ue8m0,
                                       want_normed=True, **kw)
    given = q, s, res, normed
    assert np.all(np.abs(_np(res) - h) <= dh + np.abs(h) * 2.0 ** -8 * 1.001)
    assert np.all(np.abs(_np(normed) - y) <= dy + np.abs(y) * 2.0 ** -8 * 1.001)
    if quant is None:
        assert q is None and s is None
        return given
    if quant == "fp8":
        s = _np(s).astype(np.float64)
        base = np.maximum(np.abs(y).reshape(T, H // 128, 128).max(-1), 1e-10) / 448
        slack = dy.reshape(T, H // 128, 128).max(-1) / 448 + 4 * U * base
        if ue8m0:
            base = np.maximum(base, 1e-10)
            assert np.array_equal(s, np.exp2(np.round(np.log2(s))))
            assert np.all(s >= base - slack) and np.all(s < 2 * (base + slack))
        else:
            assert np.all(np.abs(s - base) <= slack)
        s = np.repeat(s, 128, axis=1)
    else:
        e = _np(s).astype(np.int64) - 127
        amax, off = (v.reshape(T, H // 32, 32) for v in (np.abs(y), dy))
        low, high = (np.vectorize(mx_exponent)(np.maximum(v, 0)) for v in (amax.max(-1) - off.max(-1), (amax + off).max(-1)))
        assert np.all((e >= low) & (e <= high))
        s = np.repeat(np.exp2(e.astype(np.float64)), 32, axis=1)
    _check_codes(_np(q), s, y, dy + 4 * U * np.abs(y))
    return given


@pytest.mark.parametrize("quant", ["fp8", "mxfp8", None])
@pytest.mark.parametrize("T,H,top_k,shared,post,gate,residual,alpha", [
    (1, 7168, 8, True, True, "row", True, 1.0), (5, 1024, 3, False, False, None, True, 0.5),
    (3, 128, 0, False, True, "full", False, 1.0), (67, 3584, 16, True, False, "full", True, -0.75),
    (2, 8192, 0, False, True, None, True, 2.0), (9, 16384, 2, False, True, "row", True, 1.0),
    (300, 256, 1, True, False, None, False, 1.0), (40, 1152, 0, False, False, "row", True, 0.25),
    (4, 16384, 32, True, True, "full", True, 0.0)])
def test_block_norm(fme, quant, T, H, top_k, shared, post, gate, residual, alpha):
    _check_norm(fme, _norm_inputs(T, H, top_k, 1, shared, post, gate, residual), quant, alpha, ue8m0=T == 5)


@pytest.mark.parametrize("H,quant", [(8, None), (264, None), (16376, None), (32, "mxfp8"), (96, "mxfp8"), (8224, "mxfp8"),
                                     (4104, None)])
def test_block_norm_odd_widths(fme, H, quant):
    _check_norm(fme, _norm_inputs(7, H, 3, 2, True, True, "full"), quant, 0.5)
    _check_norm(fme, _norm_inputs(11, H, 0, 3, False, True, "row"), quant, 1.0)


def test_block_norm_without_second_norm(fme):
    d = _norm_inputs(6, 640, 4, 4, True, True, "row")
    dev = _to_dev(d)
    want = fme.block_norm(**dev, residual_scale=0.5)[2]
    dev["gamma"] = None
    q, s, res, normed = fme.block_norm(**dev, residual_scale=0.5)
    assert q is None and s is None and normed is None and torch.equal(res, want)


@pytest.mark.parametrize("T,H", [(1, 7168), (40, 640), (300, 3584)])
def test_block_norm_parts_match_the_single_operators(fme, T, H):
    """The combination alone is moe_finalize's, bit for bit; x + residual alone add_rmsnorm's."""
    d = _norm_inputs(T, H, 8, 5, True, residual=False)
    dev = _to_dev(d)
    res = fme.block_norm(dev["x"], None, route_weights=dev["route_weights"], shared_out=dev["shared_out"])[2]
    assert torch.equal(res, fme.moe_finalize(dev["x"], dev["route_weights"], dev["shared_out"]))
    assert np.array_equal(_np(res), oracle_finalize(d["x"], d["route_weights"], d["shared_out"]))
    d = _to_dev(_norm_inputs(T, H, 0, 6))
    res = fme.block_norm(d["x"], d["gamma"], d["residual"])[2]
    assert torch.equal(res, fme.add_rmsnorm_fp8(d["x"], d["gamma"], d["residual"])[2])


def test_block_norm_strides_in_place_and_streams(fme):
    T, H, k = 37, 640, 3
    d = _norm_inputs(T, H, k, 7, True, True, "full")
    dev = _to_dev(d)
    args = dict(residual_scale=0.5, quant="fp8", want_normed=True)
    ref = fme.block_norm(**dev, **args)
    wide = dict(dev, x=_wide(d["x"], 24), gate=_wide(d["gate"], 8), residual=_wide(d["residual"], 640))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fme.block_norm(**wide, **args)
        same = fme.block_norm(**dev, **args, residual_out=dev["residual"])
    side.synchronize()
    assert same[2] is dev["residual"]
    for a, b, c in zip(ref, got, same):
        assert torch.equal(a, b) and torch.equal(a, c)
    # One gate row for every token, as a vector and as an expanded matrix.
    dev = _to_dev(d)
    row = dev["gate"][0].contiguous()
    dev["gate"] = row
    ref = fme.block_norm(**dev, **args)
    dev["gate"] = row.expand(T, H)
    got = fme.block_norm(**dev, **args)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_block_norm_bad_values_stay_in_their_row(fme):
    T, H, k = 6, 512, 2
    d = _to_dev(_norm_inputs(T, H, k, 8, True, True, "full"))
    ref = fme.block_norm(**d, quant="fp8", want_normed=True)
    bad = {n: v.clone() for n, v in d.items()}
    bad["x"][0, 5] = float("nan")
    bad["residual"][2, 7] = float("inf")
    bad["gate"][4, 1] = float("nan")
    got = fme.block_norm(**bad, quant="fp8", want_normed=True)
    for a, b in zip(ref, got):
        assert torch.equal(a[1::2], b[1::2])
    assert torch.isnan(got[3][0]).all() and torch.isnan(got[3][4]).all()


def test_block_norm_no_tokens_and_offsets_past_32_bits(fme):
    H, ld, T = 256, 1 << 28, 10
    g = torch.ones(H, dtype=BF, device=DEV)
    q, s, res, normed = fme.block_norm(torch.empty(0, H, dtype=BF, device=DEV), g, quant="fp8")
    assert q.shape == (0, H) and s.shape == (0, 2) and res.shape == (0, H) and normed is None
    buf = torch.zeros((T - 1) * ld + H, dtype=BF, device=DEV)
    x = buf.as_strided((T, H), (ld, 1))
    x.copy_(torch.randn(T, H, device=DEV))
    a = fme.block_norm(x, g, x, gate=x, quant="mxfp8")
    c = x.contiguous()
    b = fme.block_norm(c, g, c, gate=c, quant="mxfp8")
    assert all(torch.equal(i, j) for i, j in zip(a[:3], b[:3]))
    w = torch.rand(5, 2, device=DEV)
    assert torch.equal(fme.block_norm(x, g, route_weights=w)[2], fme.block_norm(c, g, route_weights=w)[2])


# --------------------------------------------------------------------------- streams and graphs
def test_graph_of_the_operators_replays_with_new_inputs(fme):
    T, H, E, k = 150, 1024, 64, 4
    x, r = torch.randn(T, H, device=DEV).to(BF), torch.randn(T, H, device=DEV).to(BF)
    g = torch.ones(H, dtype=BF, device=DEV)
    w = (torch.randn(E, H, device=DEV) / 32).to(BF)
    down = (torch.randn(H, E, device=DEV)).to(BF)

    def step():
        q, s, h, n = fme.block_norm(x, g, r, post_gamma=g, quant="fp8", want_normed=True)
        logits = fme.linear_bf16(n, w, out_dtype=torch.float32)
        routed = fme.moe_route_groups(logits, None, k, "softmax", groups=8, top_groups=3)
        y = fme.linear_bf16(logits.to(BF), down, None, "silu", h)
        return [q, s, h, n, logits, *routed, y]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(step())
    for _ in range(3):
        x.normal_()
        r.normal_()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        ref = step()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert fme.kept_workspace_error() == 0


def test_streams_of_the_operators_share_nothing(fme):
    M, N, K = 100, 300, 5000
    ins = [(torch.randn(M, K, device=DEV).to(BF), torch.randn(N, K, device=DEV).to(BF)) for _ in range(2)]
    ref = [fme.linear_bf16(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fme.linear_bf16(*ins[i]))
    torch.cuda.synchronize()
    for r, runs in zip(ref, got):
        assert all(torch.equal(r, g) for g in runs)


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("T,routing", [(1, dict(groups=8, top_groups=4)), (90, dict(score="softmax", renormalise=False)),
                                       (300, dict(groups=4, top_groups=2, group_top=1)), (40, dict())])
def test_routed_block(fme, T, routing):
    """A block from its norm to the next block's: each step against the oracle on the step before it, the whole equal to
    the steps bit for bit."""
    cfg = W.RAGGED
    rng = np.random.default_rng(T)
    w13h, w2h = W.fp8_weights_host(cfg, 61)
    s13, s2 = W.fp8_weight_scales(cfg, 61)
    experts = [_dev(v) for v in (w13h.full(), s13, w2h.full(), s2)]
    x, r, g, pg = _bf(rng, T, cfg.H), _bf(rng, T, cfg.H), _bf(rng, cfg.H), _bf(rng, cfg.H)
    router = codecs.bf16_round(_bf(rng, cfg.E, cfg.H) / np.float32(32))
    bias = (0.1 * rng.normal(size=cfg.E)).astype(np.float32)
    shared = _bf(rng, T, cfg.H)
    dg, dpg, dsh, drouter, dbias = _dev(g, BF), _dev(pg, BF), _dev(shared, BF), _dev(router, BF), _dev(bias)
    xq, sx, h, normed = fme.block_norm(_dev(x, BF), dg, _dev(r, BF), quant="fp8", want_normed=True)
    args = (cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0)
    got = fme.moe_prompt_block_fp8(xq, sx, normed, h, drouter, dbias, *experts, *args, next_gamma=dg, post_gamma=dpg,
                                   gate=dpg, residual_scale=0.5, quant="fp8", shared_out=dsh, **routing)

    logits = fme.linear_bf16(normed, drouter, out_dtype=torch.float32)
    y, tol = oracle_linear.linear(_np(normed), router)
    assert np.all(np.abs(_np(logits) - y) <= tol + U * np.abs(y))
    rows, ids, weights = fme.moe_prompt_rows_fp8(xq, sx, logits, dbias, *experts, *args, **routing)
    full = {"groups": 1, **routing}
    full.setdefault("top_groups", full["groups"])
    full.setdefault("group_top", 2)
    rid, rw, gaps = routing_oracle(_np(logits), bias, cfg.top_k, scale=cfg.scale, **full)
    sure = gaps > 32 * U
    assert sure.mean() > 0.9 and np.array_equal(_np(ids)[sure], rid[sure])
    assert np.all(np.abs(_np(weights) - rw)[sure] <= 80 * U * np.abs(rw)[sure])
    d = dict(x=_np(rows), gamma=g, residual=_np(h), route_weights=_np(weights), shared_out=shared, post_gamma=pg, gate=pg)
    dev = dict(x=rows, gamma=dg, residual=h, route_weights=weights, shared_out=dsh, post_gamma=dpg, gate=dpg)
    last = _check_norm(fme, d, "fp8", 0.5, dev=dev)
    for a, b in zip(got, (*last, ids, weights)):
        assert torch.equal(a, b)
    # The same routes combined by themselves.
    y, pid, pw = fme.moe_prompt_fp8(xq, sx, logits, dbias, *experts, *args, shared_out=dsh, **routing)
    assert torch.equal(pid, ids) and torch.equal(pw, weights)
    assert torch.equal(y, fme.moe_finalize(rows, weights, dsh))


def test_routed_block_without_tokens(fme):
    cfg = W.RAGGED
    w13h, w2h = W.fp8_weights_host(cfg, 62)
    s13, s2 = W.fp8_weight_scales(cfg, 62)
    experts = [_dev(v) for v in (w13h.full(), s13, w2h.full(), s2)]
    g = torch.ones(cfg.H, dtype=BF, device=DEV)
    none = torch.empty(0, cfg.H, dtype=BF, device=DEV)
    xq, sx, h, normed = fme.block_norm(none, g, none, quant="fp8", want_normed=True)
    got = fme.moe_prompt_block_fp8(xq, sx, normed, h, torch.zeros(cfg.E, cfg.H, dtype=BF, device=DEV), None, *experts,
                                   cfg.top_k, cfg.limit, cfg.scale, cfg.ue8m0, next_gamma=g, quant="fp8", groups=4,
                                   top_groups=2)
    assert [tuple(t.shape) for t in got] == [(0, cfg.H), (0, cfg.H // 128), (0, cfg.H), (0, cfg.H), (0, cfg.top_k),
                                             (0, cfg.top_k)]
