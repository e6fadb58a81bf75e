"""Pins of the prompt oracle: closed forms, a library sort and the decode oracle."""

import numpy as np

from oracle import codecs, moe_fp8, prompt, quant


def test_norm_closed_forms():
    x = np.full((2, 128), 3.0, np.float32)
    z, y = prompt.add_rmsnorm(x, None, np.full(128, 2.0, np.float32), 0.0)
    assert np.array_equal(z, x) and np.allclose(y, 2.0, rtol=1e-15)
    # the residual sum is rounded to BF16 before the norm sees it
    z, _ = prompt.add_rmsnorm(np.full((1, 128), 256.0, np.float32), np.full((1, 128), 0.75, np.float32),
                              np.ones(128, np.float32), 0.0)
    assert np.all(z == 256.0)
    # scaling the row changes nothing without eps; a zero row stays zero with it
    rng = np.random.default_rng(0)
    v = codecs.bf16_round(rng.normal(size=(3, 256)).astype(np.float32))
    g = codecs.bf16_round(rng.normal(size=256).astype(np.float32))
    assert np.allclose(prompt.add_rmsnorm(v, None, g, 0.0)[1], prompt.add_rmsnorm(4 * v, None, g, 0.0)[1], rtol=1e-14)
    assert np.all(prompt.add_rmsnorm(0 * v, None, g, 1e-5)[1] == 0)


def test_groups_are_a_stable_sort():
    rng = np.random.default_rng(1)
    ids = np.stack([rng.permutation(7)[:3] for _ in range(50)])
    off, rows, tok = prompt.group_routes(ids, 9)
    assert np.array_equal(rows, np.argsort(ids.reshape(-1), kind="stable"))
    assert np.array_equal(tok, rows // 3)
    assert np.array_equal(np.diff(off), np.bincount(ids.reshape(-1), minlength=9))


def test_grouped_product_is_the_decode_gemv_row_by_row():
    rng = np.random.default_rng(2)
    E, N, K = 3, 256, 384
    w = codecs.e4m3_encode(rng.normal(size=(E, N, K)).astype(np.float32))
    sw = np.exp2(rng.uniform(-8, -4, size=(E, N // 128, K // 128))).astype(np.float32)
    a, sa = quant.fp8_quant_mul(rng.normal(size=(5, K)).astype(np.float32), False)
    off, rows = np.array([0, 2, 2, 6]), np.array([4, 0, 1, 1, 3, 2])
    y, size = prompt.grouped_product(a, sa, w, sw, off, rows)
    for p, e in enumerate([0, 0, 2, 2, 2, 2]):
        ref = moe_fp8.block_scaled_gemv(w[e], sw[e], a[rows[p]], sa[rows[p]])
        assert np.allclose(y[p], ref, rtol=1e-12, atol=1e-12 * np.abs(ref).max())
    assert np.all(size >= np.abs(y) * (1 - 1e-12))
