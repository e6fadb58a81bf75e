"""The prompt side of the routed layer: norm with residual, routes grouped by
expert, and the products grouped by expert.

Oracle (test infrastructure only; see the package docstring).

"vllm.models.glm5next.nvidia.specialized_decode.mega_moe" defines the routing,
the block-scaled products and the SwiGLU; here they are taken over any number
of rows, each row with the weights of its group. Sums are float64.
"""

import numpy as np

from .codecs import bf16_round, e4m3_decode
from .quant import GROUP


def add_rmsnorm(x, residual, gamma, eps):
    """(z, y): z = bf16(float32(x + residual)) (x without a residual), y = z / sqrt(mean z^2 + eps) * gamma in
    float64, not rounded. x, residual [T, H] and gamma [H] are float32 arrays of BF16 values."""
    z = np.asarray(x, dtype=np.float32)
    if residual is not None:
        z = bf16_round((z + np.asarray(residual, dtype=np.float32)).astype(np.float32))
    d = z.astype(np.float64)
    y = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps) * np.asarray(gamma, dtype=np.float64)
    return z, y


def group_routes(ids, E):
    """(offsets [E + 1], rows, tokens): the routes t * top_k + r of ids [T, top_k] by expert, ascending within one."""
    ids = np.asarray(ids)
    T, k = ids.shape
    groups = [[] for _ in range(E)]
    for t in range(T):
        for r in range(k):
            groups[int(ids[t, r])].append(t * k + r)
    rows = np.array([p for g in groups for p in g], dtype=np.int32)
    offsets = np.cumsum([0] + [len(g) for g in groups]).astype(np.int32)
    return offsets, rows, (rows // k).astype(np.int32)


def grouped_product(a, sa, w, sw, offsets, in_rows=None):
    """(y, size) float64 [R, N] with R = offsets[-1]: for place p of group e and r = in_rows[p],
    y = sum_b P * float32(sw[e, n/128, b] * sa[r, b]) with P the exact product over block b, and
    size = sum_b |scale| * sum_k |w a| (what rounding errors of the sums scale with)."""
    E, N, K = w.shape
    R = int(offsets[-1])
    rows = np.arange(R) if in_rows is None else np.asarray(in_rows)[:R]
    A = e4m3_decode(a).reshape(len(a), K // GROUP, GROUP)
    y, size = np.zeros((R, N)), np.zeros((R, N))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi <= lo:
            continue
        W = e4m3_decode(w[e]).reshape(N, K // GROUP, GROUP)
        s_w = np.repeat(sw[e], GROUP, axis=0).astype(np.float32)
        r = rows[lo:hi]
        for b in range(K // GROUP):
            s = (s_w[None, :, b] * np.asarray(sa, dtype=np.float32)[r, b][:, None]).astype(np.float32)
            y[lo:hi] += A[r, b] @ W[:, b].T * s
            size[lo:hi] += np.abs(A[r, b]) @ np.abs(W[:, b]).T * np.abs(s)
    return y, size


def block_norm(x, gamma, residual=None, route_weights=None, shared_out=None, post_gamma=None, gate=None,
               residual_scale=1.0, eps=1e-5):
    """(h, y, dh, dy) float64: what stands between a block and the next. o = x, or the weighted sum of each token's
    routes (+ shared_out); p = o / sqrt(mean o^2 + eps) * post_gamma; h = residual_scale * residual + gate * p; y = h /
    sqrt(mean h^2 + eps) * gamma; nothing rounded. dh and dy bound what FP32 arithmetic may be off (u = 2^-24):
    a sum of n terms by n u of their magnitudes, a row's mean square, of sums of at most 64 terms, by 80 u and what its
    values are off, each product and addition by u."""
    u = 2.0 ** -24
    f = lambda v: None if v is None else np.asarray(v, dtype=np.float64)  # noqa: E731
    x, gamma, residual, w, shared_out, post_gamma, gate = map(f, (x, gamma, residual, route_weights, shared_out,
                                                                   post_gamma, gate))

    def norm(v, dv, g):
        r = 1 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
        length = np.sqrt((v * v).sum(axis=1, keepdims=True))
        off = np.sqrt((dv * dv).sum(axis=1, keepdims=True)) / np.where(length > 0, length, 1.0)
        return v * r * g, (dv * r + np.abs(v) * r * (48 * u + off)) * np.abs(g)

    o, do = x, np.zeros_like(x)
    if w is not None:
        T, k = w.shape
        terms = x.reshape(T, k, -1) * w[:, :, None]
        o, size = terms.sum(axis=1), np.abs(terms).sum(axis=1)
        if shared_out is not None:
            o, size = o + shared_out, size + np.abs(shared_out)
        do = (k + 3) * u * size
    if post_gamma is not None:
        o, do = norm(o, do, post_gamma)
    if gate is not None:
        o, do = o * gate, do * np.abs(gate) + u * np.abs(o * gate)
    h, dh = o, do
    if residual is not None:
        h = h + residual_scale * residual
        dh = dh + u * (np.abs(residual_scale * residual) + np.abs(h))
    if gamma is None:
        return h, None, dh, None
    y, dy = norm(h, dh, gamma)
    return h, y, dh, dy
