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
