"""Operators of a routed-expert layer for prompts (any number of tokens), measured on the GPU.

norm    h = x + residual, RMSNorm(h) * gamma, quantised to E4M3 with one FP32 scale per 128 values ("fp8") or one
        E8M0 scale per 32 values ("mxfp8"); the BF16 norm (router input) and the new residual come with it.
route   top-k of sigmoid scores + bias per token, and the routes sorted by expert (stable).
swiglu  per expert, the product of its tokens' rows with the gate and up weights, clamped SwiGLU, E4M3 with one FP32
        scale per 128 hidden values.
gemm    per expert, the product of its hidden rows with the down weights, written to route order in BF16.

Weights and activations are E4M3; activations carry one FP32 scale per row and 128 values, weights one per 128 x 128
block. `own` selects the framework's kernels; otherwise the operators are plain torch in 32 bits.
"""

import math
import random

import torch

own = False

EPS = 1e-5
LIMIT = 7.0
ROUTE_SCALE = 2.5
# (H, I, E, top_k, bias spread): the repository's routed shapes (tiny, ragged, DeepSeek-V3, latent) and one generic.
SHAPES = {
    "tiny": (512, 256, 8, 2, 0.1),
    "ragged": (1024, 384, 40, 3, 0.1),
    "generic": (2048, 640, 64, 6, 0.2),
    "dsv3": (7168, 2048, 256, 8, 0.05),
    "latent": (3584, 2048, 896, 16, 0.5),
}
MAX_FLOPS = 2.0 * 16384 * 8 * 4096 * 7168  # the largest listed product


def listed():
    return [
        # One decode token of the DeepSeek-V3 shape: pure latency.
        {"name": "norm_1", "op": "norm", "form": "fp8", "T": 1, "H": 7168, "residual": True, "pad": 0},
        # An odd prompt of the latent shape in the MXFP8 format, first layer (no residual), rows of a wider buffer.
        {"name": "norm_mx_ragged", "op": "norm", "form": "mxfp8", "T": 1533, "H": 3584, "residual": False, "pad": 512},
        # A long prompt of the DeepSeek-V3 shape: memory-bound.
        {"name": "norm_16k", "op": "norm", "form": "fp8", "T": 16384, "H": 7168, "residual": True, "pad": 0},
        # Routing of one decode token.
        {"name": "route_1", "op": "route", "shape": "dsv3", "T": 1, "bf16": True},
        # Routing of an odd prompt over 896 experts with a skewed bias, FP32 logits.
        {"name": "route_latent", "op": "route", "shape": "latent", "T": 1533, "bf16": False},
        # Routing of a long prompt, BF16 logits.
        {"name": "route_16k", "op": "route", "shape": "dsv3", "T": 16384, "bf16": True},
        # The gate/up product of one decode token: eight experts of one row each, weight streaming.
        {"name": "swiglu_1", "op": "swiglu", "shape": "dsv3", "T": 1},
        # A prompt just above the decode batch: every expert touched, a few rows each.
        {"name": "swiglu_200", "op": "swiglu", "shape": "dsv3", "T": 200},
        # A batch of long prompts: 512 rows per expert on average, arithmetic.
        {"name": "swiglu_16k", "op": "swiglu", "shape": "dsv3", "T": 16384},
        # The down product of one decode token.
        {"name": "gemm_1", "op": "gemm", "shape": "dsv3", "T": 1},
        # Odd sizes: 40 experts, three 128-blocks of hidden values, ragged groups of about 100 rows.
        {"name": "gemm_ragged", "op": "gemm", "shape": "ragged", "T": 1333},
        # The down product of a long prompt: weights, hidden rows and arithmetic weigh about the same.
        {"name": "gemm_8k", "op": "gemm", "shape": "dsv3", "T": 8192},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "route", "swiglu", "gemm"])
    if op == "norm":
        form = rng.choice(["fp8", "mxfp8"])
        step = 128 if form == "fp8" else 32
        H = step * _log_int(rng, 256 // step, 7168 // step)
        return {"op": op, "form": form, "T": _log_int(rng, 1, 16384), "H": H, "residual": rng.random() < 0.7,
                "pad": rng.choice([0, 0, 8, 136])}
    shape = rng.choice(sorted(SHAPES))
    H, I, E, k, _ = SHAPES[shape]
    if op == "route":
        return {"op": op, "shape": shape, "T": _log_int(rng, 1, min(16384, 16384 * 256 // E)),
                "bf16": rng.random() < 0.5}
    most = int(MAX_FLOPS / (2.0 * k * (2 if op == "swiglu" else 1) * I * H))
    return {"op": op, "shape": shape, "T": _log_int(rng, 1, min(16384, most))}


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _block_scales(g, *shape):
    return torch.exp2(torch.rand(*shape, generator=g, device="cuda") * 5 - 9)


def _codes(g, E, rows, cols):
    """E4M3 bytes of N(0, 1), an expert at a time."""
    out = torch.empty(E, rows, cols, dtype=torch.uint8, device="cuda")
    for e in range(E):
        out[e] = _randn(g, rows, cols).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _activations(v):
    """E4M3 codes [R, K] and FP32 scales [R, K / 128] of v."""
    R, K = v.shape
    b = v.view(R, K // 128, 128)
    s = b.abs().amax(-1).clamp_min(1e-10) / 448
    q = (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(R, K), s


def _logits(g, T, E, bias, top_k, bf16):
    """Router logits whose picks do not hang on the last bit: a token whose deciding keys lie within 2^-17 of one
    another is drawn again."""
    out = _randn(g, T, E)
    if bf16:
        out = out.bfloat16().float()
    n = min(E, top_k + 1)
    for _ in range(40):
        keys = (torch.sigmoid(out.double()) + bias.double()).topk(n).values
        close = (keys[:, :-1] - keys[:, 1:] < 2.0 ** -17).any(1)
        fresh = _randn(g, T, E)
        if bf16:
            fresh = fresh.bfloat16().float()
        out = torch.where(close[:, None], fresh, out)
    return out.bfloat16() if bf16 else out


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # A residual stream with a few loud channels; one all-zero (padding) token.
        loud = torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        x = torch.zeros(T, H + case["pad"], dtype=torch.bfloat16, device="cuda")[:, :H]
        x.copy_(_randn(g, T, H) * loud)
        residual = (3 * _randn(g, T, H) * loud).bfloat16() if case["residual"] else None
        if T > 2:
            x[T // 2] = 0
            if residual is not None:
                residual[T // 2] = 0
        gamma = (1 + 0.2 * _randn(g, H)).bfloat16()
        return {"op": "norm", "form": case["form"], "x": x, "residual": residual, "gamma": gamma}
    H, I, E, k, spread = SHAPES[case["shape"]]
    T = case["T"]
    bias = spread * _randn(g, E)
    if case["op"] == "route":
        return {"op": "route", "logits": _logits(g, T, E, bias, k, case["bf16"]), "bias": bias, "k": k}
    # The routes of T tokens, sorted by expert.
    ids = (torch.sigmoid(_randn(g, T, E)) + bias).topk(k).indices.reshape(-1)
    rows = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    s = {"op": case["op"], "offsets": offsets, "bounds": offsets.tolist()}
    if case["op"] == "swiglu":
        s["a"], s["sa"] = _activations(_randn(g, T, H))
        s["index"] = (rows // k).int()
        s["w"], s["sw"] = _codes(g, E, 2 * I, H), _block_scales(g, E, 2 * I // 128, H // 128)
    else:
        gate, up = _randn(g, T * k, I), _randn(g, T * k, I)
        s["a"], s["sa"] = _activations(gate * torch.sigmoid(gate) * up)
        s["index"] = rows.int()
        s["w"], s["sw"] = _codes(g, E, H, I), _block_scales(g, E, H // 128, I // 128)
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "route": _plain_route, "swiglu": _plain_swiglu, "gemm": _plain_gemm}[state["op"]](state)


def _run_own(s):
    import fp4_moe_expert_gb300 as fme

    if s["op"] == "norm":
        if s["form"] == "fp8":
            q, sc, res, normed = fme.add_rmsnorm_fp8(s["x"], s["gamma"], s["residual"], EPS, want_normed=True)
        else:
            q, sc, res, normed = fme.add_rmsnorm_mxfp8(s["x"], s["gamma"], s["residual"], EPS, want_normed=True)
            sc = sc.view(torch.float8_e8m0fnu)
        return [q.view(torch.float8_e4m3fn), sc, normed] + ([] if res is None else [res])
    if s["op"] == "route":
        ids, weights, offsets, rows, tokens = fme.moe_route(s["logits"], s["bias"], s["k"], ROUTE_SCALE)
        return [ids, weights, offsets, rows, tokens]
    if s["op"] == "swiglu":
        q, sh = fme.moe_grouped_swiglu_fp8(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], in_rows=s["index"],
                                           limit=LIMIT)
        return [q.view(torch.float8_e4m3fn), sh]
    return fme.moe_grouped_gemm_fp8(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], out_rows=s["index"])


def _plain_norm(s):
    x, residual = s["x"].float(), s["residual"]
    if residual is not None:
        residual = (x + residual.float()).bfloat16()
        x = residual.float()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * s["gamma"].float()
    T, H = y.shape
    if s["form"] == "fp8":
        b = y.view(T, H // 128, 128)
        sc = b.abs().amax(-1).clamp_min(1e-10) / 448
        q = b * (1 / sc)[..., None]
    else:
        b = y.view(T, H // 32, 32)
        amax = b.abs().amax(-1)
        exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(-127, 127)
        q = torch.ldexp(b, -exponent[..., None])
        sc = (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    q = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(T, H)
    return [q, sc, y.bfloat16()] + ([] if residual is None else [residual])


def _plain_route(s):
    score = torch.sigmoid(s["logits"].float())
    T, E = score.shape
    k = s["k"]
    ids = torch.sort(score + s["bias"], dim=1, descending=True, stable=True).indices[:, :k]
    picked = score.gather(1, ids)
    weights = picked / picked.sum(1, keepdim=True) * ROUTE_SCALE
    flat = ids.reshape(-1)
    rows = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return [ids.int(), weights, offsets.int(), rows.int(), (rows // k).int()]


def _dequant(codes, scales, rows_per_scale):
    """FP32 values of E4M3 codes [R, K] with one scale per rows_per_scale rows and 128 columns."""
    R, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(R // rows_per_scale, rows_per_scale, K // 128, 128)
    return (v * scales[:, None, :, None]).view(R, K)


def _plain_swiglu(s):
    a = _dequant(s["a"], s["sa"], 1)
    E, two_i, _ = s["w"].shape
    I, R = two_i // 2, s["index"].numel()
    h = torch.empty(R, I, device="cuda")
    b = s["bounds"]
    # One product per expert: the groups are ragged.
    for e in range(E):
        if b[e + 1] > b[e]:
            y = a[s["index"][b[e]:b[e + 1]]] @ _dequant(s["w"][e], s["sw"][e], 128).t()
            up, gate = y[:, :I].clamp(-LIMIT, LIMIT), y[:, I:].clamp_max(LIMIT)
            h[b[e]:b[e + 1]] = gate / (1 + torch.exp(-gate)) * up
    h = h.view(R, I // 128, 128)
    sh = h.abs().amax(-1).clamp_min(1e-10) / 448
    q = (h / sh[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(R, I)
    return [q, sh]


def _plain_gemm(s):
    a = _dequant(s["a"], s["sa"], 1)
    E, N, _ = s["w"].shape
    out = torch.empty(a.shape[0], N, dtype=torch.bfloat16, device="cuda")
    b = s["bounds"]
    # One product per expert: the groups are ragged.
    for e in range(E):
        if b[e + 1] > b[e]:
            y = a[b[e]:b[e + 1]] @ _dequant(s["w"][e], s["sw"][e], 128).t()
            out[s["index"][b[e]:b[e + 1]]] = y.bfloat16()
    return out


# --------------------------------------------------------------------------- what a pass needs
def _touched(T, E, k):
    """Experts that T tokens of k picks touch, picks spread evenly."""
    return E * (1 - (1 - k / E) ** T)


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        per_value = 2 + 1 + 2 + (4 if case["residual"] else 0)
        scales = H / 128 * 4 if case["form"] == "fp8" else H / 32
        return {"bytes": T * (H * per_value + scales) + 2 * H, "flops": 8 * T * H}
    H, I, E, k, _ = SHAPES[case["shape"]]
    R = T * k
    if case["op"] == "route":
        return {"bytes": T * E * (2 if case["bf16"] else 4) + 4 * E + 16 * R + 4 * (E + 1), "flops": T * E * 6}
    n, kk = (2 * I, H) if case["op"] == "swiglu" else (H, I)
    weights = _touched(T, E, k) * (n * kk + 4 * (n // 128) * (kk // 128))
    if case["op"] == "swiglu":
        moved = T * (H + H / 32) + R * (I + I / 32) + 4 * R
    else:
        moved = R * (I + I / 32) + 2 * R * H + 4 * R
    return {"bytes": weights + moved + 4 * (E + 1), "flops": 2.0 * R * n * kk}


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """Values before their last rounding, in 64 bits. Quantised values are given as value / scale, unrounded."""
    if case["op"] in ("swiglu", "gemm") and work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        z = s["x"].double()
        out_res = []
        if s["residual"] is not None:
            z = z + s["residual"].double()
            out_res = [z]
            z = z.float().bfloat16().double()
        y = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["gamma"].double()
        n = 128 if s["form"] == "fp8" else 32
        blocks = y.unflatten(1, (-1, n))
        top = blocks.abs().amax(-1)
        if s["form"] == "fp8":
            sc = torch.maximum(top, torch.full_like(top, 1e-10)) / 448
        else:
            sc = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 8), 2.0 ** -127)
        return [(blocks / sc[..., None]).flatten(1), sc, y] + out_res
    if case["op"] == "route":
        score = 1 / (1 + torch.exp(-s["logits"].double()))
        order = (score + s["bias"].double()).argsort(dim=1, descending=True)[:, :s["k"]]
        p = torch.take_along_dim(score, order, 1)
        return [None, p * (ROUTE_SCALE / p.sum(1, keepdim=True)), None, None, None]

    def wide(codes, scales):
        v = codes.view(torch.float8_e4m3fn).double()
        each = torch.ones(v.shape[0] // scales.shape[0], 128, dtype=torch.float64, device="cuda")
        return v * torch.kron(scales.double(), each)

    groups = [(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])) if hi > lo]
    act = wide(s["a"], s["sa"])
    if case["op"] == "gemm":
        out = torch.zeros(act.shape[0], s["w"].shape[1], dtype=torch.float64, device="cuda")
        for e, part in groups:
            out[s["index"][part].long()] = act[part].matmul(wide(s["w"][e], s["sw"][e]).T)
        return out
    hidden = []
    for e, part in groups:
        up, gate = act[s["index"][part].long()].matmul(wide(s["w"][e], s["sw"][e]).T).chunk(2, dim=1)
        gate = torch.minimum(gate, torch.full_like(gate, LIMIT))
        hidden.append(gate * torch.sigmoid(gate) * up.clamp(min=-LIMIT, max=LIMIT))
    hidden = torch.cat(hidden).unflatten(1, (-1, 128))
    sh = hidden.abs().amax(-1).clamp(min=1e-10) / 448
    return [(hidden / sh[..., None]).flatten(1), sh]
