"""Operators around a routed-expert block, for prompts and for single tokens, measured on the GPU.

linear  act(x W^T + bias) + residual in one launch, BF16 operands: the router's product and a layer's dense projections.
route   top-k routing with softmax or sigmoid scores, an optional selection bias, the experts limited to each token's
        best groups, weights renormalised or not; the routes come sorted by expert (stable).
norm    what stands between a block and the next: the weighted sum of the routes (where the block is the experts), the
        norm after the block, its gate, the scaled residual, the norm before the next block, 8-bit quantisation.

`own` selects the framework's kernels; otherwise the operators are plain torch in 32 bits.
"""

import math
import random

import torch

own = False

EPS = 1e-5
ROUTE_SCALE = 2.5
# (E, top_k, bias spread): the repository's routers (tiny, ragged, DeepSeek-V3, latent, NVFP4) and one generic.
ROUTERS = {
    "tiny": (8, 2, 0.1),
    "ragged": (40, 3, 0.1),
    "generic": (64, 6, 0.2),
    "dsv3": (256, 8, 0.05),
    "nvfp4": (384, 6, 0.05),
    "latent": (896, 16, 0.5),
}
ACTIVATIONS = (None, "relu", "silu", "gelu", "sigmoid")
MAX_FLOPS = 2.0 * 16384 * 4096 * 7168   # the largest listed product
MAX_VALUES = 16384 * 7168 * 4.0         # values a listed norm reads at most


def listed():
    return [
        # The router's logits of one decode token of the DeepSeek-V3 shape: pure latency.
        {"name": "linear_router_1", "op": "linear", "M": 1, "N": 256, "K": 7168, "pad": 0, "bias": False, "act": None,
         "residual": False, "f32": True},
        # The projection back to the residual stream of a decode batch: the weights' stream.
        {"name": "linear_down_64", "op": "linear", "M": 64, "N": 7168, "K": 2048, "pad": 0, "bias": False, "act": None,
         "residual": True, "f32": False},
        # Odd sizes, rows of wider buffers: a gate of the latent shape over an odd prompt.
        {"name": "linear_ragged", "op": "linear", "M": 1533, "N": 895, "K": 3581, "pad": 24, "bias": True,
         "act": "sigmoid", "residual": False, "f32": False},
        # The router's logits of a long prompt: reading the tokens and the arithmetic weigh alike.
        {"name": "linear_router_16k", "op": "linear", "M": 16384, "N": 256, "K": 7168, "pad": 0, "bias": False,
         "act": None, "residual": False, "f32": True},
        # A dense expansion with bias and SiLU over a long prompt: arithmetic.
        {"name": "linear_up_16k", "op": "linear", "M": 16384, "N": 4096, "K": 7168, "pad": 0, "bias": True,
         "act": "silu", "residual": False, "f32": False},
        # Routing of one decode token, four of eight groups.
        {"name": "route_groups_1", "op": "route", "router": "dsv3", "T": 1, "bf16": True, "score": "sigmoid",
         "groups": 8, "top_groups": 4, "group_top": 2, "bias": True, "renormalise": True},
        # An odd prompt over 896 experts, softmax scores with a skewed bias and no groups.
        {"name": "route_softmax", "op": "route", "router": "latent", "T": 1533, "bf16": False, "score": "softmax",
         "groups": 1, "top_groups": 1, "group_top": 1, "bias": True, "renormalise": False},
        # A long prompt, four of eight groups, BF16 logits.
        {"name": "route_groups_16k", "op": "route", "router": "dsv3", "T": 16384, "bf16": True, "score": "sigmoid",
         "groups": 8, "top_groups": 4, "group_top": 2, "bias": True, "renormalise": True},
        # One decode token's routes and shared expert combined, normed, gated, added and normed again.
        {"name": "norm_routes_1", "op": "norm", "T": 1, "H": 7168, "top_k": 8, "shared": True, "post": True,
         "gate": "row", "residual": True, "quant": "fp8", "pad": 0},
        # An odd prompt of the latent shape, a plain block's rows of a wider buffer, the MXFP8 format.
        {"name": "norm_mx_ragged", "op": "norm", "T": 1533, "H": 3584, "top_k": 0, "shared": False, "post": True,
         "gate": None, "residual": True, "quant": "mxfp8", "pad": 512},
        # The routes of a prompt combined: eight rows read for each one written.
        {"name": "norm_routes_4k", "op": "norm", "T": 4096, "H": 7168, "top_k": 8, "shared": True, "post": False,
         "gate": None, "residual": True, "quant": "fp8", "pad": 0},
        # A long prompt with a gate for every value: memory-bound.
        {"name": "norm_gate_16k", "op": "norm", "T": 16384, "H": 7168, "top_k": 0, "shared": False, "post": True,
         "gate": "full", "residual": True, "quant": "fp8", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["linear", "route", "norm"])
    if op == "linear":
        N, K = _log_int(rng, 1, 7168), _log_int(rng, 8, 7168)
        M = _log_int(rng, 1, min(16384, int(MAX_FLOPS / (2.0 * N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "pad": rng.choice([0, 0, 8, 136]), "bias": rng.random() < 0.5,
                "act": rng.choice(ACTIVATIONS), "residual": rng.random() < 0.5, "f32": rng.random() < 0.4}
    if op == "route":
        router = rng.choice(sorted(ROUTERS))
        E, k, _ = ROUTERS[router]
        groups = rng.choice([g for g in range(1, 17) if E % g == 0])
        fewest = -(-k // (E // groups))
        score, bias = rng.choice(["sigmoid", "softmax"]), rng.random() < 0.6
        # (Renormalised sigmoid scores with a bias and no groups are the routing that the framework has already.)
        again = rng.random() < 0.6 and not (score == "sigmoid" and bias and groups == 1)
        return {"op": op, "router": router, "T": _log_int(rng, 1, min(16384, 16384 * 256 // E)),
                "bf16": rng.random() < 0.5, "score": score, "groups": groups,
                "top_groups": rng.randint(fewest, groups), "group_top": rng.choice([1, 2]) if E // groups > 1 else 1,
                "bias": bias, "renormalise": again}
    top_k = rng.choice([0, 0, 2, 6, 8, 16])
    quant = rng.choice(["fp8", "mxfp8", None])
    step = {"fp8": 128, "mxfp8": 32, None: 8}[quant]
    H = step * _log_int(rng, 256 // step, 7168 // step)
    most = min(16384, int(MAX_VALUES / (H * (3 + top_k))))
    return {"op": op, "T": _log_int(rng, 1, most), "H": H, "top_k": top_k, "shared": top_k > 0 and rng.random() < 0.5,
            "post": rng.random() < 0.6, "gate": rng.choice([None, "row", "full"]), "residual": rng.random() < 0.8,
            "quant": quant, "pad": rng.choice([0, 0, 8, 136])}


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(v, pad):
    """BF16 rows of v in a buffer whose rows are whole 16-byte units, `pad` values apart."""
    n, k = v.shape
    buf = torch.zeros(n, (k + 7) // 8 * 8 + pad, dtype=torch.bfloat16, device="cuda")[:, :k]
    return buf.copy_(v)


def _logits(g, case, bias):
    """Router logits whose picks do not hang on the last bits: a token whose deciding keys or group scores lie within
    2^-17 of one another (and are not equal) is drawn again."""
    E, k, _ = ROUTERS[case["router"]]
    T, G = case["T"], case["groups"]

    def fresh():
        v = 1.5 * _randn(g, T, E)
        return v.bfloat16().float() if case["bf16"] else v

    def near(v):
        gap = v[:, :-1] - v[:, 1:]
        return ((gap > 0) & (gap < 2.0 ** -17 * v[:, :-1].abs())).any(1)

    out = fresh()
    for _ in range(40):
        keys = torch.softmax(out.double(), 1) if case["score"] == "softmax" else torch.sigmoid(out.double())
        if bias is not None:
            keys = keys + bias.double()
        close = torch.zeros(T, dtype=torch.bool, device="cuda")
        if G > 1:
            best = keys.view(T, G, E // G).topk(case["group_top"], dim=2).values.sum(2)
            order = best.sort(1, descending=True)
            if case["top_groups"] < G:
                close |= near(order.values[:, case["top_groups"] - 1:case["top_groups"] + 1])
            open_ = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(
                1, order.indices[:, :case["top_groups"]], True)
            keys = keys.masked_fill(~open_.repeat_interleave(E // G, 1), -9.0)
        close |= near(keys.topk(min(E, k + 1)).values)
        out = torch.where(close[:, None], fresh(), out)
    return out.bfloat16() if case["bf16"] else out


def prepare(case, seed):
    g = _generator(seed)
    s = {k: v for k, v in case.items() if k != "name"}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _rows(_randn(g, M, K), case["pad"])
        s["w"] = _rows(_randn(g, N, K) / math.sqrt(K), case["pad"])
        s["b"] = _randn(g, N) if case["bias"] else None
        s["r"] = None
        if case["residual"]:
            s["r"] = _randn(g, M, N) if case["f32"] else _randn(g, M, N).bfloat16()
        return s
    if case["op"] == "route":
        E, _, spread = ROUTERS[case["router"]]
        s["b"] = spread * _randn(g, E) if case["bias"] else None
        s["logits"] = _logits(g, case, s["b"])
        return s
    T, H, k = case["T"], case["H"], case["top_k"]
    # A block's output and a residual stream, each with a few loud channels; one all-zero (padding) token.
    loud = torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    s["x"] = _rows(_randn(g, T * max(k, 1), H) * loud, case["pad"])
    s["weights"] = s["sh"] = s["pg"] = s["g"] = s["r"] = None
    if k:
        p = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["weights"] = p / p.sum(1, keepdim=True) * ROUTE_SCALE
    if case["shared"]:
        s["sh"] = _randn(g, T, H).bfloat16()
    if case["post"]:
        s["pg"] = (1 + 0.2 * _randn(g, H)).bfloat16()
    if case["gate"]:
        s["g"] = torch.sigmoid(_randn(g, *((H,) if case["gate"] == "row" else (T, H)))).bfloat16()
    if case["residual"]:
        s["r"] = (3 * _randn(g, T, H) * loud).bfloat16()
    if T > 2:
        n = T // 2
        s["x"][n * max(k, 1):(n + 1) * max(k, 1)] = 0
        for name in ("sh", "r"):
            if s[name] is not None:
                s[name][n] = 0
    s["gamma"] = (1 + 0.2 * _randn(g, H)).bfloat16()
    s["alpha"] = 0.75
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"linear": _plain_linear, "route": _plain_route, "norm": _plain_norm}[state["op"]](state)


def _run_own(s):
    import fp4_moe_expert_gb300 as fme

    if s["op"] == "linear":
        return fme.linear_bf16(s["x"], s["w"], s["b"], s["act"], s["r"],
                               out_dtype=torch.float32 if s["f32"] else torch.bfloat16)
    if s["op"] == "route":
        return list(fme.moe_route_groups(s["logits"], s["b"], ROUTERS[s["router"]][1], score=s["score"],
                                         groups=s["groups"], top_groups=s["top_groups"], group_top=s["group_top"],
                                         renormalise=s["renormalise"], scale=ROUTE_SCALE))
    q, sc, h, normed = fme.block_norm(s["x"], s["gamma"], s["r"], route_weights=s["weights"], shared_out=s["sh"],
                                      post_gamma=s["pg"], gate=s["g"], residual_scale=s["alpha"], eps=EPS,
                                      quant=s["quant"], want_normed=True)
    if s["quant"] is None:
        return [h, normed]
    return [h, normed, q.view(torch.float8_e4m3fn), sc if s["quant"] == "fp8" else sc.view(torch.float8_e8m0fnu)]


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        y = y + s["b"]
    if s["act"] == "relu":
        y = y.clamp_min(0)
    elif s["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif s["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif s["act"] == "sigmoid":
        y = 1 / (1 + torch.exp(-y))
    if s["r"] is not None:
        y = y + s["r"].float()
    return y if s["f32"] else y.bfloat16()


def _plain_route(s):
    logits = s["logits"].float()
    T, E = logits.shape
    k, G = ROUTERS[s["router"]][1], s["groups"]
    if s["score"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    keys = score if s["b"] is None else score + s["b"]
    if G > 1:
        best = torch.sort(keys.view(T, G, E // G), dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        chosen = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        group = torch.arange(E, device="cuda") // (E // G)
        keys = torch.where((chosen[:, :, None] == group).any(1), keys, -math.inf)
    ids = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :k]
    weights = score.gather(1, ids)
    if s["renormalise"]:
        weights = weights / weights.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    rows = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return [ids.int(), weights * ROUTE_SCALE, offsets.int(), rows.int(), (rows // k).int()]


def _plain_norm(s):
    o = s["x"].float()
    T, H = s["T"], s["H"]
    if s["top_k"]:
        o = (o.view(T, s["top_k"], H) * s["weights"][:, :, None]).sum(1)
        if s["sh"] is not None:
            o = o + s["sh"].float()
    if s["pg"] is not None:
        o = o / torch.sqrt((o * o).mean(1, keepdim=True) + EPS) * s["pg"].float()
    if s["g"] is not None:
        o = o * s["g"].float()
    h = o if s["r"] is None else s["alpha"] * s["r"].float() + o
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["gamma"].float()
    out = [h.bfloat16(), y.bfloat16()]
    if s["quant"] == "fp8":
        b = y.view(T, H // 128, 128)
        sc = b.abs().amax(-1).clamp_min(1e-10) / 448
        q = b * (1 / sc)[..., None]
    elif s["quant"] == "mxfp8":
        b = y.view(T, H // 32, 32)
        amax = b.abs().amax(-1)
        exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp(-127, 127)
        q = torch.ldexp(b, -exponent[..., None])
        sc = (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        return out
    return out + [q.clamp(-448, 448).to(torch.float8_e4m3fn).view(T, H), sc]


# --------------------------------------------------------------------------- what a pass needs
def work(case):
    if case["op"] == "linear":
        M, N, K, size = case["M"], case["N"], case["K"], 4 if case["f32"] else 2
        moved = 2 * K * (M + N) + M * N * size * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": moved, "flops": 2.0 * M * N * K}
    T = case["T"]
    if case["op"] == "route":
        E, k, _ = ROUTERS[case["router"]]
        return {"bytes": T * E * (2 if case["bf16"] else 4) + (4 * E if case["bias"] else 0) + 16 * T * k + 4 * (E + 1),
                "flops": T * E * 8}
    H, k = case["H"], case["top_k"]
    read = 2 * max(k, 1) + 2 * case["shared"] + 2 * (case["gate"] == "full") + 2 * case["residual"]
    written = 4 + (1 if case["quant"] else 0)
    scales = {"fp8": H / 32, "mxfp8": H / 32, None: 0}[case["quant"]]
    vectors = 2 * H * (1 + case["post"] + (case["gate"] == "row"))
    return {"bytes": T * (H * (read + written) + scales + 4 * k) + vectors, "flops": T * H * (16 + 2 * k)}


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """Values before their last rounding, in 64 bits. Quantised values are given as value / scale, unrounded."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
        if s["b"] is not None:
            z += s["b"].double()
        z = {None: lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.special.expit(v),
             "gelu": lambda v: v * torch.special.ndtr(v), "sigmoid": torch.special.expit}[case["act"]](z)
        return z if s["r"] is None else z.add_(s["r"].double())
    if case["op"] == "route":
        E, k, _ = ROUTERS[case["router"]]
        lg = s["logits"].double()
        p = torch.special.expit(lg) if case["score"] == "sigmoid" else torch.exp(lg - torch.logsumexp(lg, 1, keepdim=True))
        sel = p + (0 if s["b"] is None else s["b"].double())
        if case["groups"] > 1:
            per = sel.unflatten(1, (case["groups"], -1))
            first = per.amax(2)
            total = first.clone()
            if case["group_top"] == 2:
                total += per.kthvalue(per.shape[2] - 1, dim=2).values
            rank = total.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
            per[rank >= case["top_groups"]] = -math.inf
            sel = per.flatten(1)
        order = sel.argsort(dim=1, descending=True, stable=True)[:, :k]
        w = torch.take_along_dim(p, order, 1) * ROUTE_SCALE
        if case["renormalise"]:
            w *= ROUTE_SCALE / w.sum(1, keepdim=True)
        return [None, w, None, None, None]

    def rms(v):
        return torch.linalg.vector_norm(v, dim=1, keepdim=True).square().div(v.shape[1]).add(EPS).rsqrt()

    o = s["x"].double()
    if case["top_k"]:
        o = torch.bmm(s["weights"].double()[:, None], o.unflatten(0, (-1, case["top_k"])))[:, 0]
    if s["sh"] is not None:
        o = o + s["sh"].double()
    if s["pg"] is not None:
        o = o * rms(o) * s["pg"].double()
    if s["g"] is not None:
        o = o * s["g"].double()
    if s["r"] is not None:
        o = o.add(s["r"].double(), alpha=s["alpha"])
    y = o * rms(o) * s["gamma"].double()
    if case["quant"] is None:
        return [o, y]
    blocks = y.unflatten(1, (-1, 128 if case["quant"] == "fp8" else 32))
    top = blocks.abs().amax(-1)
    if case["quant"] == "fp8":
        sc = torch.maximum(top, torch.full_like(top, 1e-10)) / 448
    else:
        sc = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 8), 2.0 ** -127)
    return [o, y, (blocks / sc[..., None]).flatten(1), sc]
