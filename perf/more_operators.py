"""Measured cases of the operators for serving a few tokens: the whole layer for 1 to 64 tokens (bf16, FP8 and 4-bit
expert weights; from the router's logits or from its weights) and the product of a few rows with 4-bit weights.

`run` makes one pass: with `own` false in plain torch operations (fp32, whatever the inputs' type; the router's logits
in fp64, because the choice of experts turns on their last bits), with `own` true through the library's entry points.
`exact` restates each operator in 64 bits.
"""
import math

import torch

own = False


def listed():
    """Sizes: the layer shapes of workloads/ (tiny; small, the 7B-A1B class; t1, one layer of the 951.9B model) and odd
    ones between them."""
    return [
        # latency: one token through the tiny layer
        dict(name="few, 1 token, tiny layer", kind="few", weights="bf16", T=1, d=128, E=8, k=2, f=64),
        # decoding one sequence with a 7B-A1B-class layer
        dict(name="few, 1 token, 7B-A1B layer", kind="few", weights="bf16", T=1, d=2048, E=64, k=8, f=1024),
        # decoding a batch of 64: nearly every expert is hit
        dict(name="few, 64 tokens, 7B-A1B layer", kind="few", weights="bf16", T=64, d=2048, E=64, k=8, f=1024),
        # a small batch on one layer of the 951.9B model
        dict(name="few, 4 tokens, 1T layer", kind="few", weights="bf16", T=4, d=6144, E=384, k=8, f=1792),
        # one token of that layer from the hidden state alone: router, choice and experts
        dict(name="few routed, 1 token, 1T layer", kind="few_routed", weights="bf16", T=1, d=6144, E=384, k=8, f=1792),
        # an odd layer: 40 experts, 5 a token, sizes that are multiples of 64 alone
        dict(name="few routed, 23 tokens, odd layer", kind="few_routed", weights="bf16", T=23, d=832, E=40, k=5,
             f=1472),
        # FP8 weights: one sequence, 7B-A1B class
        dict(name="few fp8, 1 token, 7B-A1B layer", kind="few", weights="fp8", T=1, d=2048, E=64, k=8, f=1024),
        # FP8 weights: a batch of 32 on the 951.9B model's layer
        dict(name="few fp8, 32 tokens, 1T layer", kind="few", weights="fp8", T=32, d=6144, E=384, k=8, f=1792),
        # 4-bit weights: one sequence on the 951.9B model's layer
        dict(name="few int4, 1 token, 1T layer", kind="few", weights="int4", group=128, T=1, d=6144, E=384, k=8,
             f=1792),
        # 4-bit weights with short groups, a batch of 48, 7B-A1B class
        dict(name="few int4, 48 tokens, 7B-A1B layer", kind="few", weights="int4", group=32, T=48, d=2048, E=64, k=8,
             f=1024),
        # a dense projection beside the layer, one token: latency
        dict(name="linear int4, 1 x 2048 x 2048", kind="linear", group=128, M=1, K=2048, N=2048),
        # an output head over a large, odd vocabulary for 13 sequences
        dict(name="linear int4, 13 x 6144 x 128001", kind="linear", group=64, M=13, K=6144, N=128001),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["few", "few", "few", "few_routed", "linear"])
    if kind == "linear":
        K, N = _log_int(rng, 64, 16384) // 8 * 8, _log_int(rng, 1, 131072)
        return dict(kind=kind, group=rng.choice([32, 64, 128]), M=rng.randint(1, 16), K=K, N=min(N, 786_000_000 // K))
    weights = "bf16" if kind == "few_routed" else rng.choice(["bf16", "fp8", "int4"])
    unit = 64 if weights == "bf16" else 128
    E = _log_int(rng, 1, 384)
    case = dict(kind=kind, weights=weights, T=_log_int(rng, 1, 64), d=max(1, _log_int(rng, 64, 8192) // unit) * unit, E=E,
                k=rng.randint(1, min(E, 10)), f=max(1, _log_int(rng, 64, 4096) // unit) * unit)
    while 3 * case["E"] * case["d"] * case["f"] > (3.0e9 if weights == "bf16" else 4.2e9):
        case["f"] = max(1, case["f"] // unit // 2) * unit
    if weights == "int4":
        case["group"] = rng.choice([32, 64, 128])
    return case


# ------------------------------------------------------------------ inputs
def _codes4(shape, gen):
    """4-bit codes of normal weights (mean 8, 15 steps over the range), two rows of K a byte."""
    q = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(2.4).add_(8).round_().clamp_(0, 15)
    q = q.to(torch.uint8)
    return q[..., 0::2, :] | (q[..., 1::2, :] << 4)


def _matrices(case, K, N, gen):
    """Weights [E, K, N] that multiply rows of K values: bf16, or codes with their scales."""
    E, unit = case.get("E"), 1.0 / math.sqrt(K)
    lead = () if E is None else (E,)
    kind = case.get("weights", "int4")
    if kind == "bf16":
        return torch.randn(*lead, K, N, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(unit)
    if kind == "fp8":  # one scale for 128 stored values, the largest near 448
        codes = torch.randn(*lead, K, N, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(160).clamp_(-448, 448)
        scales = torch.exp(0.2 * torch.randn(E * K * N // 128, generator=gen, device="cuda")).mul_(unit / 160)
        return codes.to(torch.float8_e4m3fn).view(torch.uint8), scales
    groups = -(-K // case["group"])
    scales = torch.exp(0.2 * torch.randn(*lead, groups, N, generator=gen, device="cuda")).mul_(unit / 2.4)
    return _codes4((*lead, K, N), gen), scales.to(torch.bfloat16)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, width = (case["M"], case["K"]) if case["kind"] == "linear" else (case["T"], case["d"])
    # hidden states behind a norm: channels of different size
    channel = torch.exp(0.3 * torch.randn(width, generator=gen, device="cuda"))
    s = dict(case=case, x=(torch.randn(rows, width, generator=gen, device="cuda") * channel).to(torch.bfloat16))
    if case["kind"] == "linear":
        s["w"] = _matrices(case, case["K"], case["N"], gen)
        return s
    E, d, f = case["E"], case["d"], case["f"]
    if case["kind"] == "few":
        bias = 0.3 * torch.randn(E, generator=gen, device="cuda")  # some experts are preferred
        s["logits"] = torch.randn(rows, E, generator=gen, device="cuda") + bias
    else:
        s["router"] = (torch.randn(d, E, generator=gen, device="cuda") / math.sqrt(d)).to(torch.bfloat16)
    s["gate"], s["up"], s["down"] = (_matrices(case, K, N, gen) for K, N in ((d, f), (d, f), (f, d)))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    # a serving program has the weights in the library's layout, and keeps a workspace
    import sparse_expert_gb300 as moe
    if case["kind"] == "linear":
        s["w"] = moe.moe_pack_linear_int4(*s["w"], case["K"], case["N"], case["group"])
        return s
    sizes = [case[n] for n in ("E", "d", "f")]
    mats = [s.pop(n) for n in ("gate", "up", "down")]
    if case["weights"] == "bf16":
        s["packed"] = moe.moe_pack_weights(*mats)
    elif case["weights"] == "fp8":
        s["packed"] = moe.moe_pack_weights_fp8(*mats, *sizes)
    else:
        s["packed"] = moe.moe_pack_weights_int4(*mats, *sizes, case["group"])
    if case["kind"] == "few_routed":
        s["router"] = moe.moe_pack_router_weights(s["router"])
    s["workspace"] = torch.empty(moe.moe_forward_few_workspace_bytes(case["T"], case["E"], case["k"], case["d"], case["f"]),
                                 dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_expert_gb300 as moe
    c = s["case"]
    if c["kind"] == "linear":
        return moe.moe_linear_int4(s["x"], s["w"], c["N"], c["group"])
    call, route = (moe.moe_forward_few, "logits") if c["kind"] == "few" else (moe.moe_forward_few_routed, "router")
    return call(s["x"], s[route], s["packed"], c["E"], c["k"], c["f"], weights=c["weights"], group=c.get("group", 128),
                workspace=s["workspace"])


def _fp32(w, case, pick):
    """The matrices `pick` ([n, K, N], or all of them) in fp32."""
    if case.get("weights") == "bf16":
        return (w if pick is None else w[pick]).float()
    codes, scales = w
    if case.get("weights") == "fp8":
        scales = scales.view(*codes.shape[:2], -1)
        codes, scales = (codes, scales) if pick is None else (codes[pick], scales[pick])
        v = codes.view(torch.float8_e4m3fn).float().view(*scales.shape, 128)
        return (v * scales[..., None]).view(codes.shape)
    codes, scales = (codes, scales) if pick is None else (codes[pick], scales[pick])
    q = torch.stack([codes & 15, codes >> 4], -2).flatten(-3, -2).float() - 8.0
    return q * scales.float().repeat_interleave(case["group"], -2)[..., : q.shape[-2], :]


def _run_plain(s):
    c, x = s["case"], s["x"].float()
    if c["kind"] == "linear":
        return (x @ _fp32(s["w"], c, None)).to(torch.bfloat16)
    logits = s["logits"] if c["kind"] == "few" else x.double() @ s["router"].double()
    best, idx = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: the lowest index first
    best, idx = best[:, : c["k"]].float(), idx[:, : c["k"]]
    w = torch.exp(best - best[:, :1])
    w = w / w.sum(1, keepdim=True)
    if idx.numel() <= c["E"]:  # the chosen experts' matrices, pair by pair
        rows, pick = x.repeat_interleave(c["k"], 0)[:, None, :], idx.reshape(-1)
    else:                      # every expert on every token, weighted by its gate or by nothing
        rows, pick = x[None], None
    g, u = rows @ _fp32(s["gate"], c, pick), rows @ _fp32(s["up"], c, pick)
    y = (g / (1.0 + torch.exp(-g)) * u) @ _fp32(s["down"], c, pick)
    if pick is not None:
        y = (y.view(*idx.shape, -1) * w[..., None]).sum(1)
    else:
        gates = torch.zeros(x.shape[0], c["E"], device=x.device).scatter_(1, idx, w)
        y = (y * gates.T[..., None]).sum(0)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["kind"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return dict(bytes=K * N / 2 + 2 * -(-K // case["group"]) * N + 2 * M * (K + N), flops=2 * M * K * N)
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    per = {"bf16": 2.0, "fp8": 1.0 + 4 / 128, "int4": 0.5 + 2 / case.get("group", 128)}[case["weights"]]
    hit = E * (1.0 - (1.0 - k / E) ** T)  # experts that T tokens hit, if each expert is as likely as the others
    route = 4 * T * E if case["kind"] == "few" else 2 * d * E
    return dict(bytes=3 * hit * d * f * per + 4 * T * d + route,
                flops=6 * T * k * d * f + (2 * T * d * E if case["kind"] == "few_routed" else 0))


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    s = _inputs(case, seed)
    x = s["x"].double()

    def times(rows, w, e=None):
        """rows @ W_e, the scales applied to partial sums over their groups of inputs."""
        if case.get("weights") == "bf16":
            return torch.mm(rows, w[e].double())
        codes, scales = w if e is None else (w[0][e], None)
        if case.get("weights") == "fp8":
            K, N = codes.shape
            unit = w[1][e * K * N // 128:(e + 1) * K * N // 128].double().view(K, N // 128)
            value = codes.view(torch.float8_e4m3fn).to(torch.float64).unflatten(1, (N // 128, 128))
            return torch.einsum("tk,kb,kbn->tbn", rows, unit, value).flatten(1)
        unit = (w[1] if e is None else w[1][e]).double()
        out = torch.zeros(rows.shape[0], codes.shape[1], dtype=torch.float64, device=rows.device)
        half = case["group"] // 2
        for g in range(unit.shape[0]):
            b = codes[g * half:(g + 1) * half]
            r = rows[:, g * 2 * half:(g + 1) * 2 * half]
            low, high = torch.remainder(b, 16).double(), torch.div(b, 16, rounding_mode="floor").double()
            out += unit[g] * (r[:, 0::2] @ low + r[:, 1::2] @ high - 8.0 * r.sum(1, keepdim=True))
        return out

    if case["kind"] == "linear":
        return times(x, s["w"])
    logits = s["logits"].double() if case["kind"] == "few" else torch.mm(x, s["router"].double())
    out = torch.zeros_like(x)
    top = torch.argsort(logits, dim=1, descending=True, stable=True)[:, : case["k"]]
    share = torch.softmax(torch.gather(logits, 1, top), 1)
    for e in torch.unique(top).tolist():
        token, slot = torch.nonzero(top == e, as_tuple=True)
        r = x[token]
        h = torch.nn.functional.silu(times(r, s["gate"], e)) * times(r, s["up"], e)
        out.index_add_(0, token, share[token, slot, None] * times(h, s["down"], e))
    return out
