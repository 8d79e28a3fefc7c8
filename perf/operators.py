"""Measured cases of the operators around the layer in a training step: layer norm (forward and backward, with the
residual sum), the router's auxiliary losses with their gradient, the global gradient norm and the AdamW step.

`run` makes one pass: with `own` false in plain torch operations (fp32, whatever the inputs' type), with `own` true
through the library's entry points.  `exact` restates each operator in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5                       # layer norm
BALANCE, ZLOSS = 1e-2, 1e-3      # coefficients of the two router losses
HYPER = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
STEP = 1000                      # optimizer steps done before the pass
BLOCK = 128                      # values per scale of the 8-bit states
E4M3_MAX = 448.0
TINY = 2.0 ** -100               # a block whose maximum is below this is stored as zeros


def listed():
    """Sizes: the layer shapes of workloads/ (tiny; small, the 7B-A1B class; t1 and long, one layer of the 951.9B
    model) and odd ones between them."""
    return [
        # latency of the norm before the tiny layer
        dict(name="norm fwd, tiny layer", kind="norm_fwd", T=256, d=128, dtype="bfloat16", wdtype="float32",
             bias=True, residual=False),
        # one 64k-token sequence, the residual stream updated on the way
        dict(name="norm fwd, 64k tokens + residual", kind="norm_fwd", T=65536, d=6144, dtype="bfloat16",
             wdtype="bfloat16", bias=True, residual=True),
        # a ragged batch of a fp32 model of odd width
        dict(name="norm bwd, odd fp32", kind="norm_bwd", T=4095, d=1001, dtype="float32", wdtype="float32",
             bias=True, residual=False),
        # the 951.9B model's layer, the residual path's gradient added
        dict(name="norm bwd, 1T layer + residual", kind="norm_bwd", T=16384, d=6144, dtype="bfloat16",
             wdtype="float32", bias=True, residual=True),
        # router losses of the tiny layer: latency
        dict(name="router loss, tiny layer", kind="router_loss", T=256, E=8, k=2, padding=0, accumulate=False),
        # 64k tokens over 384 experts with a padded tail, added to the layer's logit gradient
        dict(name="router loss, 64k tokens", kind="router_loss", T=65536, E=384, k=8, padding=3001, accumulate=True),
        # gradient norm of a few tiny layers: 24 small tensors, latency
        dict(name="grad norm, 4 tiny layers", kind="grad_norm", layers=4, E=8, d=128, f=64, param="float32"),
        # gradient norm of a 7B-A1B-class layer, bf16 gradients
        dict(name="grad norm, 7B-A1B layer", kind="grad_norm", layers=1, E=64, d=2048, f=1024, param="bfloat16"),
        # fp32 training of a few tiny layers: 24 small tensors, latency
        dict(name="adamw, 4 tiny layers", kind="adamw", layers=4, E=8, d=128, f=64, param="float32", master=False,
             bits=32),
        # a 7B-A1B-class layer, bf16 weights with fp32 masters and fp32 states
        dict(name="adamw, 7B-A1B layer", kind="adamw", layers=1, E=64, d=2048, f=1024, param="bfloat16",
             master=True, bits=32),
        # ragged tensors that end inside a block of scales, 8-bit states, no masters
        dict(name="adamw 8-bit, odd tensors", kind="adamw", layers=6, E=5, d=333, f=211, param="bfloat16",
             master=False, bits=8),
        # 16 of the 384 experts of the 951.9B model's layer (one of 24 ranks), 8-bit states with fp32 masters
        dict(name="adamw 8-bit, 16 experts of the 1T layer", kind="adamw", layers=1, E=16, d=6144, f=1792,
             param="bfloat16", master=True, bits=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd", "router_loss", "grad_norm", "adamw", "adamw",
                       "adamw"])
    if kind in ("norm_fwd", "norm_bwd"):
        d = _log_int(rng, 32, 16384)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        # the backward reads and writes half as much again as the forward: up to the listed sizes
        T = _log_int(rng, 1, max(1, min(65536, (65536 if kind == "norm_fwd" else 16384) * 6144 // d)))
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        if dtype == "float32":
            T = max(1, T // 2)
        return dict(kind=kind, T=T, d=d, dtype=dtype, wdtype=rng.choice(["float32", dtype]), bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5)
    if kind == "router_loss":
        T, E = _log_int(rng, 1, 65536), _log_int(rng, 2, 384)
        return dict(kind=kind, T=T, E=E, k=rng.randint(1, min(E, 8)),
                    padding=rng.randint(0, T // 4) if rng.random() < 0.5 else 0, accumulate=rng.random() < 0.5)
    layers, E = _log_int(rng, 1, 32), _log_int(rng, 1, 64)
    d, f = _log_int(rng, 32, 6144), _log_int(rng, 16, 1792)
    if rng.random() < 0.5:
        d, f = max(64, d // 64 * 64), max(64, f // 64 * 64)
    while layers > 1 and 3 * layers * E * d * f > 400e6:
        layers //= 2
    while 3 * layers * E * d * f > 400e6:
        E //= 2
    case = dict(kind=kind, layers=layers, E=E, d=d, f=f, param=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))
    if kind == "adamw":
        case.update(master=case["param"] != "float32" and rng.random() < 0.7, bits=rng.choice([8, 32]))
    return case


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return getattr(torch, name)


def _rows(T, d, dtype, gen, spread=1.0):
    """Hidden states: normal rows with channels of different size, a few large ones, and an offset."""
    channel = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    channel[:: 61] *= 8.0
    shift = 0.3 * torch.randn(d, generator=gen, device="cuda")
    out = torch.empty(T, d, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // d)
    for r in range(0, T, step):
        n = min(step, T - r)
        out[r:r + n] = spread * (torch.randn(n, d, generator=gen, device="cuda") * channel + shift)
    return out


def _norm_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, d, dt, wdt = case["T"], case["d"], _dtype(case["dtype"]), _dtype(case["wdtype"])
    s = dict(w=(1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(wdt),
             b=(0.1 * torch.randn(d, generator=gen, device="cuda")).to(wdt) if case["bias"] else None)
    s["x"] = _rows(T, d, dt, gen)
    s["res"] = _rows(T, d, dt, gen, 0.5) if case["residual"] else None
    if case["kind"] == "norm_bwd":
        # what the forward left: the normalised rows' statistics, and the gradients that reach y and the residual sum
        mean, rstd = torch.empty(2, T, device="cuda").unbind(0)
        step = max(1, (1 << 27) // d)
        for r in range(0, T, step):
            z = s["x"][r:r + step].double()
            mean[r:r + step] = z.mean(1)
            rstd[r:r + step] = 1.0 / torch.sqrt(z.var(1, unbiased=False) + EPS)
        s["stats"] = torch.stack([mean, rstd])
        s["dy"] = _rows(T, d, dt, gen, 1e-3)
        if case["residual"]:
            s["res"] = s["res"] * 2e-3
    return s


def _router_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, E, k = case["T"], case["E"], case["k"]
    bias = torch.randn(E, generator=gen, device="cuda")  # some experts are preferred
    logits = torch.randn(T, E, generator=gen, device="cuda") + bias
    keep = None
    if case["padding"]:
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[T - case["padding"]:] = False
    top = torch.topk(logits[: T - case["padding"]], k, dim=1).indices.reshape(-1)
    counts = torch.bincount(top, minlength=E).to(torch.int32)
    grad = 1e-4 * torch.randn(T, E, generator=gen, device="cuda") if case["accumulate"] else None
    return dict(logits=logits, counts=counts, keep=keep, grad=grad)


def _sizes(case):
    """Values of each tensor of the list: (matrices, vectors).  A layer has its experts' three projections and the
    router as matrices, and the norm's weight and bias as vectors."""
    E, d, f = case["E"], case["d"], case["f"]
    return [E * d * f, E * d * f, E * d * f, d * E] * case["layers"], [d, d] * case["layers"]


def _offsets(sizes):
    at, o = [], 0
    for n in sizes:
        at.append(o)
        o += -(-n // BLOCK) * BLOCK
    return at, o


def _list_inputs(case, seed):
    """Tensors as views of one buffer for each role, each at a multiple of 128 values: the gradients, and for the
    optimizer the parameters, masters and states in mid-training.  The vectors are fp32 with fp32 states, undecayed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    groups = []
    for vec, sizes in enumerate(_sizes(case)):
        at, total = _offsets(sizes)
        valid = torch.ones(total, dtype=torch.bool, device="cuda")
        for o, n, e in zip(at, sizes, at[1:] + [total]):
            valid[o + n:e] = False
        rows = total // BLOCK
        size = 1e-4 * torch.exp(1.5 * torch.randn(rows, 1, generator=gen, device="cuda"))

        def normal():
            return (torch.randn(rows, BLOCK, generator=gen, device="cuda") * size).reshape(-1) * valid

        dt = torch.float32 if vec else _dtype(case["param"])
        g = dict(sizes=sizes, at=at, grad=normal().to(dt))
        if case["kind"] == "adamw":
            p = 0.02 * torch.randn(total, generator=gen, device="cuda") * valid
            g["master"] = p if case["master"] and not vec else None
            g["param"] = p.to(dt) if dt != torch.float32 else p
            g["m"] = 0.3 * normal()
            g["v"] = (0.05 * normal().square() + 0.4 * normal().square()) * valid
            g["decay"] = 0.0 if vec else 1.0
            g["ms"] = g["vs"] = None
            if case["bits"] == 8 and not vec:
                g["m"], g["ms"] = _encode(g["m"], False)
                g["v"], g["vs"] = _encode(torch.sqrt(g["v"]), True)
        groups.append(g)
    s = dict(groups=groups, step=STEP)
    if case["kind"] == "adamw":
        s["clip"] = torch.tensor([2.5, 0.4], device="cuda")  # a gradient norm of 2.5 clipped to 1
    return s


def _views(group, role):
    t = group[role]
    if t is None:
        return [None] * len(group["sizes"])
    if role in ("ms", "vs"):
        return [t[o // BLOCK: o // BLOCK + -(-n // BLOCK)] for o, n in zip(group["at"], group["sizes"])]
    return [t[o:o + n] for o, n in zip(group["at"], group["sizes"])]


def prepare(case, seed):
    kind = case["kind"]
    if kind in ("norm_fwd", "norm_bwd"):
        s = _norm_inputs(case, seed)
    elif kind == "router_loss":
        s = _router_inputs(case, seed)
    else:
        s = _list_inputs(case, seed)
        if own:  # the handle that a training program keeps for its list of tensors
            import sparse_expert_gb300 as moe
            every = {r: [t for g in s["groups"] for t in _views(g, r)]
                     for r in (("grad",) if kind == "grad_norm" else ("param", "grad", "master", "m", "v", "ms", "vs"))}
            if kind == "grad_norm":
                s["plan"] = moe.moe_tensor_list(every["grad"])
            else:
                s["plan"] = moe.moe_adamw_plan(every["param"], every["grad"], every["m"], every["v"],
                                               m_scales=every["ms"], v_scales=every["vs"], masters=every["master"],
                                               decay=[g["decay"] for g in s["groups"] for _ in g["sizes"]])
    s["case"] = case
    return s


# --------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_expert_gb300 as moe
    kind = s["case"]["kind"]
    if kind == "norm_fwd":
        return moe.moe_layer_norm(s["x"], s["w"], s["b"], eps=EPS, residual=s["res"])
    if kind == "norm_bwd":
        return moe.moe_layer_norm_backward(s["dy"], s["x"], s["stats"], s["w"], bias=s["b"] is not None, dz=s["res"])
    if kind == "router_loss":
        return moe.moe_router_loss(s["logits"], s["counts"], BALANCE, ZLOSS, mask=s["keep"], accumulate=s["grad"])
    if kind == "grad_norm":
        return moe.moe_grad_norm(s["plan"], max_norm=1.0)
    s["step"] += 1
    moe.moe_adamw_step(s["plan"], step=s["step"], clip=s["clip"], **HYPER)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """The updated buffers; 8-bit states as E4M3 values beside their scales."""
    return [{r: g[r].view(torch.float8_e4m3fn) if g[r].dtype == torch.uint8 else g[r]
             for r in ("param", "master", "m", "v", "ms", "vs") if g[r] is not None} for g in s["groups"]]


def _run_plain(s):
    kind = s["case"]["kind"]
    if kind == "norm_fwd":
        z = s["x"]
        if s["res"] is not None:
            z = (z.float() + s["res"].float()).to(z.dtype)
        y, stats = _norm_plain(z.float(), s["w"].float(), 0.0 if s["b"] is None else s["b"].float())
        return (y.to(z.dtype), stats) if s["res"] is None else (y.to(z.dtype), stats, z)
    if kind == "norm_bwd":
        dx, dw, db = _norm_bwd_plain(s["dy"].float(), s["x"].float(), s["stats"], s["w"].float())
        if s["res"] is not None:
            dx = dx + s["res"].float()
        return dict(dx=dx.to(s["x"].dtype), dweight=dw, dbias=db if s["b"] is not None else None)
    if kind == "router_loss":
        return _router_plain(s["logits"], s["counts"], s["keep"], s["grad"])
    if kind == "grad_norm":
        norm = torch.sqrt(torch.stack([g["grad"].float().square().sum() for g in s["groups"]]).sum())
        return torch.stack([norm, torch.where(norm > 1.0, torch.ones_like(norm) / norm, torch.ones_like(norm))])
    s["step"] += 1
    [_adamw_plain(g, s["step"], s["clip"][1]) for g in s["groups"]]
    return _adamw_outputs(s)


def _norm_plain(z, w, b):
    mean = z.mean(1)
    c = z - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + EPS)
    return c * rstd[:, None] * w + b, torch.stack([mean, rstd])


def _norm_bwd_plain(dy, z, stats, w):
    xhat = (z - stats[0][:, None]) * stats[1][:, None]
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    return (g - c1 - xhat * c2) * stats[1][:, None], (dy * xhat).sum(0), dy.sum(0)


def _router_plain(logits, counts, keep, grad):
    T, E = logits.shape
    f = counts.float() / counts.sum()
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    p, lse = e / total, top + torch.log(total)
    dot = (p * f).sum(1, keepdim=True)
    live = torch.ones(T, 1, device=logits.device) if keep is None else keep.float()[:, None]
    n = live.sum()
    d = p * (BALANCE * E * (f - dot) + 2.0 * ZLOSS * lse) * (live / n)
    losses = torch.stack([E * (dot * live).sum() / n, (lse * lse * live).sum() / n])
    if grad is not None:
        d = grad.add_(d)
    return losses, d


def _encode(x, positive):
    """E4M3 codes and one scale for every 128 values; a positive value keeps at least the smallest code."""
    rows = x.reshape(-1, BLOCK)
    top = rows.abs().amax(1)
    small = top < TINY
    scale = torch.where(small, torch.ones_like(top), top * (1.0 / E4M3_MAX))
    inv = torch.where(small, torch.ones_like(top), torch.full_like(top, E4M3_MAX) / top)
    q = (rows * inv[:, None]).to(torch.float8_e4m3fn)
    if positive:
        q = torch.where((rows > 0) & (q.float() == 0), torch.full_like(rows, 2.0 ** -9), q.float()).to(q.dtype)
    return q.view(torch.uint8).reshape(-1), scale


def _decode(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float().reshape(-1, BLOCK) * scales[:, None]).reshape(-1)


def _adamw_plain(g, step, scale):
    b1, b2 = HYPER["betas"]
    grad = g["grad"].float() * scale
    m = g["m"] if g["ms"] is None else _decode(g["m"], g["ms"])
    v = g["v"] if g["vs"] is None else _decode(g["v"], g["vs"]).square()
    m = m * b1 + grad * (1.0 - b1)
    v = v * b2 + (grad * grad) * (1.0 - b2)
    root = torch.sqrt(v)
    update = m * (HYPER["lr"] / (1.0 - b1 ** step)) / (root * (1.0 / math.sqrt(1.0 - b2 ** step)) + HYPER["eps"])
    p = g["param"].float() if g["master"] is None else g["master"]
    p = p - (p * (HYPER["lr"] * HYPER["weight_decay"] * g["decay"]) + update)
    g["param"].copy_(p)
    if g["master"] is not None:
        g["master"].copy_(p)
    if g["ms"] is None:
        g["m"].copy_(m)
        g["v"].copy_(v)
    else:
        for values, role, scales, positive in ((m, "m", "ms", False), (root, "v", "vs", True)):
            codes, sc = _encode(values, positive)
            g[role].copy_(codes)
            g[scales].copy_(sc)


# ------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    kind = case["kind"]
    size = {"bfloat16": 2, "float16": 2, "float32": 4}
    if kind in ("norm_fwd", "norm_bwd"):
        n, e = case["T"] * case["d"], size[case["dtype"]]
        w = case["d"] * size[case["wdtype"]]
        if kind == "norm_fwd":
            return dict(bytes=n * e * (4 if case["residual"] else 2) + w * (1 + case["bias"]) + 8 * case["T"],
                        flops=n * (8 + case["residual"]))
        return dict(bytes=n * e * (4 if case["residual"] else 3) + w + 4 * case["d"] * (1 + case["bias"]) + 8 * case["T"],
                    flops=n * (14 + case["residual"]))
    if kind == "router_loss":
        live, n = (case["T"] - case["padding"]) * case["E"], case["T"] * case["E"]
        # with an accumulated gradient the padded rows need not be touched; without one they are written
        return dict(bytes=4 * (3 * live if case["accumulate"] else live + n) + (case["T"] if case["padding"] else 0)
                    + 4 * case["E"] + 8, flops=10 * live)
    mats, vecs = (sum(s) for s in _sizes(case))
    p = size[case["param"]]
    if kind == "grad_norm":
        return dict(bytes=mats * p + vecs * 4 + 8, flops=2 * (mats + vecs))
    per = p + (4 + 4 + p if case["master"] else 2 * p)          # gradient in; weights in and out
    per += 16 if case["bits"] == 32 else 4 + 16 / BLOCK         # states in and out
    return dict(bytes=mats * per + vecs * 28, flops=16 * (mats + vecs))


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    kind = case["kind"]
    if kind in ("norm_fwd", "norm_bwd"):
        s = _norm_inputs(case, seed)
        return _exact_norm(s) if kind == "norm_fwd" else _exact_norm_bwd(s)
    if kind == "router_loss":
        return _exact_router(**_router_inputs(case, seed))
    s = _list_inputs(case, seed)
    if kind == "grad_norm":
        norm = math.sqrt(sum(float(g["grad"].double().pow(2).sum()) for g in s["groups"]))
        return torch.tensor([norm, min(1.0, 1.0 / norm) if norm > 0 else 1.0], dtype=torch.float64)
    return [_exact_adamw(g, float(s["clip"][1]), case) for g in s["groups"]]


def _exact_norm(s):
    T, d = s["x"].shape
    y, stats = torch.empty(T, d, dtype=torch.float64, device="cuda"), torch.empty(2, T, dtype=torch.float64, device="cuda")
    z_all = torch.empty_like(s["x"])
    for t in range(0, T, 8192):
        r = slice(t, t + 8192)
        z = s["x"][r].double()
        if s["res"] is not None:
            z_all[r] = z + s["res"][r].double()
            z = z_all[r].double()
        mu = z.sum(1) / d
        rstd = (torch.pow(z - mu[:, None], 2).sum(1) / d + EPS).rsqrt()
        stats[0, r], stats[1, r] = mu, rstd
        y[r] = (z - mu[:, None]) * rstd[:, None] * s["w"].double()
        if s["b"] is not None:
            y[r] += s["b"].double()
    return (y, stats) if s["res"] is None else (y, stats, z_all.double())


def _exact_norm_bwd(s):
    T, d = s["x"].shape
    dx = torch.empty(T, d, dtype=torch.float64, device="cuda")
    dw, db = torch.zeros(2, d, dtype=torch.float64, device="cuda")
    for t in range(0, T, 8192):
        r = slice(t, t + 8192)
        mu, rstd = s["stats"][0, r, None].double(), s["stats"][1, r, None].double()
        n = (s["x"][r].double() - mu) * rstd
        dy = s["dy"][r].double()
        dw += torch.einsum("td,td->d", dy, n)
        db += dy.sum(0)
        dn = dy * s["w"].double()
        dx[r] = rstd * (dn - (dn.sum(1, keepdim=True) + n * (dn * n).sum(1, keepdim=True)) / d)
        if s["res"] is not None:
            dx[r] += s["res"][r].double()
    return dict(dx=dx, dweight=dw, dbias=db if s["b"] is not None else None)


def _exact_router(logits, counts, keep, grad):
    T, E = logits.shape
    share = counts.double() / float(counts.sum())
    live = torch.ones(T, dtype=torch.float64, device="cuda") if keep is None else keep.double()
    l64 = logits.double()
    lse = torch.logsumexp(l64, 1)
    p = torch.exp(l64 - lse[:, None])
    n = float(live.sum())
    # balance = E sum_e share_e mean_t p_te,  z = mean_t lse_t^2, differentiated through the softmax
    dp = BALANCE * E * share / n
    dl = p * (dp[None, :] - (p @ dp)[:, None]) + (2.0 * ZLOSS / n * lse)[:, None] * p
    dl = dl * live[:, None]
    balance = E * float((share * ((p * live[:, None]).sum(0) / n)).sum())
    losses = torch.tensor([balance, float((lse.pow(2) * live).sum()) / n], dtype=torch.float64)
    return losses, dl if grad is None else grad.double() + dl


def _exact_adamw(g, scale, case):
    b1, b2 = HYPER["betas"]
    t = STEP + 1

    def state(codes, scales):
        return codes.double() if scales is None else \
            codes.view(torch.float8_e4m3fn).to(torch.float64) * scales.double().repeat_interleave(BLOCK)

    grad = g["grad"].double() * scale
    m = b1 * state(g["m"], g["ms"]) + (1 - b1) * grad
    v = state(g["v"], g["vs"])
    v = b2 * (v if g["vs"] is None else v * v) + (1 - b2) * grad * grad
    del grad
    p = (g["param"] if g["master"] is None else g["master"]).double()
    p = p - HYPER["lr"] * (m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + HYPER["eps"])
                           + HYPER["weight_decay"] * g["decay"] * p)
    out = dict(param=p, m=m, v=v)
    if g["master"] is not None:
        out["master"] = p
    if g["ms"] is not None:
        for role, x in (("m", m), ("v", v.sqrt_())):
            rows = x.view(-1, BLOCK)
            top = rows.abs().amax(1, keepdim=True)
            unit = torch.where(top < TINY, 1.0, top / E4M3_MAX)
            code = (rows / unit).float().to(torch.float8_e4m3fn).float()
            if role == "v":
                code[(rows > 0) & (code == 0)] = 2.0 ** -9
            out[role], out[role + "s"] = code.reshape(-1), unit.reshape(-1)
    return out
