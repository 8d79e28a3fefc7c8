"""AdamW over lists of tensors and the gradient norm, against 64 bits; the
8-bit states also bit for bit against a plain fp32 restatement whose products
and sums are rounded one by one.

Tolerances: u = 2^-24 for each fp32 operation and each coefficient; m and v
take at most five each, the update at most twelve more.
"""
import gc
import math
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
LR, BETAS, EPS, WD = 1e-2, (0.9, 0.95), 1e-8, 0.1
ROLES = ("params", "grads", "m", "v", "m_scales", "v_scales", "masters")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_expert_gb300 as m
    return m


def encode(x, positive):
    """E4M3 codes and scales of blocks of 128 (fp32, any device)."""
    n = x.numel()
    rows = torch.nn.functional.pad(x.reshape(-1), (0, -n % 128)).view(-1, 128)
    top = rows.abs().amax(1)
    small = top < 2.0 ** -100
    one = torch.ones_like(top)
    scale = torch.where(small, one, top * torch.tensor(1.0 / 448.0, dtype=torch.float32, device=x.device))
    inv = torch.where(small, one, torch.full_like(top, 448.0) / top)
    code = (rows * inv[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        code = torch.where((rows > 0) & (code == 0), torch.ones_like(code), code)
    return code.reshape(-1)[:n].view(x.shape), scale


def decode(codes, scales, dtype=torch.float32):
    v = codes.reshape(-1).view(torch.float8_e4m3fn).to(dtype)
    return (v * scales.to(dtype).repeat_interleave(128)[: v.numel()]).view(codes.shape)


def tensors(sizes, param, grad, master, bits, seed, shift=0):
    """Lists in mid-training; with a shift, views that start so many values into their buffers."""
    g = torch.Generator().manual_seed(seed)

    def own(x):
        buf = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")
        buf[shift:] = x.reshape(-1).cuda()
        return buf[shift:]
    out = {r: [] for r in ROLES}
    for n in sizes:
        size = 1e-3 * torch.exp(2.0 * torch.randn(n, generator=g))
        p = 0.1 * torch.randn(n, generator=g)
        out["params"].append(own(p.to(param)))
        out["masters"].append(own(p) if master else None)
        out["grads"].append(own((torch.randn(n, generator=g) * size).to(grad)))
        m = 0.3 * torch.randn(n, generator=g) * size
        v = (size * torch.rand(n, generator=g)).square()
        if bits == 8:
            mc, ms = encode(m, False)
            vc, vs = encode(v.sqrt(), True)
            out["m"].append(own(mc)), out["v"].append(own(vc))
            out["m_scales"].append(own(ms)), out["v_scales"].append(own(vs))
        else:
            out["m"].append(own(m)), out["v"].append(own(v))
            out["m_scales"].append(None), out["v_scales"].append(None)
    return out


def plan_of(moe, lists, decay=None):
    return moe.moe_adamw_plan(lists["params"], lists["grads"], lists["m"], lists["v"], lists["m_scales"],
                              lists["v_scales"], lists["masters"], decay)


def copy(lists):
    return {r: [None if t is None else t.clone() for t in lists[r]] for r in ROLES}


def one_step_64(lists, i, step, factor, decay):
    """(p, m, v) of tensor i after a step, and their tolerances in fp32 before the final rounding."""
    b1, b2 = BETAS
    g = lists["grads"][i].double() * factor
    if lists["m"][i].dtype == torch.uint8:
        m = decode(lists["m"][i], lists["m_scales"][i], torch.float64)
        v = decode(lists["v"][i], lists["v_scales"][i], torch.float64).square()
    else:
        m, v = lists["m"][i].double(), lists["v"][i].double()
    p = (lists["masters"][i] if lists["masters"][i] is not None else lists["params"][i]).double()
    tol_m = 5 * U * ((b1 * m).abs() + ((1 - b1) * g).abs()) + 1e-44
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    tol_v = 8 * U * v + 1e-44
    denom = (v / (1 - b2 ** step)).sqrt() + EPS
    update = LR / (1 - b1 ** step) * m / denom
    tol_p = 14 * U * update.abs() + LR / (1 - b1 ** step) * tol_m / denom + 4 * U * LR * WD * decay * p.abs()
    p = p - (LR * WD * decay * p + update)
    return p, m, v, tol_p + U * p.abs(), tol_m, tol_v


def check_step(before, after, step, factor=1.0, decay=None):
    for i in range(len(before["params"])):
        p, m, v, tol_p, tol_m, tol_v = one_step_64(before, i, step, factor, 1.0 if decay is None else decay[i])
        got = after["params"][i]
        if after["masters"][i] is not None:
            assert torch.all((after["masters"][i].double() - p).abs() <= tol_p)
            assert torch.equal(got, after["masters"][i].to(got.dtype))
        tol = tol_p + 1.01 * ROUND[got.dtype] * p.abs() + TINY[got.dtype]
        err = (got.double() - p).abs()
        assert torch.all(err <= tol), (i, (err - tol).max().item())
        if after["m"][i].dtype == torch.uint8:
            # a code is off by half a step: 2^-4 of the value, or 2^-10 of the scale among the smallest
            for name, want, t in (("m", m, tol_m), ("v", v.sqrt(), U * 6 * v.sqrt())):
                scale = after[name + "_scales"][i].double().repeat_interleave(128)[: want.numel()]
                err = (decode(after[name][i], after[name + "_scales"][i], torch.float64) - want).abs()
                smallest = 2.0 ** (-9 if name == "v" else -10)   # a small root is kept at the smallest code
                assert torch.all(err <= 1.001 * (want.abs() / 16 + smallest * scale) + t)
        else:
            assert torch.all((after["m"][i].double() - m).abs() <= tol_m)
            assert torch.all((after["v"][i].double() - v).abs() <= tol_v)


def step_in_fp32(lists, i, step, factor):
    """The 8-bit states after a step, every product and sum rounded to fp32 on the CPU."""
    f32 = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    b1, b2 = BETAS
    g = lists["grads"][i].cpu().float() * f32(factor)
    m = decode(lists["m"][i].cpu(), lists["m_scales"][i].cpu())
    root = decode(lists["v"][i].cpu(), lists["v_scales"][i].cpu())
    m = m * f32(b1) + g * f32(1 - b1)
    v = (root * root) * f32(b2) + (g * g) * f32(1 - b2)
    return encode(m, False), encode(v.sqrt(), True)


SIZES = [1, 2, 127, 128, 129, 1000, 4095, 4096, 4097, 50000, 262144 + 77]
COMBOS = [(torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False),
          (torch.bfloat16, torch.bfloat16, True), (torch.bfloat16, torch.bfloat16, False),
          (torch.bfloat16, torch.float32, True), (torch.float16, torch.float16, True),
          (torch.float16, torch.float32, False), (torch.float32, torch.float16, True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", COMBOS)
@pytest.mark.parametrize("shift", [0, 1, 4, 8])
def test_step(moe, param, grad, master, bits, shift):
    lists = tensors(SIZES, param, grad, master, bits, seed=bits + shift, shift=shift)
    clip = torch.tensor([3.0, 0.37], device="cuda")
    plan = plan_of(moe, lists)
    for step in (1, 2, 1000):
        before = copy(lists)
        moe.moe_adamw_step(plan, lr=LR, step=step, betas=BETAS, eps=EPS, weight_decay=WD, clip=clip)
        factor = clip[1].item()
        check_step(before, lists, step, factor)
        if bits == 8:
            for i in range(len(SIZES)):
                (mc, ms), (vc, vs) = step_in_fp32(before, i, step, factor)
                assert torch.equal(lists["m"][i].cpu(), mc) and torch.equal(lists["m_scales"][i].cpu(), ms)
                assert torch.equal(lists["v"][i].cpu(), vc) and torch.equal(lists["v_scales"][i].cpu(), vs)


@pytest.mark.parametrize("n_tensors", [1, 8, 9, 48, 49, 200, 384, 385, 900])
def test_lists_of_any_length(moe, n_tensors):
    """Mixed types and states in one list, tensors without values among them."""
    sizes = [(7 * i) % 300 for i in range(n_tensors)]
    lists = {r: [] for r in ROLES}
    for i, n in enumerate(sizes):
        param, grad, master = COMBOS[i % len(COMBOS)]
        t = tensors([n], param, grad, master, 8 if i % 3 == 0 else 32, seed=i)
        for r in ROLES:
            lists[r] += t[r]
    decay = [float(i % 2) for i in range(n_tensors)]
    before = copy(lists)
    plan = plan_of(moe, lists, decay)
    assert len(plan) == n_tensors
    moe.moe_adamw_step(plan, lr=LR, step=5, betas=BETAS, eps=EPS, weight_decay=WD)
    check_step(before, lists, 5, 1.0, decay)
    want = math.sqrt(sum(g.double().square().sum().item() for g in before["grads"]))
    out = moe.moe_grad_norm(plan, max_norm=want / 2 if want else 1.0)
    assert abs(out[0].item() - want) <= 400 * U * want
    assert abs(out[1].item() - (0.5 if want else 1.0)) <= 400 * U


def test_plans_keep_their_tensors(moe):
    """Emptying the lists that a plan was made from frees nothing that its records point to."""
    lists = tensors([1000, 77], torch.bfloat16, torch.bfloat16, True, 8, seed=6)
    plan = plan_of(moe, lists)
    grads = [torch.ones(50, device="cuda") for _ in range(3)]
    listed = moe.moe_tensor_list(grads)
    kept = [weakref.ref(t) for ts in (*lists.values(), grads) for t in ts]
    for ts in (*lists.values(), grads):
        ts.clear()
    gc.collect()
    assert all(r() is not None for r in kept)
    assert len(plan) == 2 and len(listed) == 3


def test_neighbours_are_not_touched(moe):
    """Tensors side by side in one buffer, only every other one in the list."""
    n = 777
    lists = tensors([n * 6], torch.bfloat16, torch.bfloat16, True, 32, seed=3)
    before = copy(lists)
    cut = {r: [None if lists[r][0] is None else lists[r][0][k * n:(k + 1) * n] for k in (1, 3)] for r in ROLES}
    moe.moe_adamw_step(plan_of(moe, cut), lr=LR, step=1, betas=BETAS, eps=EPS, weight_decay=WD)
    for r in ("params", "masters", "m", "v"):
        for k in range(6):
            same = torch.equal(lists[r][0][k * n:(k + 1) * n], before[r][0][k * n:(k + 1) * n])
            assert same == (k not in (1, 3)), (r, k)


@pytest.mark.parametrize("bits", [32, 8])
def test_state_from_zero_over_steps(moe, bits):
    """Twenty steps from zero states follow the 64-bit recurrence: exactly up
    to rounding with fp32 states; with 8 bits each step's update has the right
    sign and at most a fifth off in size (two codes of 1/16, their history)."""
    n = 3000
    g = torch.Generator().manual_seed(8)
    p = (0.1 * torch.randn(n, generator=g)).cuda()
    grad = torch.empty(n, device="cuda")
    state = moe.moe_adamw_state([p], bits)
    plan = moe.moe_adamw_plan([p], [grad], **state)
    size = torch.exp(torch.randn(n, generator=g)).cuda() * 1e-2
    p64, m64, v64 = p.double(), torch.zeros(n, dtype=torch.float64, device="cuda"), None
    v64 = torch.zeros_like(m64)
    for t in range(1, 21):
        grad.copy_(size * (2.0 + 0.2 * torch.randn(n, generator=g).cuda()))
        moe.moe_adamw_step(plan, lr=1e-3, step=t, betas=BETAS, eps=EPS, weight_decay=0.0)
        m64 = 0.9 * m64 + 0.1 * grad.double()
        v64 = 0.95 * v64 + 0.05 * grad.double().square()
        p64 = p64 - 1e-3 * (m64 / (1 - 0.9 ** t)) / ((v64 / (1 - 0.95 ** t)).sqrt() + EPS)
    moved = 20 * 1e-3
    assert (p.double() - p64).abs().max().item() <= (20 * 40 * U * 1e-3 + 20 * U if bits == 32 else 0.2 * moved)


def test_zero_and_tiny_blocks(moe):
    """A block without gradient and state stays zero; tiny and wide blocks
    keep every positive root above zero, so no update exceeds the step."""
    n = 128 * 4
    p = torch.zeros(n, device="cuda")
    grad = torch.zeros(n, device="cuda")
    grad[128:256] = 1e-18                                     # squares at the edge of fp32
    grad[256:384] = 10.0 ** torch.linspace(-12, 0, 128, device="cuda")
    grad[384:] = 1e-40
    state = moe.moe_adamw_state([p], 8)
    plan = moe.moe_adamw_plan([p], [grad], **state)
    for t in range(1, 6):
        moe.moe_adamw_step(plan, lr=1e-2, step=t, betas=BETAS, eps=0.0 if t == 0 else 1e-30, weight_decay=0.0)
        assert torch.isfinite(p).all()
        assert not p[:128].any() and p.abs().max().item() <= 1.5e-2 * t
    assert not state["m"][0][:128].any() and torch.all(state["v"][0][256:384] > 0)
    assert torch.equal(state["m_scales"][0][:1], torch.ones(1, device="cuda"))


def test_gradients_that_are_not_finite(moe):
    lists = tensors([128 * 3], torch.bfloat16, torch.float32, True, 8, seed=1)
    wide = tensors([300], torch.float32, torch.float32, False, 32, seed=2)
    lists = {r: lists[r] + wide[r] for r in ROLES}
    lists["grads"][0][130] = float("nan")
    lists["grads"][1][7] = float("inf")
    before = copy(lists)
    plan = plan_of(moe, lists)
    norm = moe.moe_grad_norm(plan, max_norm=1.0)
    assert torch.isnan(norm).all() or (torch.isinf(norm[0]) and torch.isnan(norm[1]))
    moe.moe_adamw_step(plan, lr=LR, step=1, clip=norm)         # the whole step is skipped
    assert all(torch.equal(a, b) for r in ROLES if r != "grads" for a, b in zip(lists[r], before[r]) if a is not None)
    moe.moe_adamw_step(plan, lr=LR, step=1)                    # without a factor, NaN shows where it belongs
    assert torch.isnan(lists["m_scales"][0]).tolist() == [False, True, False]
    assert torch.isnan(lists["masters"][0]).nonzero().flatten().tolist() == [130]
    assert torch.isfinite(lists["params"][1]).sum().item() == 299


def test_infinite_gradient_norm(moe):
    g = torch.ones(1000, device="cuda")
    g[3] = float("inf")
    out = moe.moe_grad_norm([g], max_norm=1.0)
    assert math.isinf(out[0].item()) and math.isnan(out[1].item())


def test_hyper_on_the_device_and_graph_replay(moe):
    lists = tensors(SIZES, torch.bfloat16, torch.bfloat16, True, 8, seed=4)
    direct = copy(lists)
    plan, plan_direct = plan_of(moe, lists), plan_of(moe, direct)
    hyper, clip = torch.empty(8, device="cuda"), torch.empty(2, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    start = copy(lists)
    hyper.copy_(moe.moe_adamw_hyper(LR, 1, BETAS, EPS, WD))
    moe.moe_grad_norm(plan, 0.01, out=clip, workspace=ws)
    moe.moe_adamw_step(plan, hyper=hyper, clip=clip)           # warm up outside the capture
    for r in ROLES:
        for a, b in zip(lists[r], start[r]):
            if a is not None:
                a.copy_(b)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            moe.moe_grad_norm(plan, 0.01, out=clip, workspace=ws, stream=stream)
            moe.moe_adamw_step(plan, hyper=hyper, clip=clip, stream=stream)
    for step in (1, 2, 3):
        hyper.copy_(moe.moe_adamw_hyper(LR / step, step, BETAS, EPS, WD))
        for a, b in zip(lists["grads"], direct["grads"]):
            new = torch.randn(a.numel(), device="cuda").to(a.dtype) * step
            a.copy_(new), b.copy_(new)
        graph.replay()
        c = moe.moe_grad_norm(plan_direct, 0.01)
        moe.moe_adamw_step(plan_direct, lr=LR / step, step=step, betas=BETAS, eps=EPS, weight_decay=WD, clip=c)
        torch.cuda.synchronize()
        assert torch.equal(c, clip)
        assert all(torch.equal(a, b) for r in ROLES for a, b in zip(lists[r], direct[r]) if a is not None)


def test_on_another_stream(moe):
    lists = tensors([100000], torch.float32, torch.float32, False, 32, seed=5)
    other = copy(lists)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    moe.moe_adamw_step(plan_of(moe, lists), lr=LR, step=3)
    moe.moe_adamw_step(plan_of(moe, other), lr=LR, step=3, stream=s)
    a, b = moe.moe_grad_norm(lists["grads"]), moe.moe_grad_norm(other["grads"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(x, y) for r in ("params", "m", "v") for x, y in zip(lists[r], other[r]))


# ------------------------------------------------------------------ the norm
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,shift", [(0, 0), (1, 0), (5, 1), (4096, 0), (100003, 3), (3000000, 0), (20000001, 1)])
def test_grad_norm(moe, n, shift, dtype):
    g = (torch.randn(n + shift, generator=torch.Generator().manual_seed(n)) * 0.01).to(dtype).cuda()[shift:]
    want = g.double().square().sum().sqrt().item()
    out = moe.moe_grad_norm([g], max_norm=0.5)
    # squares of one sign: a relative error of one u for each addition of a thread, halved by the root
    assert abs(out[0].item() - want) <= 400 * U * want
    factor = 0.5 / want if want > 0.5 else 1.0
    assert abs(out[1].item() - factor) <= 400 * U
    again = moe.moe_grad_norm(moe.moe_tensor_list([g]), max_norm=0.5)
    assert torch.equal(out, again)
    assert moe.moe_grad_norm([g])[1].item() == 1.0


def test_grad_norm_of_nothing(moe):
    assert moe.moe_grad_norm([]).tolist() == [0.0, 1.0]


def test_offsets_beyond_32_bits(moe):
    """A tensor of more than 2^32 values: its last ones are updated and counted."""
    n = (1 << 32) + 300
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    grad[-200:] = 3.0
    state = moe.moe_adamw_state([p], 8)
    plan = moe.moe_adamw_plan([p], [grad], **state)
    assert abs(moe.moe_grad_norm(plan)[0].item() - 3.0 * math.sqrt(200)) <= 1e-4
    moe.moe_adamw_step(plan, lr=0.25, step=1, betas=BETAS, weight_decay=0.0)
    assert torch.all(p[-200:] == -0.25) and not p[:-200].any()


def test_refusals(moe):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    s32, s8 = moe.moe_adamw_state([p], 32), moe.moe_adamw_state([p], 8)
    plan = moe.moe_adamw_plan([p], [g], **s32)
    with pytest.raises(ValueError):
        moe.moe_adamw_state([p], 16)
    with pytest.raises(ValueError):
        moe.moe_adamw_plan([p], [g, g], **s32)
    with pytest.raises(ValueError):
        moe.moe_adamw_plan([p], [g[:32]], **s32)
    with pytest.raises(ValueError):
        moe.moe_adamw_plan([p], [g], s8["m"], s8["v"])
    with pytest.raises(ValueError):
        moe.moe_adamw_plan([p.view(8, 8).t()], [g], **s32)
    with pytest.raises(ValueError):
        moe.moe_adamw_plan([p.cpu()], [g], **s32)
    with pytest.raises(TypeError):
        moe.moe_adamw_plan([p.double()], [g], **s32)
    with pytest.raises(TypeError):
        moe.moe_adamw_plan([p], [g], s32["m"], s8["v"])
    with pytest.raises(TypeError):
        moe.moe_adamw_plan([p], [g], masters=[p.half()], **s32)
    with pytest.raises(ValueError):
        moe.moe_adamw_step(moe.moe_tensor_list([g]), lr=1e-3, step=1)
    with pytest.raises(ValueError):
        moe.moe_adamw_step(plan)
    with pytest.raises(ValueError):
        moe.moe_adamw_step(plan, lr=1e-3, step=1, hyper=torch.zeros(8, device="cuda"))
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)),
                dict(eps=-1e-8), dict(weight_decay=float("inf"))):
        with pytest.raises(moe.MoEError) as e:
            moe.moe_adamw_step(plan, **{**dict(lr=1e-3, step=1), **bad})
        assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.moe_adamw_step(moe.moe_adamw_plan([p], [g], decay=[-1.0], **s32), lr=1e-3, step=1)
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.moe_grad_norm([g], max_norm=0.0)
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.moe_grad_norm([g], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
    with pytest.raises(TypeError):
        moe.moe_grad_norm([g.double()])
    assert not p.any()
