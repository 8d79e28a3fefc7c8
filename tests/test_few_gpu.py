"""The whole layer for a few tokens against its 64-bit form: every weight format, every count of tokens that a unit of
16 can end at, routings that leave experts empty or give them everything, workspaces, streams and graphs."""
import pytest
import torch

from tests import few_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_expert_gb300")

KINDS = ["bf16", "fp8", "int4"]


def inputs(T, d, E, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    x = (torch.randn(T, d, generator=gen, device="cuda") * torch.exp(0.3 * torch.randn(d, generator=gen, device="cuda")))
    return x.to(torch.bfloat16), torch.randn(T, E, generator=gen, device="cuda")


def run(kind, T, d, E, k, f, group=128, renormalize=True, logits=None, seed=0, **kw):
    packed, mats = ref.weights(kind, E, d, f, group, seed)
    x, l = inputs(T, d, E, seed)
    l = l if logits is None else logits
    idx_out = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w_out = torch.full((T, k), -7.0, device="cuda")
    out = moe.moe_forward_few(x, l, packed, E, k, f, weights=kind, group=group, renormalize=renormalize, topk_idx=idx_out,
                              topk_w=w_out, **kw)
    idx, w = ref.route(l, k, renormalize)
    assert torch.equal(idx_out.long(), idx)
    assert float((w_out - w).abs().max()) <= 2.0 ** -20
    want, bound = ref.layer(x, idx, w, mats, kind)
    ref.check(out, want, bound)
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64])
def test_tokens(kind, T):
    run(kind, T, 256, 12, 3, 384, seed=T)


@pytest.mark.parametrize("d,f", [(64, 64), (64, 192), (192, 64), (320, 576), (1088, 832), (2048, 1024)])
def test_bf16_sizes(d, f):
    run("bf16", 5, d, 6, 2, f)


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("d,f", [(128, 128), (128, 640), (896, 128), (1152, 768), (2048, 1024)])
def test_coded_sizes(kind, d, f):
    run(kind, 5, d, 6, 2, f)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 12])
def test_int4_groups(group, T):
    run("int4", T, 384, 5, 2, 256, group=group)


@pytest.mark.parametrize("kind", KINDS)
def test_long_rows(kind):
    run(kind, 3, 8192, 3, 2, 128)
    run(kind, 3, 128, 3, 2, 8192)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 16, 17, 40, 64])
def test_one_expert_has_every_token(kind, T):
    """A dense layer: units of 16 tokens, the last one short."""
    run(kind, T, 256, 1, 1, 256)


@pytest.mark.parametrize("kind", KINDS)
def test_all_tokens_choose_alike(kind):
    logits = torch.arange(40, 0, -1, device="cuda").float().repeat(50, 1) * 0.1
    run(kind, 50, 128, 40, 4, 128, logits=logits)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (32, 32), (33, 32), (100, 7), (512, 8), (700, 9), (1024, 32)])
def test_experts(E, k):
    run("bf16", 6, 64, E, k, 64)


def test_ties_and_gates_without_renormalisation():
    logits = torch.zeros(11, 70, device="cuda")
    logits[3] = -0.0
    logits[5, 60:] = 1.0
    run("bf16", 11, 64, 70, 6, 128, renormalize=False, logits=logits)


def test_experts_taken_out_by_minus_infinity():
    _, logits = inputs(9, 64, 20, 3)
    logits[:, ::2] = -float("inf")
    logits[4, 5:] = -float("inf")  # two left, and two are chosen
    run("bf16", 9, 64, 20, 2, 64, logits=logits)


def test_infinite_weights_of_experts_not_chosen():
    """Nothing of an expert that no token chose, or of a token that another expert has, gets into a result."""
    E, d, f, T = 5, 128, 128, 10
    packed, mats = ref.weights("bf16", E, d, f)
    per_gu, per_dn = 2 * d * f, d * f
    flat = packed.view(torch.bfloat16)
    flat[3 * per_gu:4 * per_gu] = float("nan")
    flat[E * per_gu + 3 * per_dn:E * per_gu + 4 * per_dn] = float("inf")
    x, logits = inputs(T, d, E)
    logits[:, 3] = -50.0
    x[6] = float("nan")  # token 6's own output alone is lost
    out = moe.moe_forward_few(x, logits, packed, E, 2, f)
    keep = [t for t in range(T) if t != 6]
    idx, w = ref.route(logits[keep], 2)
    want, bound = ref.layer(x[keep], idx, w, mats, "bf16")
    ref.check(out[keep], want, bound)
    assert torch.isnan(out[6]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,d,E,k,f", [(1, 128, 8, 2, 128), (19, 256, 40, 5, 384), (64, 128, 130, 8, 128),
                                       (7, 1024, 384, 8, 128), (40, 128, 512, 3, 128)])
def test_routed(kind, T, d, E, k, f):
    packed, mats = ref.weights(kind, E, d, f)
    x, _ = inputs(T, d, E, 5)
    gen = torch.Generator(device="cuda").manual_seed(77)
    w_router = (torch.randn(d, E, generator=gen, device="cuda") / d ** 0.5).to(torch.bfloat16)
    router = moe.moe_pack_router_weights(w_router)
    logits = x.double() @ w_router.double()
    # 64 products by the tensor cores, K blocks and warps in fp32 registers
    d_logit = float((80 * 2.0 ** -23 * (x.double().abs() @ w_router.double().abs())).max())
    top = torch.sort(logits, dim=1, descending=True)[0]
    gap = (top[:, :k] - top[:, 1:k + 1]).min() if k < E else 1.0
    assert gap > 2 * 2.0 ** -20, "these inputs do not tell which experts are right"
    idx_out = torch.empty(T, k, dtype=torch.int32, device="cuda")
    out = moe.moe_forward_few_routed(x, router, packed, E, k, f, weights=kind, topk_idx=idx_out)
    idx, w = ref.route(logits, k)
    assert torch.equal(idx_out.long(), idx)
    want, bound = ref.layer(x, idx, w, mats, kind, d_logit)
    ref.check(out, want, bound)


def test_same_bits_every_time_whatever_the_workspace_held():
    E, d, f, T, k = 24, 512, 256, 30, 4
    packed, _ = ref.weights("bf16", E, d, f)
    x, logits = inputs(T, d, E)
    size = moe.moe_forward_few_workspace_bytes(T, E, k, d, f)
    first = moe.moe_forward_few(x, logits, packed, E, k, f)
    for fill in (0, 255, 127):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        guard = torch.full((T + 2, d), 3.0, dtype=torch.bfloat16, device="cuda")
        out = guard[1:T + 1]
        moe.moe_forward_few(x, logits, packed, E, k, f, workspace=ws, out=out)
        assert torch.equal(out, first)
        assert (guard[0] == 3.0).all() and (guard[-1] == 3.0).all()
        assert moe.moe_read_device_status(ws) == 0


def test_calls_of_other_sizes_on_one_workspace():
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for i, (T, d, E, k, f) in enumerate([(64, 256, 12, 4, 256), (1, 64, 3, 1, 64), (33, 128, 200, 6, 192), (2, 512, 2, 2, 64)]):
        run("bf16", T, d, E, k, f, seed=i, workspace=ws)


def test_no_tokens():
    packed, _ = ref.weights("bf16", 3, 64, 64)
    x, logits = inputs(0, 64, 3)
    ws = torch.full((4096,), 255, dtype=torch.uint8, device="cuda")
    assert moe.moe_forward_few(x, logits, packed, 3, 2, 64, workspace=ws).shape == (0, 64)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_near_moe_forward(kind):
    """The layer's other form, on the same packed weights, differs by roundings alone."""
    E, d, f, T, k = 16, 512, 256, 20, 4
    packed, _ = ref.weights("bf16" if kind == "int4" else kind, E, d, f)
    x, logits = inputs(T, d, E)
    if kind == "fp8":
        a, b = moe.moe_forward_fp8(x, logits, packed, E, k, f), moe.moe_forward_few(x, logits, packed, E, k, f, "fp8")
    else:
        a, b = moe.moe_forward(x, logits, packed, E, k, f), moe.moe_forward_few(x, logits, packed, E, k, f)
    rel = float((a.float() - b.float()).norm() / b.float().norm())
    # weights, x * scale, h, h * scale, y and out each rounded on one side or both
    assert rel <= 1.25 * (8 ** 0.5) * ref.U / 3.0 ** 0.5


def test_streams_side_by_side():
    """Calls on two streams at once, each with its own workspace."""
    E, d, f, k = 32, 1024, 512, 4
    packed, _ = ref.weights("bf16", E, d, f)
    sets = [inputs(T, d, E, T) for T in (3, 40)]
    want = [moe.moe_forward_few(x, l, packed, E, k, f) for x, l in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (s, (x, l)) in enumerate(zip(streams, sets)):
            got[i].append(moe.moe_forward_few(x, l, packed, E, k, f, stream=s))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(o, w) for o in g)


@pytest.mark.parametrize("kind", KINDS)
def test_captured_graphs_that_share_a_workspace(kind):
    """Two graphs replayed in turn, with inputs that change between replays."""
    E, d, f, k = 20, 256, 128, 3
    packed, mats = ref.weights(kind, E, d, f)
    router_w = (torch.randn(d, E, device="cuda") / 16).to(torch.bfloat16)
    router = moe.moe_pack_router_weights(router_w)
    ws = torch.empty(moe.moe_forward_few_workspace_bytes(30, E, k, d, f), dtype=torch.uint8, device="cuda")
    (x1, l1), (x2, _) = inputs(30, d, E), inputs(5, d, E)
    o1, o2 = torch.empty_like(x1), torch.empty_like(x2)

    def one():
        moe.moe_forward_few(x1, l1, packed, E, k, f, kind, workspace=ws, out=o1)

    def two():
        moe.moe_forward_few_routed(x2, router, packed, E, k, f, kind, workspace=ws, out=o2)
    one(), two()
    torch.cuda.synchronize()
    graphs = []
    for call in (one, two):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for seed in range(3):
        nx, nl = inputs(30, d, E, 10 + seed)
        x1.copy_(nx), l1.copy_(nl), x2.copy_(inputs(5, d, E, 20 + seed)[0])
        o1.fill_(float("nan")), o2.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        idx, w = ref.route(l1, k)
        ref.check(o1, *ref.layer(x1, idx, w, mats, kind))
        logits = x2.double() @ router_w.double()
        idx, w = ref.route(logits, k)
        ref.check(o2, *ref.layer(x2, idx, w, mats, kind, 1e-4))


def test_argument_checks():
    packed, _ = ref.weights("bf16", 4, 64, 64)
    x, logits = inputs(3, 64, 4)
    call = moe.moe_forward_few
    for bad in (dict(weights="int8"), dict(k=5), dict(f=96), dict(E=3), dict(f=128), dict(out=torch.empty(3, 64, device="cuda")),
                dict(out=torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")), dict(weights="int4"), dict(weights="fp8"),
                dict(topk_idx=torch.empty(3, 2, dtype=torch.int64, device="cuda")), dict(x=x.cpu()), dict(x=x.float()),
                dict(x=x.t()), dict(logits=logits.double()), dict(logits=logits[:, :3]), dict(packed=packed[:-1]),
                dict(packed=packed.view(torch.bfloat16)), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        kw = dict(x=x, logits=logits, packed=packed, E=4, k=2, f=64)
        kw.update(bad)
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            call(**kw)
    with pytest.raises(moe.MoEError):
        xl, ll = inputs(65, 64, 4)
        call(xl, ll, packed, 4, 2, 64)
    with pytest.raises(ValueError):
        moe.moe_forward_few_routed(x, torch.empty(10, dtype=torch.uint8, device="cuda"), packed, 4, 2, 64)
