"""The layer for a few tokens and 4-bit products where values, codes, groups and sizes are at their ends."""
import math

import pytest
import torch

from tests import few_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_expert_gb300")

KINDS = ["bf16", "fp8", "int4"]


def bf16(*shape, value):
    return torch.full(shape, value, dtype=torch.bfloat16, device="cuda")


def test_h_up_to_the_largest_fp32_value_and_infinity():
    """h = x^2 (129 * 254 / 2^13) of rows whose x is one power of two: 2^127 * 1.99988, which a bf16 alone would round
    to infinity, is kept; beyond fp32 h is an infinity, and so is out, not NaN."""
    d = f = 64
    # 64 equal products: the sums are exact
    gate, up = bf16(1, d, f, value=2.0 ** -6 * 129 / 128), bf16(1, d, f, value=2.0 ** -5 * 254 / 128)
    down = bf16(1, f, d, value=2.0 ** -40)
    down[..., ::2] *= -1.0
    packed = moe.moe_pack_weights(gate, up, down)
    x = torch.tensor([64.0, 2.0 ** 63, 2.0 ** 65, -(2.0 ** 62)], device="cuda")[:, None].repeat(1, d).to(torch.bfloat16)
    out = moe.moe_forward_few(x, torch.zeros(4, 1, device="cuda"), packed, 1, 1, f)
    sign = torch.where(torch.arange(d, device="cuda") % 2 == 0, -1.0, 1.0).double()
    for row, v in ((0, 64.0), (1, 2.0 ** 63)):
        # h is good to U^2 and the gate's 2^-20, out to U
        want = v * v * (129 * 254 / 2 ** 13) * 2.0 ** -34 * sign
        assert float(((out[row].double() - want) / want).abs().max()) <= ref.U + ref.U ** 2 + 2.0 ** -20 + ref.gamma(64)
    assert torch.equal(out[2].double(), math.inf * sign)
    assert (out[3] == 0).all()  # silu of a large negative number


@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_scales_up_to_the_quantisers_largest(group):
    """Weights near bf16's largest value: their scales are near 2^125."""
    K, N = 256, 70
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = (torch.rand(K, N, generator=gen, device="cuda") * 2 - 1).mul_(2.0 ** 127 * 1.98).to(torch.bfloat16)
    w[0::group] = 2.0 ** 127 * 1.984375  # of every group: the scale is 2^127 * 1.984375 / 7
    codes, scales = moe.moe_quantize_int4(w, group)
    assert float(scales.float().max()) >= 2.0 ** 125
    x = (torch.randn(3, K, generator=gen, device="cuda") * 2.0 ** -20).to(torch.bfloat16)
    out = moe.moe_linear_int4(x, moe.moe_pack_linear_int4(codes, scales, K, N, group), N, group)
    dense = ref.dequantize_int4(codes, scales, group)
    want, size = x.double() @ dense, x.double().abs() @ (8.0 * scales.double().repeat_interleave(group, 0))
    ref.check(out, want, ref.U * want.abs() + 7.0 * ref.gamma(K) * size)


@pytest.mark.parametrize("packed_with,called_with", [(32, 64), (32, 128), (64, 128), (64, 32), (128, 64), (128, 32)])
def test_weights_of_another_group_are_refused(packed_with, called_with):
    """A buffer that was packed with other groups has another size."""
    K, N, E = 256, 96, 3
    codes, scales = moe.moe_quantize_int4(torch.randn(K, N, device="cuda").to(torch.bfloat16), packed_with)
    x = torch.randn(2, K, device="cuda").to(torch.bfloat16)
    matrix = moe.moe_pack_linear_int4(codes, scales, K, N, packed_with)
    moe.moe_linear_int4(x, matrix, N, packed_with)
    with pytest.raises(ValueError):
        moe.moe_linear_int4(x, matrix, N, called_with)
    experts, _ = ref.weights("int4", E, K, 128, packed_with)
    logits = torch.randn(2, E, device="cuda")
    moe.moe_forward_few(x, logits, experts, E, 2, 128, weights="int4", group=packed_with)
    router = moe.moe_pack_router_weights(torch.randn(K, E, device="cuda").to(torch.bfloat16))
    for call, route in ((moe.moe_forward_few, logits), (moe.moe_forward_few_routed, router)):
        with pytest.raises(ValueError):
            call(x, route, experts, E, 2, 128, weights="int4", group=called_with)


def test_gates_that_change_from_call_to_call():
    """Calls one after the other on one workspace, whose gates and choices differ: each uses its own."""
    E, d, f, T, k = 6, 128, 128, 9, 3
    packed, _ = ref.weights("bf16", E, d, f)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    routes = [torch.randn(T, E, generator=gen, device="cuda") * s for s in (0.1, 3.0, 1.0, 10.0)]
    want = [moe.moe_forward_few(x, l, packed, E, k, f) for l in routes]
    torch.cuda.synchronize()
    ws = torch.empty(moe.moe_forward_few_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    got = [moe.moe_forward_few(x, routes[i % 4], packed, E, k, f, workspace=ws, topk_idx=idx, topk_w=w) for i in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))


@pytest.mark.parametrize("T", [5, 6, 7, 8])
def test_fp8_rings_of_three_slots(T):
    """5 to 8 tokens leave room for three stages of rows (and of weights), which two groups of warps take in turn: the
    same bits every time, whatever the caches hold, and the right ones."""
    E, d, f, k = 6, 2048, 1024, 3
    packed, mats = ref.weights("fp8", E, d, f)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    flush = torch.empty(64 << 20, device="cuda")
    first = moe.moe_forward_few(x, logits, packed, E, k, f, weights="fp8")
    ref.check(first, *ref.layer(x, *ref.route(logits, k), mats, "fp8"))
    for i in range(60):
        if i % 2:
            flush.fill_(float(i))
        assert torch.equal(moe.moe_forward_few(x, logits, packed, E, k, f, weights="fp8"), first)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k", [(64, 20, 9), (64, 64, 32), (17, 33, 31), (64, 1024, 32)])
def test_more_pairs_than_units_kept_in_shared_memory(kind, T, E, k):
    """T * k > 512; with 1,024 experts nearly every pair is a unit."""
    d = f = 128
    packed, mats = ref.weights(kind, E, d, f)
    gen = torch.Generator(device="cuda").manual_seed(T + k)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    out = moe.moe_forward_few(x, logits, packed, E, k, f, weights=kind)
    idx, w = ref.route(logits, k)
    ref.check(out, *ref.layer(x, idx, w, mats, kind))


@pytest.mark.parametrize("T", [2, 13])
def test_subnormal_fp8_codes(T):
    """Weights of subnormal E4M3 codes (0x01 to 0x07 and their negatives) alone, with scales that make them matter."""
    E, d, f, k = 4, 256, 128, 2
    gen = torch.Generator(device="cuda").manual_seed(11)
    coded, mats = [], []
    for K, N in ((d, f), (d, f), (f, d)):
        codes = torch.randint(1, 8, (E, K, N), generator=gen, device="cuda", dtype=torch.uint8)
        codes |= torch.randint(0, 2, (E, K, N), generator=gen, device="cuda", dtype=torch.uint8) << 7
        scales = torch.exp(0.2 * torch.randn(E * K * N // 128, generator=gen, device="cuda")) * (2.0 ** 7 / math.sqrt(K))
        coded.append((codes, scales))
        mats.append(ref.dequantize_fp8(codes, scales, (E, K, N)))
    packed = moe.moe_pack_weights_fp8(*coded, E, d, f)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    out = moe.moe_forward_few(x, logits, packed, E, k, f, weights="fp8")
    idx, w = ref.route(logits, k)
    want, bound = ref.layer(x, idx, w, mats, "fp8")
    ref.check(out, want, bound)
    assert float((want.abs() > 10 * bound).double().mean()) > 0.5  # a lost code would be seen


@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_experts_near_moe_forward(group):
    """4-bit experts beside the layer's other form on the same weights in bf16."""
    E, d, f, T, k = 16, 512, 256, 20, 4
    packed, mats = ref.weights("int4", E, d, f, group)
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    a = moe.moe_forward(x, logits, moe.moe_pack_weights(*[m.to(torch.bfloat16) for m in mats]), E, k, f)
    b = moe.moe_forward_few(x, logits, packed, E, k, f, weights="int4", group=group)
    rel = float((a.float() - b.float()).norm() / b.float().norm())
    # gate, up and down weights, h, y and out rounded on one side, out on the other: seven roundings, each U / sqrt(3)
    # in the mean over evenly spread values
    assert rel <= 1.25 * 7 ** 0.5 * ref.U / 3.0 ** 0.5


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,f", [(65536, 128), (128, 65536)])
def test_longest_rows(kind, d, f):
    E, T, k = 2, 18, 2
    packed, mats = ref.weights(kind, E, d, f, seed=6)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    out = moe.moe_forward_few(x, logits, packed, E, k, f, weights=kind)
    ref.check(out, *ref.layer(x, *ref.route(logits, k), mats, kind))


def test_routed_by_the_longest_rows():
    E, T, k, d, f = 6, 5, 2, 65536, 64
    packed, mats = ref.weights("bf16", E, d, f, seed=7)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    w_router = (torch.randn(d, E, generator=gen, device="cuda") / d ** 0.5).to(torch.bfloat16)
    logits = x.double() @ w_router.double()
    # 64 additions inside a K block, d / 1024 blocks a warp, 16 warps; any of them may cut off
    d_logit = float(((80 + d / 1024) * 2.0 ** -23 * (x.double().abs() @ w_router.double().abs())).max())
    top = torch.sort(logits, dim=1, descending=True)[0]
    assert (top[:, :k] - top[:, 1:k + 1]).min() > 2 * d_logit, "these inputs do not tell which experts are right"
    out = moe.moe_forward_few_routed(x, moe.moe_pack_router_weights(w_router), packed, E, k, f)
    ref.check(out, *ref.layer(x, *ref.route(logits, k), mats, "bf16", d_logit))


@pytest.mark.parametrize("kind,E", [("bf16", 300), ("fp8", 600), ("int4", 1000)])
def test_experts_beyond_32_bits(kind, E):
    """The last experts of a layer whose gate and up weights alone take more than 2^32 bytes."""
    d = f = 2048
    chosen, T, k = [E - 1, E // 2, 1], 4, 2
    gen = torch.Generator(device="cuda").manual_seed(E)
    mats = [(torch.randn(3, d, f, generator=gen, device="cuda") / d ** 0.5).to(torch.bfloat16) for _ in range(3)]

    def spread(values, at):  # the chosen experts' values among others that are never read
        full = torch.zeros(E, *values.shape[1:], dtype=values.dtype, device="cuda")
        full[chosen] = values
        return full.reshape(-1) if at else full
    if kind == "bf16":
        packed = moe.moe_pack_weights(*[spread(m, 0) for m in mats])
        mats = [m.double() for m in mats]
    elif kind == "fp8":
        coded = [moe.moe_quantize_fp8_blockwise(m) for m in mats]
        mats = [ref.dequantize_fp8(c, s, (3, d, f)) for c, s in coded]
        packed = moe.moe_pack_weights_fp8(*[(spread(c.view(torch.uint8).reshape(3, d, f), 0), spread(s.reshape(3, -1), 1))
                                            for c, s in coded], E, d, f)
    else:
        coded = [moe.moe_quantize_int4(m) for m in mats]
        mats = [ref.dequantize_int4(c, s, 128) for c, s in coded]
        packed = moe.moe_pack_weights_int4(*[(spread(c, 0), spread(s, 0)) for c, s in coded], E, d, f)
    assert packed.numel() * packed.element_size() > 1.5 * 2 ** 32
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    few_logits = torch.randn(T, 3, generator=gen, device="cuda")
    logits = torch.full((T, E), -40.0, device="cuda")
    logits[:, chosen] = few_logits
    out = moe.moe_forward_few(x, logits, packed, E, k, f, weights=kind)
    ref.check(out, *ref.layer(x, *ref.route(few_logits, k), mats, kind))


def test_matrix_beyond_32_bits():
    """The last columns of a 4-bit matrix of more than 2^32 bytes."""
    K, N, M, last = 65536, 140_003, 3, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (K // 2, N), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand(K // 128, N, generator=gen, device="cuda").to(torch.bfloat16)
    packed = moe.moe_pack_linear_int4(codes, scales, K, N)
    assert packed.numel() > 2 ** 32
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    out = moe.moe_linear_int4(x, packed, N)
    for part in (slice(0, last), slice(N // 2, N // 2 + last), slice(N - last, N)):
        w = ref.dequantize_int4(codes[:, part].contiguous(), scales[:, part], 128)
        want = x.double() @ w
        size = x.double().abs() @ (8.0 * scales[:, part].double().repeat_interleave(128, 0))
        ref.check(out[:, part], want, ref.U * want.abs() + 7.0 * ref.gamma(K) * size)


def test_fp8_range_of_scaled_inputs():
    """x * scale and h * scale up to 2^67 in size are right; beyond, the token's output is not finite, and the others'
    are untouched."""
    d = f = 128
    one = torch.zeros(1, d, f, dtype=torch.uint8, device="cuda")
    one[:, 0] = 0x38  # 1.0 in E4M3, for the first input alone
    coded = [(codes, torch.full((d,), scale, device="cuda")) for codes, scale in
             ((one, 1.0), (one, 2.0 ** -70), (torch.full_like(one, 0x38), 2.0 ** -60))]
    packed = moe.moe_pack_weights_fp8(*coded, 1, d, f)
    x = torch.zeros(5, d, device="cuda")
    x[:, 0] = torch.tensor([2.0 ** 40, 1.5 * 2.0 ** 66, 2.0 ** 69, 2.0 ** 66, 2.0 ** 50])
    out = moe.moe_forward_few(x.to(torch.bfloat16), torch.zeros(5, 1, device="cuda"), packed, 1, 1, f, weights="fp8")
    # silu(g) = g; every value is a power of two or 1.5 times one
    want = (x[:, :1].double() ** 2 * 2.0 ** -70 * 2.0 ** -60 * f).expand(-1, d)
    keep = [0, 1, 3, 4]
    assert float(((out[keep].double() - want[keep]) / want[keep]).abs().max()) <= ref.U
    assert not torch.isfinite(out[2]).any()


def test_infinite_inputs_of_4_bit_experts():
    """An infinite input makes its own token's output NaN, no other's."""
    E, d, f, T = 3, 128, 128, 12
    packed, mats = ref.weights("int4", E, d, f)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    x[5, 77] = math.inf
    logits = torch.randn(T, E, generator=gen, device="cuda")
    out = moe.moe_forward_few(x, logits, packed, E, 2, f, weights="int4")
    keep = [t for t in range(T) if t != 5]
    ref.check(out[keep], *ref.layer(x[keep], *ref.route(logits[keep], 2), mats, "int4"))
    assert torch.isnan(out[5]).all()


def test_weights_of_another_format_are_refused():
    """bf16 weights take more bytes than the same in FP8 or 4 bits: too many are refused as too few are."""
    E, d, f = 3, 128, 256
    x, logits = bf16(2, d, value=1.0), torch.randn(2, E, device="cuda")
    packed = {kind: ref.weights(kind, E, d, f)[0] for kind in KINDS}
    for kind in KINDS:
        for other in KINDS:
            if kind == other:
                moe.moe_forward_few(x, logits, packed[kind], E, 2, f, weights=kind)
            else:
                with pytest.raises(ValueError):
                    moe.moe_forward_few(x, logits, packed[other], E, 2, f, weights=kind)
