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
