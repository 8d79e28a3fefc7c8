"""A serving step as a user runs it: norm, the layer for a few tokens from its router's weights, an output head in
4 bits; eagerly and as one captured graph, for every format of expert weights."""
import pytest
import torch

from tests import few_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_expert_gb300")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("T", [1, 11])
def test_decode_step(kind, T):
    d, E, k, f, vocab = 256, 16, 4, 384, 1003
    packed, mats = ref.weights(kind, E, d, f, 64)
    gen = torch.Generator(device="cuda").manual_seed(9)
    router_w = (torch.randn(d, E, generator=gen, device="cuda") / 16).to(torch.bfloat16)
    head_w = (torch.randn(d, vocab, generator=gen, device="cuda") / 16).to(torch.bfloat16)
    router = moe.moe_pack_router_weights(router_w)
    codes, scales = moe.moe_quantize_int4(head_w, 32)
    head = moe.moe_pack_linear_int4(codes, scales, d, vocab, 32)
    ws = torch.empty(moe.moe_forward_few_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device="cuda")
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    norm = torch.ones(d, device="cuda")

    def step():
        n, _ = moe.moe_layer_norm(x, norm)
        y = moe.moe_forward_few_routed(n, router, packed, E, k, f, weights=kind, group=64, workspace=ws)
        return n, y, moe.moe_linear_int4(y, head, vocab, 32)

    def check(n, y, logits):
        # each operator on what the one before it gave
        scores = n.double() @ router_w.double()
        idx, w = ref.route(scores, k)
        d_logit = float((80 * 2.0 ** -23 * (n.double().abs() @ router_w.double().abs())).max())
        ref.check(y, *ref.layer(n, idx, w, mats, kind, d_logit))
        want = y.double() @ ref.dequantize_int4(codes, scales, 32)
        size = y.double().abs() @ (8.0 * scales.double().abs().repeat_interleave(32, 0))
        ref.check(logits, want, ref.U * want.abs() + 7.0 * ref.gamma(d) * size + 2.0 ** -120)

    first = step()
    check(*first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))
    x.copy_(torch.randn(T, d, generator=gen, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    check(*held)
    assert moe.moe_read_device_status(ws) == 0
