"""Waits that run out in the layer for a few tokens and in 4-bit products: the launch ends by itself, says so, and the
next call is right.  What never comes is a count that nothing reaches, or rows that nothing asks for; the limits of the
waits are short, and no fault is made."""
import time

import pytest
import torch

from tests import few_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_expert_gb300")

KINDS = ["bf16", "fp8", "int4"]  # one, two and one group of multiplying warps
TIMEOUT = 4
E, d, f, k = 8, 1024, 512, 3


class Layer:
    def __init__(self, kind, T):
        gen = torch.Generator(device="cuda").manual_seed(T)
        self.kind, self.T = kind, T
        self.packed, _ = ref.weights(kind, E, d, f)
        self.x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
        self.logits = torch.randn(T, E, generator=gen, device="cuda")
        self.ws = torch.empty(moe.moe_forward_few_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device="cuda")
        self.want = self.call()
        assert moe.moe_read_device_status(self.ws) == 0

    def call(self):
        return moe.moe_forward_few(self.x, self.logits, self.packed, E, k, f, weights=self.kind, workspace=self.ws)

    def spoiled(self, counter, limit_ns):
        out = moe.moe_selftest_few_wait(self.x, self.logits, self.packed, E, k, f, self.kind, self.ws, counter, limit_ns)
        return out, moe.moe_read_device_status(self.ws)

    def right_again(self):
        assert torch.equal(self.call(), self.want) and moe.moe_read_device_status(self.ws) == 0


@pytest.mark.parametrize("T", [1, 6, 13, 40])
@pytest.mark.parametrize("what", ["unit", "strip"])
@pytest.mark.parametrize("kind", KINDS)
def test_a_count_that_is_never_reached(kind, what, T):
    """A unit whose h is never complete, and a strip of outputs that some unit never finishes."""
    layer = Layer(kind, T)
    t0 = time.perf_counter()
    _, status = layer.spoiled(0 if what == "unit" else T * k + 3, 20_000_000)
    assert status == TIMEOUT
    assert time.perf_counter() - t0 < 1.5
    layer.right_again()


@pytest.mark.parametrize("T", [1, 6, 13, 40])
@pytest.mark.parametrize("kind", KINDS)
def test_limits_that_any_wait_may_meet(kind, T):
    """Blocks give up in different places, or not at all."""
    layer = Layer(kind, T)
    for limit_ns in (1, 500, 1_000, 2_000, 4_000, 8_000, 16_000, 32_000, 64_000):
        out, status = layer.spoiled(-1, limit_ns)
        assert status in (0, TIMEOUT)
        if status == 0:
            assert torch.equal(out, layer.want)
    layer.right_again()


def linear(M, K, N, group):
    gen = torch.Generator(device="cuda").manual_seed(N)
    codes = torch.randint(0, 256, (K // 2, N), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand(-(-K // group), N, generator=gen, device="cuda").to(torch.bfloat16)
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    packed = moe.moe_pack_linear_int4(codes, scales, K, N, group)
    return x, packed, moe.moe_linear_int4(x, packed, N, group)


@pytest.mark.parametrize("M", [1, 13])
@pytest.mark.parametrize("K,N,row_strips", [(1024, 40001, 0), (1024, 40001, 5), (1024, 40001, 400), (1000, 40001, 624),
                                            (4096, 500, 0), (4096, 500, 3), (2176, 2048, 31)])
def test_rows_that_are_never_asked_for(K, N, row_strips, M):
    """Strips walked by blocks that stay, and strips whose inputs are split over a cluster."""
    x, packed, want = linear(M, K, N, 64)
    t0 = time.perf_counter()
    out = moe.moe_selftest_linear_int4_wait(x, packed, N, row_strips, 20_000_000, group=64)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.5
    assert torch.equal(out[:, :64 * row_strips], want[:, :64 * row_strips])
    assert torch.isnan(out[:, 64 * row_strips:]).all()
    assert torch.equal(moe.moe_linear_int4(x, packed, N, 64), want)


@pytest.mark.parametrize("K,N", [(6144, 40001), (4096, 500)])
def test_limits_that_any_wait_of_a_product_may_meet(K, N):
    x, packed, want = linear(9, K, N, 32)
    for limit_ns in (1, 500, 1_000, 2_000, 4_000, 8_000, 16_000, 32_000):
        out = moe.moe_selftest_linear_int4_wait(x, packed, N, 1 << 20, limit_ns, group=32)
        lost = torch.isnan(out)
        assert torch.equal(out[~lost], want[~lost])
    assert torch.equal(moe.moe_linear_int4(x, packed, N, 32), want)
