"""4-bit weights: the quantiser's codes and scales, and products of a few rows against their 64-bit form."""
import pytest
import torch

from tests import few_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("sparse_expert_gb300")


def matrix(K, N, group, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (K // 2, N), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.exp(torch.randn(-(-K // group), N, generator=gen, device="cuda") - 3.0).to(torch.bfloat16)
    scales[:, ::7] *= -1  # a scale may have either sign
    return codes, scales


def check_linear(x, codes, scales, group, out):
    w = ref.dequantize_int4(codes, scales, group)
    want = x.double() @ w
    K = w.shape[0]
    # a code may be multiplied as 16 + code (below 32) with 24 times the inputs' sum taken off again: 56 scales a product
    bound = ref.U * want.abs() + ref.gamma(K) * 7.0 * (x.double().abs() @ (8.0 * scales.double().abs().repeat_interleave(
        group, 0)[:K])) + 2.0 ** -120
    # (the whole is then within U too; less, U / sqrt(3), is what roundings come to on average, and a few values that
    # make up most of the norm need not keep to the average)
    ref.check(out, want, bound)


@pytest.mark.parametrize("M", list(range(1, 17)))
def test_rows(M):
    codes, scales = matrix(512, 200, 64)
    x = torch.randn(M, 512, device="cuda").to(torch.bfloat16)
    out = moe.moe_linear_int4(x, moe.moe_pack_linear_int4(codes, scales, 512, 200, 64), 200, 64)
    check_linear(x, codes, scales, 64, out)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [8, 24, 32, 40, 64, 96, 120, 128, 136, 200, 1000, 4104])
def test_lengths(K, group):
    codes, scales = matrix(K, 67, group)
    x = torch.randn(3, K, device="cuda").to(torch.bfloat16)
    out = moe.moe_linear_int4(x, moe.moe_pack_linear_int4(codes, scales, K, 67, group), 67, group)
    check_linear(x, codes, scales, group, out)


@pytest.mark.parametrize("N", [1, 2, 31, 63, 64, 65, 128, 1000, 4096, 20001])
@pytest.mark.parametrize("M", [1, 9])
def test_widths(N, M):
    codes, scales = matrix(256, N, 128)
    x = torch.randn(M, 256, device="cuda").to(torch.bfloat16)
    out = moe.moe_linear_int4(x, moe.moe_pack_linear_int4(codes, scales, 256, N, 128), N)
    check_linear(x, codes, scales, 128, out)


@pytest.mark.parametrize("K,N", [(65536, 70), (16384, 500), (2048, 30000)])
def test_large(K, N):
    codes, scales = matrix(K, N, 128)
    x = torch.randn(16, K, device="cuda").to(torch.bfloat16)
    out = moe.moe_linear_int4(x, moe.moe_pack_linear_int4(codes, scales, K, N, 128), N)
    check_linear(x, codes, scales, 128, out)


def test_strided_rows_and_what_lies_between_them():
    codes, scales = matrix(264, 70, 64)
    packed = moe.moe_pack_linear_int4(codes, scales, 264, 70, 64)
    wide = torch.full((5, 320), float("nan"), device="cuda", dtype=torch.bfloat16)
    x = wide[:, 8:272]
    x.copy_(torch.randn(5, 264, device="cuda"))
    into = torch.full((7, 99), 5.0, device="cuda", dtype=torch.bfloat16)
    out = into[1:6, 3:73]
    assert moe.moe_linear_int4(x, packed, 70, 64, out=out) is out
    check_linear(x, codes, scales, 64, out)
    rest = into.clone()
    rest[1:6, 3:73] = 5.0
    assert (rest == 5.0).all()


def test_nan_and_infinity_stay_in_their_row():
    codes, scales = matrix(256, 64, 32)
    packed = moe.moe_pack_linear_int4(codes, scales, 256, 64, 32)
    x = torch.randn(12, 256, device="cuda").to(torch.bfloat16)
    x[4, 100] = float("nan")
    x[9, 3] = float("inf")
    out = moe.moe_linear_int4(x, packed, 64, 32)
    assert torch.isnan(out[4]).all() and not torch.isfinite(out[9]).any()
    keep = [i for i in range(12) if i not in (4, 9)]
    check_linear(x[keep], codes, scales, 32, out[keep])


def test_rows_of_an_offset():
    """Values with a large common part, where a sum of codes has most to cancel."""
    codes, scales = matrix(4096, 100, 128)
    x = (100.0 + torch.randn(4, 4096, device="cuda")).to(torch.bfloat16)
    out = moe.moe_linear_int4(x, moe.moe_pack_linear_int4(codes, scales, 4096, 100, 128), 100)
    check_linear(x, codes, scales, 128, out)


def test_no_rows_other_streams_and_graphs():
    codes, scales = matrix(512, 300, 128)
    packed = moe.moe_pack_linear_int4(codes, scales, 512, 300)
    x = torch.randn(6, 512, device="cuda").to(torch.bfloat16)
    assert moe.moe_linear_int4(x[:0], packed, 300).shape == (0, 300)
    want = moe.moe_linear_int4(x, packed, 300)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [moe.moe_linear_int4(x, packed, 300, stream=s) for s in (side, None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_linear_int4(x, packed, 300, out=out)
    x.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -2.0 * want)


@pytest.mark.parametrize("shape,group", [((256, 100), 128), ((3, 64, 65), 32), ((200, 7), 64), ((2, 2, 128, 16), 128),
                                         ((8, 1), 128)])
def test_quantiser(shape, group):
    w = torch.randn(*shape, device="cuda").to(torch.bfloat16)
    w.view(-1)[:3] *= 30
    w[..., :4, 0] = 0
    if shape[-2] == 200:
        w[..., 64:128, :] = 0  # a group of zeros
    codes, scales = moe.moe_quantize_int4(w, group)
    K = shape[-2]
    groups = -(-K // group)
    pad = torch.nn.functional.pad(w.float(), (0, 0, 0, groups * group - K))
    blocks = pad.unflatten(-2, (groups, group))
    amax = blocks.abs().amax(-2)
    s = (amax / 7.0).to(torch.bfloat16)
    s = torch.where(s > 0, s, torch.ones_like(s))
    assert torch.equal(scales, s)
    q = torch.clamp(torch.round(blocks / s.float()[..., None, :]) + 8, 0, 15).flatten(-3, -2)[..., :K, :]
    got = torch.stack([codes & 15, codes >> 4], -2).flatten(-3, -2)
    assert torch.equal(got.float(), q)
    # codes -7 .. 7 of scales that are at most 2^-8 too small: within half a scale
    err = (ref.dequantize_int4(codes, scales, group) - w.double()).abs()
    assert (err <= 0.51 * s.double().repeat_interleave(group, -2)[..., :K, :]).all()


def test_argument_checks():
    codes, scales = matrix(128, 32, 64)
    packed = moe.moe_pack_linear_int4(codes, scales, 128, 32, 64)
    x = torch.zeros(2, 128, device="cuda", dtype=torch.bfloat16)
    wide = torch.zeros(2, 132, device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: moe.moe_linear_int4(x.float(), packed, 32, 64), lambda: moe.moe_linear_int4(x, packed, 33 + 64, 64),
                lambda: moe.moe_linear_int4(x, packed, 32, 48), lambda: moe.moe_linear_int4(x[0], packed, 32, 64),
                lambda: moe.moe_linear_int4(wide[:, :128], packed, 32, 64), lambda: moe.moe_linear_int4(wide[:, 1:129], packed, 32, 64),
                lambda: moe.moe_linear_int4(x.repeat(9, 1), packed, 32, 64), lambda: moe.moe_linear_int4(x.cpu(), packed, 32, 64),
                lambda: moe.moe_linear_int4(x, packed.cpu(), 32, 64), lambda: moe.moe_linear_int4(x, packed[:-4], 32, 64),
                lambda: moe.moe_linear_int4(x, packed, 32, 64, out=torch.zeros(2, 32, device="cuda")),
                lambda: moe.moe_pack_linear_int4(codes, scales, 128, 33, 64), lambda: moe.moe_pack_linear_int4(codes, scales, 128, 32, 32),
                lambda: moe.moe_pack_linear_int4(codes.cpu(), scales, 128, 32, 64), lambda: moe.moe_quantize_int4(x, 100),
                lambda: moe.moe_quantize_int4(x[:, :12].contiguous(), 32), lambda: moe.moe_quantize_int4(x.float(), 32)):
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            bad()
