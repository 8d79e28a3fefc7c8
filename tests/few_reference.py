"""Plain 64-bit forms of the layer for a few tokens and of 4-bit weights, with bounds on what rounding may add.

A rounding to bf16 is off by at most U = 2^-8 of the value, two bf16 (a value and what its rounding left) by U^2.  The
kernels round out to bf16, keep h as two, and with FP8 weights the products x * scale and h * scale too.  Sums of K
products in fp32 are off by at most gamma(K) = K 2^-23 of the sum of the products' sizes (every addition cut off, in any
order).
"""
import math

import torch

U = 2.0 ** -8


def gamma(K):
    return K * 2.0 ** -23


def dequantize_int4(codes, scales, group):
    """fp64 weights [..., K, N] of codes [..., K/2, N] and scales [..., ceil(K/group), N]."""
    q = torch.stack([codes & 15, codes >> 4], dim=-2).flatten(-3, -2).double() - 8.0
    return q * scales.double().repeat_interleave(group, dim=-2)[..., : q.shape[-2], :]


def dequantize_fp8(codes, scales, shape):
    v = codes.view(torch.float8_e4m3fn).float().double().reshape(-1, 128) * scales.double()[:, None]
    return v.reshape(shape)


def weights(kind, E, d, f, group=128, seed=0, spread=1.0):
    """(packed by the library, [w_gate, w_up, w_down] in fp64, on the GPU)."""
    import sparse_expert_gb300 as moe

    gen = torch.Generator(device="cuda").manual_seed(seed)
    mats = [(torch.randn(E, K, N, generator=gen, device="cuda") * (spread / math.sqrt(K))).to(torch.bfloat16)
            for K, N in ((d, f), (d, f), (f, d))]
    if kind == "bf16":
        return moe.moe_pack_weights(*mats), [m.double() for m in mats]
    if kind == "fp8":
        coded = [moe.moe_quantize_fp8_blockwise(m) for m in mats]
        return moe.moe_pack_weights_fp8(*coded, E, d, f), [dequantize_fp8(*c, m.shape) for c, m in zip(coded, mats)]
    coded = [moe.moe_quantize_int4(m, group) for m in mats]
    return moe.moe_pack_weights_int4(*coded, E, d, f, group), [dequantize_int4(*c, group) for c in coded]


def route(logits, k, renormalize=True):
    """idx [T,k] (ties: the lowest index first) and gates in fp64."""
    l64 = logits.double()
    idx = torch.sort(l64, dim=1, descending=True, stable=True)[1][:, :k]
    p = torch.softmax(l64, 1).gather(1, idx)
    return idx, p / p.sum(1, keepdim=True) if renormalize else p


def layer(x, idx, w, mats, kind, d_logit=0.0):
    """(out, bound): fp64 result for the given selection, and how far each value may be off.
    d_logit: how far the logits may be off (gates then by 2 d_logit of themselves)."""
    wg, wu, wd = mats
    x = x.double()
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    d, f = wg.shape[1:]
    scaled = U * U if kind == "fp8" else 0.0
    for e in torch.unique(idx).tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        r = x[t]
        g, u = r @ wg[e], r @ wu[e]
        dg, du = ((scaled + gamma(d)) * (r.abs() @ m[e].abs()) for m in (wg, wu))
        h = g / (1.0 + torch.exp(-g)) * u
        # |silu'| <= 1.1; the exponential and the division are good to 2^-20
        dh = 1.1 * u.abs() * dg + g.abs() * du + 1.1 * dg * du + (U * U + 2.0 ** -20) * h.abs()
        y, size = h @ wd[e], h.abs() @ wd[e].abs()
        dy = dh @ wd[e].abs() * (1 + scaled) + (scaled + gamma(f)) * size
        gate = w[t, j, None]
        out.index_add_(0, t, gate * y)
        bound.index_add_(0, t, gate * (dy + (2.0 * d_logit + 2.0 ** -20) * size))
    return out, bound + U * (out.abs() + bound) + 2.0 ** -120


def check(got, want, bound):
    """Every value within its bound, which is little more than the rounding of out."""
    assert torch.isfinite(got).all()
    worst = float(((got.double() - want).abs() / bound).max())
    assert worst <= 1.0, f"{worst} times the bound"
