"""The example's training step: its gradients against automatic
differentiation of the same block in 64 bits, and training runs.

The 64-bit block takes the layer's top-k choice from the run and holds it
fixed.  Tolerance: the layer's own (2e-2 of the largest value, 5e-3 of the
mean) with one more bf16 rounding for the norm's output and for the gradient
that enters the norm's backward.
"""
import os
import sys

import pytest
import torch

from tests.conftest import ROOT

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_block
    return train_block


def test_gradients_of_the_step(example):
    import sparse_expert_gb300 as moe

    cfg = workloads.get("tiny")
    block = example.Block(cfg, bits=32)
    h, r, target, mask = example.data(cfg)
    before = {k: p.double().requires_grad_() for k, p in block.params.items()}
    out = block.train_step(h, r, target, mask, balance=0.5, z=0.1)
    # the same block in 64 bits, from the run's bf16 residual stream
    stream = (h.float() + r.float()).to(torch.bfloat16).double()
    mu = stream.mean(1, keepdim=True)
    n = (stream - mu) / (stream.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt() * before["norm_w"] + before["norm_b"]
    logits = n @ before["router"]
    idx, _ = moe.moe_route_topk((n.float().to(torch.bfloat16).float() @ block_router(before)).contiguous(), cfg.k)
    gates = torch.softmax(logits.gather(1, idx.long()), 1)
    y = torch.zeros_like(stream)
    for j in range(cfg.k):
        e = idx[:, j].long()
        gate = torch.einsum("td,tdf->tf", n, before["w_gate"][e])
        up = torch.einsum("td,tdf->tf", n, before["w_up"][e])
        y = y + gates[:, j:j + 1] * torch.einsum("tf,tfd->td", torch.nn.functional.silu(gate) * up, before["w_down"][e])
    m = mask.double()[:, None]
    diff = (stream + y - target.double()) * m
    loss = diff.square().mean()
    counts = torch.bincount(idx.flatten().long(), minlength=cfg.E).double()
    p = torch.softmax(logits, 1)
    balance = cfg.E * ((p * m).sum(0) / m.sum() * counts / counts.sum()).sum()
    z = (torch.logsumexp(logits, 1).square() * m[:, 0]).sum() / m.sum()
    (loss + 0.5 * balance + 0.1 * z).backward()
    assert abs(out["loss"].item() - loss.item()) <= 1e-2 * loss.item()
    assert abs(out["balance"].item() - balance.item()) <= 1e-2 * balance.item()
    assert abs(out["z"].item() - z.item()) <= 1e-2 * z.item()
    for k, g in block.grads.items():
        want = before[k].grad
        err = (g.double() - want).abs()
        assert err.max() <= 3e-2 * want.abs().max() and err.mean() <= 1.5e-2 * want.abs().mean(), (
            k, (err.max() / want.abs().max()).item(), (err.mean() / want.abs().mean()).item())
    norm = sum(g.double().square().sum() for g in block.grads.values()).sqrt()
    assert abs(out["grad_norm"].item() - norm.item()) <= 1e-4 * norm.item()


def block_router(params):
    return params["router"].detach().float()


@pytest.mark.parametrize("bits", [8, 32])
def test_training_lowers_the_loss(example, bits):
    cfg = workloads.get("tiny")
    block = example.Block(cfg, bits=bits)
    args = example.data(cfg)
    first = block.train_step(*args)["loss"].item()
    for _ in range(60):
        last = block.train_step(*args)
    assert last["loss"].item() < 0.9 * first and torch.isfinite(last["grad_norm"])
    for k in ("w_gate", "router"):
        assert torch.isfinite(block.params[k].float()).all()


def test_8_bit_states_follow_32_bit_ones(example):
    cfg = workloads.get("tiny")
    a, b = example.Block(cfg, bits=8), example.Block(cfg, bits=32)
    args = example.data(cfg)
    la, lb = [], []
    for _ in range(30):
        la.append(a.train_step(*args)["loss"].item())
        lb.append(b.train_step(*args)["loss"].item())
    assert all(abs(x - y) <= 0.02 * y for x, y in zip(la, lb)), list(zip(la, lb))
