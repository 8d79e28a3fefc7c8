"""Training steps of one pre-norm Mixture-of-Experts block on one GPU.

    h' = h + r                       residual stream, with the layer norm of h'
    n  = layer_norm(h')
    out = h' + moe(n)                router, dispatch, experts, combine

The loss is the mean squared difference from a target, plus the router's load
balancing and z losses.  Everything but the router's two matrix products and
the residual additions at the end runs in the library's kernels: the norm,
the layer, the router losses, the layer's and the norm's backward, the
gradient norm and AdamW with fp32 masters and 8-bit states.

    python examples/train_block.py [--workload tiny|small] [--steps N] [--bits 8|32]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_expert_gb300 as moe  # noqa: E402
import workloads  # noqa: E402


class Block:
    """Parameters, buffers and the optimizer's plan of one block."""

    def __init__(self, cfg, bits=8, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, fan_in):
            return (torch.randn(*shape, generator=gen, device="cuda") / math.sqrt(fan_in)).to(torch.bfloat16)
        d, f, E = cfg.d, cfg.f, cfg.E
        self.cfg = cfg
        self.params = dict(w_gate=normal(E, d, f, fan_in=d), w_up=normal(E, d, f, fan_in=d),
                           w_down=normal(E, f, d, fan_in=f), router=normal(d, E, fan_in=d),
                           norm_w=torch.ones(d, device="cuda"), norm_b=torch.zeros(d, device="cuda"))
        self.grads = {k: torch.zeros_like(p) for k, p in self.params.items()}
        matrices = ("w_gate", "w_up", "w_down", "router")
        names = list(self.params)
        params = [self.params[k] for k in names]
        # 8-bit states for the matrices, fp32 states and no decay for the norm's vectors
        states = [moe.moe_adamw_state([p], bits if k in matrices else 32) for k, p in zip(names, params)]
        self.plan = moe.moe_adamw_plan(
            params, [self.grads[k] for k in names], [s["m"][0] for s in states], [s["v"][0] for s in states],
            m_scales=[s["m_scales"][0] for s in states], v_scales=[s["v_scales"][0] for s in states],
            masters=[p.float() if k in matrices else None for k, p in zip(names, params)],
            decay=[1.0 if k in matrices else 0.0 for k in names])
        self.step = 0

    def train_step(self, h, r, target, mask=None, lr=1e-3, balance=1e-2, z=1e-3, max_norm=1.0):
        """One step; returns dict(loss, balance, z, grad_norm) as device scalars."""
        cfg, p, g = self.cfg, self.params, self.grads
        T, E, k, d, f = h.shape[0], cfg.E, cfg.k, cfg.d, cfg.f
        # forward
        n, stats, stream = moe.moe_layer_norm(h, p["norm_w"], p["norm_b"], residual=r)
        logits = n.float() @ p["router"].float()
        packed = moe.moe_pack_weights(p["w_gate"], p["w_up"], p["w_down"])
        ws = torch.empty(moe.moe_forward_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device="cuda")
        y = moe.moe_forward(n, logits, packed, E, k, f, cfg.renormalize, workspace=ws)
        # of every routed row: padded tokens take their place at the experts too, so the balance loss counts them in
        # the load (not in the probabilities that it weighs by it)
        counts = moe.forward_intermediates(ws, T, E, k, d, f)["counts"]
        diff = stream.float() + y.float() - target.float()
        if mask is not None:
            diff = diff * mask[:, None]
        loss = diff.square().mean()
        dout = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        # backward: the layer, its router's losses, the router's products, the norm
        lg = moe.moe_backward(n, logits, packed, dout, E, k, f, cfg.renormalize,
                              grads=dict(dx=torch.empty_like(n), d_logits=torch.empty_like(logits),
                                         dw_gate=g["w_gate"], dw_up=g["w_up"], dw_down=g["w_down"]))
        losses, d_logits = moe.moe_router_loss(logits, counts, balance, z, mask=mask, accumulate=lg["d_logits"])
        g["router"].copy_(n.float().t() @ d_logits)
        dn = (lg["dx"].float() + d_logits @ p["router"].float().t()).to(torch.bfloat16)
        moe.moe_layer_norm_backward(dn, stream, stats, p["norm_w"], dz=dout,
                                    grads=dict(dx=torch.empty_like(dn), dweight=g["norm_w"], dbias=g["norm_b"]))
        # step
        self.step += 1
        clip = moe.moe_grad_norm(self.plan, max_norm)
        moe.moe_adamw_step(self.plan, lr=lr, step=self.step, clip=clip)
        return dict(loss=loss, balance=losses[0], z=losses[1], grad_norm=clip[0])


def data(cfg, seed=1):
    """Hidden states, the previous sublayer's output, a target and a mask with a padded tail."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h, r, t = (torch.randn(cfg.T, cfg.d, generator=gen, device="cuda") for _ in range(3))
    mask = torch.ones(cfg.T, dtype=torch.bool, device="cuda")
    mask[cfg.T - cfg.T // 16:] = False
    return h.to(torch.bfloat16), (0.5 * r).to(torch.bfloat16), (0.5 * t).to(torch.bfloat16), mask


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--workload", default="tiny", choices=("tiny", "small"))
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    cfg = workloads.get(a.workload)
    block = Block(cfg, a.bits)
    h, r, target, mask = data(cfg)
    for i in range(a.steps):
        out = block.train_step(h, r, target, mask)
        if i % max(1, a.steps // 10) == 0 or i == a.steps - 1:
            print("step %3d  loss %.4f  balance %.4f  z %.3f  grad norm %.4f" % (
                i + 1, out["loss"], out["balance"], out["z"], out["grad_norm"]))


if __name__ == "__main__":
    main()
