"""Trains one pre-norm MoE block on a fixed random teacher, on one GPU.

    python examples/train_moe_layer.py [--steps 60] [--rate 1/2] [--state f8] [--tight]

Every step runs the whole chain of a training step with this package's kernels:

  h = x + residual, u = RMS norm of h                      AddRMSNorm
  logits = u W_r                                           (a library product)
  experts, weights, counts, balance loss and z-loss        Router
  dispatch, SwiGLU experts, weighted combine               RecalibratedExpertBackward.forward
  loss = mean (h + out - target)^2 / 2 + the two losses
  d alpha, d logits                                        .gate_grad, Router.backward
  score, select, compact, expert backward                  .step (the retained pairs only)
  d u -> d x, d w                                          AddRMSNorm.backward
  all weights, norm and router among them                  AdamW

With --tight, the block of a model that is short of memory (TightMoeBlock):

  experts of the best groups, with a bias that evens the loads   GroupRouter
  the saved state in 8 bits                                      PackedState, .forward, .step
  norm of the experts' output, gate, scaled residual and the
  norm in front of the next block                                BlockNorm

and the experts' buffers, [a | b] and phi among them, are one set for all blocks (here for the
teacher and the trained one).
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from demand_side_expert_gb300 import (AddRMSNorm, AdamW, BlockNorm, GroupRouter,  # noqa: E402
                                      PackedState, RecalibratedExpertBackward, Router)


def init_weights(D: int, H: int, E: int, seed: int, device="cuda") -> dict:
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def randn(*shape, scale):
        return (torch.randn(*shape, generator=gen, device=device) * scale).to(torch.bfloat16)

    return {"norm": torch.ones(D, dtype=torch.bfloat16, device=device),
            "router": randn(D, E, scale=D ** -0.5),
            "gate": randn(E, D, H, scale=D ** -0.5), "up": randn(E, D, H, scale=D ** -0.5),
            "down": randn(E, H, D, scale=H ** -0.5)}


class MoeBlock:
    """out = h + MoE(RMS norm(h)), h = x + residual, with its backward pass."""

    def __init__(self, T, D, H, E, K, weights: dict, balance_coef=0.01, z_coef=0.001):
        self.w = weights
        self.norm = AddRMSNorm(T, D, "bf16")
        self.router = Router(T, E, K, "bf16", renorm=True, balance_coef=balance_coef,
                             z_coef=z_coef)
        self.experts = RecalibratedExpertBackward(T, D, H, E, K, "bf16")
        ex = self.experts
        self.grads = {"norm": self.norm.dw, "router": torch.empty(D, E, device="cuda"),
                      "gate": ex.dw_gate, "up": ex.dw_up, "down": ex.dw_down}

    def forward(self, x, residual):
        w, ex = self.w, self.experts
        self.norm.forward(x, w["norm"], residual=residual)
        self.logits = self.norm.y @ w["router"]
        self.router.route(self.logits)
        ex.forward(self.router.topk_idx, self.router.alpha, self.norm.y, w["gate"], w["up"],
                   w["down"])
        return self.norm.h.float() + ex.out

    def backward(self, g, rate=(1, 1)):
        """g [T, D] float32: the cotangent of forward's result. Leaves the weights'
        gradients in ``grads`` and returns the one of x (and of the residual)."""
        w, ex = self.w, self.experts
        g16 = g.to(torch.bfloat16)
        dalpha = ex.gate_grad(g16)
        self.router.backward(self.logits, dalpha)
        u = self.norm.y
        ex.step(self.router.topk_idx, self.router.alpha, u, g16, ex.ab, ex.phi, w["gate"],
                w["up"], w["down"], rate=rate, gathered=True)
        dlogits = self.router.dlogits
        self.grads["router"].copy_(u.t() @ dlogits)
        du = ex.dx + (dlogits @ w["router"].t()).float()
        self.norm.backward(du, w["norm"], dh=g)
        return self.norm.dx


class TightMoeBlock:
    """y = RMS norm(h'), h' = scale * h + gate * RMS norm(MoE(RMS norm(h))), h = x + residual:
    norms on both sides of the experts. Weights beside ``init_weights``'s: "post", "next" and
    "layer_scale" [D]; ``bias`` [E] float32 is moved by the loads, not by a gradient.

    ``experts``: another block's, whose buffers then serve both, one after the other. What a
    block keeps of its own from forward to backward: h, u, h' [T, D], the logits, choices and
    weights, 8-bit rows of [a | b], the experts' output before and behind the combination (``y``
    [T*K, D], which the routing weights' gradient reads, and ``out`` [T, D] float32), and its
    weights' gradients."""

    SCALE = 0.8  # of the residual

    def __init__(self, T, D, H, E, K, weights: dict, groups=4, top_groups=2, balance_coef=0.001,
                 packed=True, experts=None):
        if experts is not None and not packed:
            raise ValueError("experts: the state in 16 bits stands in their buffers, of one block")
        self.w = weights
        self.norm = AddRMSNorm(T, D, "bf16")
        self.router = GroupRouter(T, E, K, "bf16", groups=groups, top_groups=top_groups,
                                  balance_coef=balance_coef)
        self.experts = experts or RecalibratedExpertBackward(T, D, H, E, K, "bf16")
        self.y = torch.empty(T * K, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(T, D, device="cuda")
        self.state = PackedState(T, K, H, "bf16", cols=64) if packed else None
        self.after = BlockNorm(T, D, "bf16", gate="column", residual_scale=self.SCALE)
        self.bias = torch.zeros(E, device="cuda")
        self.grads = {"norm": self.norm.dw, "router": torch.empty(D, E, device="cuda"),
                      "gate": torch.empty(E, D, H, device="cuda"),
                      "up": torch.empty(E, D, H, device="cuda"),
                      "down": torch.empty(E, H, D, device="cuda"),
                      "post": self.after.dw_post, "next": self.after.dw,
                      "layer_scale": self.after.dgate}

    def forward(self, x, residual):
        w, ex, r = self.w, self.experts, self.router
        self.norm.forward(x, w["norm"], residual=residual)
        self.logits = self.norm.y @ w["router"]
        r.route(self.logits, bias=self.bias)
        ex.y, ex.out = self.y, self.out
        ex.forward(r.topk_idx, r.alpha, self.norm.y, w["gate"], w["up"], w["down"],
                   packed=self.state)
        self.after.forward(self.out, self.norm.h, w["next"], w_post=w["post"], gate=w["layer_scale"])
        return self.after.y.float()

    def even_loads(self, rate=1e-3):
        self.router.next_bias(self.bias, rate, out=self.bias)

    def backward(self, g, rate=(1, 1)):
        """g [T, D] float32: the cotangent of forward's result. Leaves the weights'
        gradients in ``grads`` and returns the one of x (and of the residual)."""
        w, ex, r, n = self.w, self.experts, self.router, self.after
        n.backward(g, self.out, w["next"], w["post"], w["layer_scale"])
        u = self.norm.y
        saved = (ex.ab, ex.phi) if self.state is None else (self.state, None)
        ex.y, ex.dw_gate, ex.dw_up, ex.dw_down = (self.y, self.grads["gate"], self.grads["up"],
                                                  self.grads["down"])
        ex.step(r.topk_idx, r.alpha, u, n.dblock, *saved, w["gate"], w["up"], w["down"],
                rate=rate, gathered=True)
        # after the step, whose dispatch is of this block's choices
        r.backward(self.logits, ex.gate_grad(n.dblock))
        self.grads["router"].copy_(u.t() @ r.dlogits)
        du = ex.dx + (r.dlogits @ w["router"].t()).float()
        self.norm.backward(du, w["norm"], dh=n.dres)
        return self.norm.dx


def tight_weights(D: int, H: int, E: int, seed: int, device="cuda") -> dict:
    w = init_weights(D, H, E, seed, device)
    for name in ("post", "next"):
        w[name] = torch.ones(D, dtype=torch.bfloat16, device=device)
    w["layer_scale"] = torch.full((D,), 0.5, dtype=torch.bfloat16, device=device)
    return w


def train(steps=60, T=2048, D=256, H=128, E=16, K=2, rate=(1, 2), state="f32", lr=2e-3, seed=0,
          log=None, tight=False) -> list:
    """The loss of every step."""
    make, weights = (TightMoeBlock, tight_weights) if tight else (MoeBlock, init_weights)
    teacher = make(T, D, H, E, K, weights(D, H, E, seed + 1))
    shared = {"experts": teacher.experts} if tight else {}
    block = make(T, D, H, E, K, weights(D, H, E, seed + 2), **shared)
    names = list(block.w)
    opt = AdamW([block.w[n] for n in names], [block.grads[n] for n in names], lr=lr,
                betas=(0.9, 0.95),
                weight_decay=[0.0 if block.w[n].dim() == 1 else 0.01 for n in names],
                state=state, master=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    losses = []
    for i in range(steps):
        x = torch.randn(T, D, generator=gen, device="cuda").to(torch.bfloat16)
        residual = torch.randn(T, D, generator=gen, device="cuda").to(torch.bfloat16)
        target = teacher.forward(x, residual)
        diff = block.forward(x, residual) - target
        loss = diff.square().mean() / 2 + block.router.loss.sum()
        losses.append(loss.clone())
        block.backward(diff / diff.numel(), rate=rate)
        opt.step()
        if tight:
            block.even_loads()
        if log and (i % log == 0 or i == steps - 1):
            print(f"step {i:4d}  loss {loss.item():.5f}  balance {block.router.loss[0].item():.5f}"
                  f"  largest share {block.router.counts.max().item() / (T * K):.3f}")
    if block.experts.device_error() or block.router.device_error():
        raise RuntimeError("a kernel flagged bad data")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--rate", default="1/2", help="retention rate of the expert backward")
    ap.add_argument("--state", choices=("f32", "f8"), default="f32", help="AdamW's moments")
    ap.add_argument("--tight", action="store_true", help="the block that saves memory")
    a = ap.parse_args()
    num, den = (int(v) for v in a.rate.split("/"))
    train(a.steps, rate=(num, den), state=a.state, log=10, tight=a.tight)
