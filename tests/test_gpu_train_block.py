"""The operators together, as one training step of a pre-norm MoE block: the block's
gradients against torch autograd on the same weights, and a short training run."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_moe_layer
    return train_moe_layer


def test_block_gradients_match_autograd(example):
    """Plain float32 autograd of the block, with the kernels' choices of experts (a
    rounding of u can swap two nearly equal logits). The kernels round u, the logits,
    [a | b], phi, y, g and dlogits to bfloat16, 2^-9 each; about ten such roundings
    stand between the loss and a gradient, and random ones add in squares: 2e-2."""
    T, D, H, E, K = 256, 128, 64, 8, 2
    w = example.init_weights(D, H, E, 3)
    gen = torch.Generator().manual_seed(0)
    w["norm"].copy_(1 + 0.2 * torch.randn(D, generator=gen))
    block = example.MoeBlock(T, D, H, E, K, w, balance_coef=0.1, z_coef=0.05)
    x, res = (torch.randn(T, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    g = torch.randn(T, D, generator=gen).cuda()
    out = block.forward(x, res).clone()
    dx = block.backward(g)
    idx, counts = block.router.topk_idx.long(), block.router.counts.float()

    p = {k: v.float().requires_grad_(True) for k, v in w.items()}
    h = (x.float() + res.float()).requires_grad_(True)
    u = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * p["norm"]
    logits = u @ p["router"]
    probs = torch.softmax(logits, 1)
    a = probs.gather(1, idx)
    a = a / a.sum(1, keepdim=True)
    moe = torch.zeros_like(h)
    for k in range(K):
        gate = torch.einsum("td,tdh->th", u, p["gate"][idx[:, k]])
        up = torch.einsum("td,tdh->th", u, p["up"][idx[:, k]])
        moe = moe + a[:, k:k + 1] * torch.einsum(
            "th,thd->td", torch.nn.functional.silu(gate) * up, p["down"][idx[:, k]])
    ref = h + moe
    balance = 0.1 * E * (counts / (T * K) * probs.mean(0)).sum()
    z = 0.05 * torch.logsumexp(logits, 1).square().mean()
    ((ref * g).sum() + balance + z).backward()

    def rel(got, want):
        return ((got.float() - want).norm() / want.norm()).item()

    assert rel(out, ref.detach()) < 2e-2
    assert rel(dx, h.grad) < 2e-2
    for name, got in block.grads.items():
        assert rel(got, p[name].grad) < 2e-2, name
    assert abs(block.router.loss[0].item() - balance.item()) < 2e-2 * balance.item()
    assert abs(block.router.loss[1].item() - z.item()) < 2e-2 * z.item()


@pytest.mark.parametrize("state,rate", [("f32", (1, 1)), ("f8", (1, 1)), ("f8", (1, 2))])
def test_training_lowers_the_loss(example, state, rate):
    losses = example.train(steps=60, T=1024, D=128, H=64, E=8, K=2, state=state, rate=rate)
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert last < 0.8 * first, (first, last)


def test_8_bit_moments_train_like_32_bit_ones(example):
    """The same run with either kind of moments ends within a tenth of the other."""
    a = example.train(steps=60, T=1024, D=128, H=64, E=8, K=2, state="f32", rate=(1, 1))
    b = example.train(steps=60, T=1024, D=128, H=64, E=8, K=2, state="f8", rate=(1, 1))
    a, b = sum(a[-5:]) / 5, sum(b[-5:]) / 5
    assert abs(a - b) < 0.1 * a, (a, b)
