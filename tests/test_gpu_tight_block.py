"""The operators for training under tight memory together, as one training step of the
example's block: its gradients against torch autograd on the same weights, a step captured
into a graph, and the example itself."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu
SIZES = dict(T=256, D=128, H=64, E=16, K=4)


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_moe_layer
    return train_moe_layer


def make(example, packed, seed=3):
    s = SIZES
    w = example.tight_weights(s["D"], s["H"], s["E"], seed)
    gen = torch.Generator().manual_seed(seed)
    for name in ("norm", "post", "next"):
        w[name].copy_(1 + 0.2 * torch.randn(s["D"], generator=gen))
    w["layer_scale"].copy_(0.5 + 0.2 * torch.randn(s["D"], generator=gen))
    block = example.TightMoeBlock(**s, weights=w, balance_coef=0.1, packed=packed)
    block.bias.copy_(0.05 * torch.randn(s["E"], generator=gen))
    x, res = (torch.randn(s["T"], s["D"], generator=gen).to(torch.bfloat16).cuda()
              for _ in range(2))
    g = torch.randn(s["T"], s["D"], generator=gen).cuda()
    return block, x, res, g


def rel(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("packed", [False, True])
def test_block_gradients_match_autograd(example, packed):
    """Plain float32 autograd of the block, with the kernels' choices of experts. About ten
    roundings to bfloat16, 2^-9 each, stand between the loss and a gradient, and random ones
    add in squares: 2e-2. From the 8-bit state the experts' gradients carry its rounding, up
    to 2^-4 of a value and a third of that in the mean, through two factors: 2^-4 in all."""
    block, x, res, g = make(example, packed)
    E, K, T = SIZES["E"], SIZES["K"], SIZES["T"]
    out = block.forward(x, res).clone()
    dx = block.backward(g)
    idx, counts = block.router.topk_idx.long(), block.router.counts.float()
    assert block.experts.device_error() == 0 and block.router.device_error() == 0

    p = {k: v.float().requires_grad_(True) for k, v in block.w.items()}
    h = (x.float() + res.float()).requires_grad_(True)

    def norm(v, w):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w

    u = norm(h, p["norm"])
    s = torch.sigmoid(u @ p["router"])
    # the groups that the choices come from: two of four
    assert all(len({int(e) // (E // 4) for e in row}) <= 2 for row in idx)
    a = s.gather(1, idx)
    a = a / a.sum(1, keepdim=True)
    moe = torch.zeros_like(h)
    for k in range(K):
        gate = torch.einsum("td,tdh->th", u, p["gate"][idx[:, k]])
        up = torch.einsum("td,tdh->th", u, p["up"][idx[:, k]])
        moe = moe + a[:, k:k + 1] * torch.einsum(
            "th,thd->td", torch.nn.functional.silu(gate) * up, p["down"][idx[:, k]])
    after = block.SCALE * h + p["layer_scale"] * norm(moe, p["post"])
    ref = norm(after, p["next"])
    share = s / s.sum(1, keepdim=True)
    balance = 0.1 * E * (counts / (T * K) * share.mean(0)).sum()
    ((ref * g).sum() + balance).backward()

    assert rel(out, ref.detach()) < 2e-2
    assert rel(dx, h.grad) < (2.0 ** -4 if packed else 2e-2)
    for name, got in block.grads.items():
        experts = packed and name in ("gate", "up", "down", "norm")
        assert rel(got, p[name].grad) < (2.0 ** -4 if experts else 2e-2), name
    assert abs(block.router.loss[0].item() - balance.item()) < 2e-2 * balance.item()


def test_step_in_a_graph(example):
    """A captured step, forward and backward, replays on new inputs as the eager one runs,
    beside an eager block of the same shape."""
    block, x, res, g = make(example, True)
    other, _, _, _ = make(example, True, seed=4)
    for _ in range(2):
        block.forward(x, res)
        block.backward(g, rate=(1, 2))
    want = {k: v.clone() for k, v in block.grads.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    held = x.clone()
    with torch.cuda.stream(st):
        block.forward(held, res)  # the library's products pick their workspace
        block.backward(g, rate=(1, 2))
        with torch.cuda.graph(graph, stream=st):
            block.forward(held, res)
            block.backward(g, rate=(1, 2))
    other.forward(x, res)
    other.backward(g)
    graph.replay()
    torch.cuda.synchronize()
    for k, v in want.items():
        assert torch.equal(v, block.grads[k]), k
    held.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in block.grads.items()}
    block.forward(held, res)
    block.backward(g, rate=(1, 2))
    for k, v in got.items():
        assert torch.equal(v, block.grads[k]), k
    assert not torch.equal(got["gate"], want["gate"])


@pytest.mark.parametrize("rate", [(1, 1), (1, 2)])
def test_example_runs(example, rate):
    losses = example.train(steps=6, T=512, D=128, H=64, E=16, K=4, rate=rate, tight=True)
    assert len(losses) == 6 and all(v == v and 0 < v < 10 for v in losses)
