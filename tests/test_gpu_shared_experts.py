"""One set of experts' buffers for several layers: the same gradients as with a set each."""

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


@pytest.mark.parametrize("rate", [(1, 1), (1, 2)])
def test_layers_share_their_experts(example, rate):
    """Three blocks with weights of their own, forward one after the other and back again."""
    T, D, H, E, K = 256, 128, 64, 16, 4
    gen = torch.Generator().manual_seed(0)
    x, res, g = (torch.randn(T, D, generator=gen).cuda() for _ in range(3))
    got = []
    for shared in (False, True):
        experts, blocks = None, []
        for seed in (1, 2, 3):
            w = example.tight_weights(D, H, E, seed)
            blocks.append(example.TightMoeBlock(T, D, H, E, K, w, balance_coef=0.1,
                                                experts=experts))
            if shared:
                experts = blocks[0].experts
        for _ in range(2):
            v, outs = x, []
            for b in blocks:
                outs.append(b.forward(v.to(torch.bfloat16), res.to(torch.bfloat16)))
                v = outs[-1]
            d = g
            for b in reversed(blocks):
                d = b.backward(d.float(), rate=rate)
        for b in blocks:
            assert b.experts.device_error() == 0 and b.router.device_error() == 0
        got.append(outs + [d] + [b.grads[n] for b in blocks for n in sorted(b.grads)])
    assert len({b.experts for b in blocks}) == 1
    for a, b in zip(*got):
        assert torch.equal(a, b) and torch.isfinite(a).all() and (a != 0).any()


def test_calls_of_two_layers_by_hand(example):
    """The same with the calls themselves: rows of a layer's own in ``y`` and ``out``, its
    choices dispatched before ``gate_grad``."""
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward
    from workloads import generate, get_config

    T, D, H, E, K = 192, 128, 64, 8, 2
    cfg = get_config("qwen3-30b-a3b-t4k", T=T, D=D, H=H, E=E, K=K)
    layers = [{k: v.cuda() if torch.is_tensor(v) else v for k, v in
               generate(cfg, device="cpu", seed=s).items()} for s in (1, 2)]

    def weights(d):
        return d["w_gate"], d["w_up"], d["w_down"]

    def new():
        return RecalibratedExpertBackward(T, D, H, E, K, "bf16")

    def run(pipes):
        got = []
        for d, pipe in zip(layers, pipes):
            d["y"] = torch.empty(T * K, D, dtype=torch.bfloat16, device="cuda")
            d["out"] = torch.empty(T, D, device="cuda")
            d["state"] = PackedState(T, K, H, "bf16")
            pipe.y, pipe.out = d["y"], d["out"]
            pipe.forward(d["topk_idx"], d["alpha"], d["x"], *weights(d), packed=d["state"])
        for d, pipe in reversed(list(zip(layers, pipes))):
            pipe.y = d["y"]
            pipe.dispatch(d["topk_idx"])
            got.append(pipe.gate_grad(d["g"]).clone())
            pipe.step(d["topk_idx"], d["alpha"], d["x"], d["g"], d["state"], None, *weights(d),
                      rate=(1, 2), gathered=True)
            got += [getattr(pipe, n).clone() for n in ("dw_gate", "dw_up", "dw_down", "dx")]
            got += [d["out"], d["y"]]
        return got

    one = new()
    for a, b in zip(run([new(), new()]), run([one, one])):
        assert torch.equal(a, b)
