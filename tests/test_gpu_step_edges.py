"""GPU tests of what the training-step operators meet at the edges of their use: other
streams, several host threads, bad entries beside infinities, far tails, and the kernel
forms that only large blocks or many tensors take."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    from demand_side_expert_gb300 import lrm  # noqa: F401  (liblrm.so must load)
    return torch.device("cuda:0")


# -- streams ------------------------------------------------------------------
@pytest.fixture(params=["stream", "address", "default"])
def other_stream(request, dev):
    """A call's stream that is not torch's current one: (the current one, the argument)."""
    if request.param == "default":  # the legacy stream's address is 0
        return torch.cuda.Stream(), 0
    side = torch.cuda.Stream()
    return torch.cuda.default_stream(), side if request.param == "stream" else side.cuda_stream


def first_call(streams, shape, dtype, call, result):
    """``call`` allocates ``result()`` on its first run, in a block that was freed with a
    write still pending on the current stream; returns what the buffer ends up with."""
    current, argument = streams
    with torch.cuda.stream(current):
        junk = torch.empty(*shape, dtype=dtype, device="cuda")
        junk.fill_(7)
        torch.cuda._sleep(1000)  # both kernels are loaded before anything waits
        del junk
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        junk = torch.empty(*shape, dtype=dtype, device="cuda")
        at = junk.data_ptr()
        torch.cuda._sleep(200_000_000)  # 0.1 s
        junk.fill_(7)
        del junk
        call(argument)
        assert result().data_ptr() == at, "the freed block was not the one that was taken"
    torch.cuda.synchronize()
    return result().clone()


def test_first_router_gradient_on_another_stream(dev, other_stream):
    from demand_side_expert_gb300 import Router

    x = torch.randn(40000, 64, device=dev)
    r, s = Router(40000, 64, 4, "f32"), Router(40000, 64, 4, "f32")
    r.route(x)
    s.route(x)
    s.backward(x, s.alpha)
    got = first_call(other_stream, (40000, 64), torch.float32,
                     lambda st: r.backward(x, r.alpha, stream=st), lambda: r.dlogits)
    assert torch.equal(got, s.dlogits)


def test_first_norm_calls_on_another_stream(dev, other_stream):
    from demand_side_expert_gb300 import AddRMSNorm

    x, w = torch.randn(5000, 512, device=dev), torch.ones(512, device=dev)
    n, m = AddRMSNorm(5000, 512, "f32"), AddRMSNorm(5000, 512, "f32")
    m.forward(x, w, residual=x)
    m.backward(x, w)
    got = first_call(other_stream, (5000, 512), torch.float32,
                     lambda st: n.forward(x, w, residual=x, stream=st), lambda: n.h)
    assert torch.equal(got, m.h)
    got = first_call(other_stream, (5000, 512), torch.float32,
                     lambda st: n.backward(x, w, stream=st), lambda: n.dx)
    assert torch.equal(got, m.dx) and torch.equal(n.dw, m.dw)


def test_first_expert_calls_on_another_stream(dev, other_stream):
    from demand_side_expert_gb300 import RecalibratedExpertBackward

    T, D, H, E, K = 100000, 64, 64, 8, 4
    p, q = (RecalibratedExpertBackward(T, D, H, E, K, "bf16") for _ in range(2))
    gen = torch.Generator().manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).to(dev)

    idx = (torch.arange(T * K, dtype=torch.int32).view(T, K) % E).to(dev)
    alpha, x = torch.ones(T, K, device=dev), randn(T, D)
    args = (idx, alpha, x, randn(E, D, H), randn(E, D, H), randn(E, H, D))
    q.forward(*args)
    want = q.gate_grad(x).clone()
    # the layer output [T, D] float32 is the one forward buffer of that size
    got = first_call(other_stream, (T, D), torch.float32,
                     lambda st: p.forward(*args, stream=st), lambda: p.out)
    assert torch.equal(got, q.out)
    got = first_call(other_stream, (T, K), torch.float32,
                     lambda st: p.gate_grad(x, stream=st), lambda: p.dalpha)
    assert torch.equal(got, want)
