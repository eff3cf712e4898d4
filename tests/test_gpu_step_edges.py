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


# -- several host threads -------------------------------------------------------
def in_threads(jobs, times):
    """Every job in a thread and on a stream of its own; the errors that came up."""
    import threading

    errors = []

    def work(job):
        stream = torch.cuda.Stream()
        try:
            for _ in range(times):
                job(stream)
        except Exception as e:
            errors.append(repr(e))
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("copies", [1, 2])
def test_norm_gradients_in_threads(dev, copies):
    """Calls with different needs of shared memory on the same kernels (f32, two units a
    thread, 96 bytes a unit: 49 KB for a row of 4096 a CTA, 98 KB for two) at the same
    time."""
    from demand_side_expert_gb300 import AddRMSNorm

    jobs, want = [], []
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    for T, D in ((2 * sms, 4096), (sms, 4096)) * copies:
        x, w = torch.randn(T, D, device=dev), torch.ones(D, device=dev)
        n = AddRMSNorm(T, D, "f32")
        n.forward(x, w)
        n.backward(x, w, dh=x, h=x)
        want.append((n, n.dx.clone(), n.dw.clone()))
        jobs.append(lambda st, n=n, x=x, w=w: n.backward(x, w, dh=x, h=x, stream=st))
    assert in_threads(jobs, 5000) == []
    for n, dx, dw in want:
        assert torch.equal(n.dx, dx) and torch.equal(n.dw, dw)


def test_routers_in_threads(dev):
    """The same of the router's statistics: 64 KB for 512 experts, 50 KB for 400."""
    from demand_side_expert_gb300 import Router

    jobs, want = [], []
    for E in (400, 512, 400, 512):
        x = torch.randn(9000, E, device=dev).bfloat16()
        r = Router(9000, E, 4, "bf16")
        r.route(x)
        want.append((r, r.alpha.clone(), r.prob_sum.clone(), r.loss.clone()))
        jobs.append(lambda st, r=r, x=x: r.route(x, stream=st))
    assert in_threads(jobs, 5000) == []
    for r, alpha, prob_sum, loss in want:
        assert torch.equal(r.alpha, alpha) and torch.equal(r.prob_sum, prob_sum)
        assert torch.equal(r.loss, loss)


# -- routing weights' gradient ----------------------------------------------------
def gate_grad_of(g, y, inv, K, dev):
    """dalpha and the device error word; g, y, inv on the device."""
    from demand_side_expert_gb300 import lrm

    T, D = g.shape
    shape = lrm.make_shape(T, D, 8, max(K, 4), K,
                           lrm.LRM_BF16 if g.dtype is torch.bfloat16 else lrm.LRM_F32)
    n = lrm.lrm_workspace_bytes(shape)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    out = torch.full((T, K), float("nan"), device=dev)
    lrm.lrm_gate_grad(shape, g, y, inv, out, ws, n)
    return out, lrm.lrm_get_device_error(ws, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 4, 8, 9])
@pytest.mark.parametrize("tokens_per_sm", [0, 3])
def test_gate_grad_bad_entries_beside_infinities(dev, tokens_per_sm, K, dtype):
    """A bad entry of inv gives 0 also where the token's cotangent is infinite or NaN; a
    warp a token (3 tokens an SM) and a CTA a token (4 tokens)."""
    from demand_side_expert_gb300 import lrm

    T = tokens_per_sm * torch.cuda.get_device_properties(dev).multi_processor_count or 4
    D = 72
    gen = torch.Generator().manual_seed(K)
    g = torch.randn(T, D, generator=gen)
    g[0, 3], g[T - 1, 71] = float("inf"), float("nan")
    y = torch.randn(T * K, D, generator=gen)
    inv = torch.randperm(T * K, generator=gen).to(torch.int32)
    inv[0], inv[T * K - 1] = T * K, -1
    out, err = gate_grad_of(g.to(DT[dtype]).to(dev), y.to(DT[dtype]).to(dev), inv.to(dev), K, dev)
    assert out[0, 0].item() == 0 and out[T - 1, K - 1].item() == 0
    assert not torch.isfinite(out[0, 1:]).any() and not torch.isfinite(out[T - 1, :K - 1]).any()
    assert torch.isfinite(out[1:T - 1]).all()
    assert err == lrm.LRM_DEVERR_INDEX


# -- router: far tails ------------------------------------------------------------
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E", [(64, 8), (64, 300), (5000, 8), (5000, 200)])
def test_route_weights_far_below_the_largest(dev, T, E, dtype, renorm):
    """Weights of 1e-13 down to the smallest number keep float32's relative accuracy, and so
    do float32 gradients. The logits are whole numbers and the largest is 0, so differences
    are exact; every other weight is below 2^-43, so sums of up to 300 round to 1 in float32
    and are 1 + 4e-11 at most. What is left is the exponential (2 ulp) and one product."""
    from demand_side_expert_gb300 import Router

    K, low = 8, 103
    t, e = torch.arange(T)[:, None], torch.arange(E)[None]
    x = -(30 + (t * 7 + e * 11) % (low - 29)).float()
    x[:, 3] = 0
    r = Router(T, E, K, dtype, renorm=renorm, balance_coef=0.0, z_coef=0.0)
    xd = x.to(DT[dtype]).to(dev)
    r.route(xd)
    idx = r.topk_idx.cpu().long()
    p = torch.exp(x.double())
    want = p.gather(1, idx)
    err = (r.alpha.cpu().double() - want).abs()
    assert (err <= 6 * U * want + 2.0 ** -149).all(), (err / want).max().item() / U

    # dalpha 1 at the choices but the first: dx = a there, to the rest's share of 1e-12,
    # and minus their sum at the first
    r.backward(xd, (idx != 3).float().to(dev))
    got = r.dlogits.cpu().double().gather(1, idx)[:, 1:]
    # two exponentials' roundings and four products; the gradient's own type
    lim = (12 * U + (0 if dtype == "f32" else 2.0 ** -8)) * want[:, 1:]
    # below 2^-126 a product may be rounded twice to a multiple of 2^-149 (2^-133)
    lim = lim + (2.0 ** -148 if dtype == "f32" else 2.0 ** -126)
    assert ((got - want[:, 1:]).abs() <= lim).all()


def test_route_z_loss_of_even_logits(dev):
    """log 2 and log 3 to float32's accuracy: a token's lse is a logarithm and one sum."""
    import math

    from demand_side_expert_gb300 import Router

    for E in (2, 3):
        r = Router(1, E, 1, "f32", balance_coef=0.0, z_coef=1.0)
        r.route(torch.zeros(1, E, device=dev))
        want = math.log(E) ** 2
        # the logarithm 2 ulp = 4 u, squared twice that, and one product
        assert abs(r.loss[1].item() - want) <= 10 * U * want


def check_gate_grad(T, D, K, dtype, dev, bad=True):
    """All of dalpha against float64 sums; with a bad entry of inv in the middle."""
    from demand_side_expert_gb300 import lrm

    gen = torch.Generator(device=dev).manual_seed(T + D + K)
    g = torch.empty(T, D, dtype=DT[dtype], device=dev).normal_(generator=gen)
    y = torch.empty(T * K, D, dtype=DT[dtype], device=dev).normal_(generator=gen)
    inv = torch.randperm(T * K, generator=gen, device=dev).to(torch.int32)
    spot = (T // 2) * K + K - 1
    if bad:
        inv[spot] = T * K
    out, err = gate_grad_of(g, y, inv, K, dev)
    assert err == (lrm.LRM_DEVERR_INDEX if bad else 0)
    for t in range(0, T, 1024):
        rows = y[inv[t * K:(t + 1024) * K].long().clamp(max=T * K - 1)].double()
        rows = rows.view(-1, K, D)
        prod = rows * g[t:t + 1024, None].double()
        want, mag = prod.sum(2), prod.abs().sum(2)
        if bad and t <= T // 2 < t + 1024:
            want.view(-1)[spot - t * K] = 0
            assert out.view(-1)[spot].item() == 0
        # D terms, each product's and each sum's rounding
        off = (out[t:t + 1024].double() - want).abs() > (D + 1) * U * mag
        assert not off.any(), (t, int(off.sum()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 3, 8, 9, 32])
@pytest.mark.parametrize("D", [8, 72, 1000])
def test_gate_grad_by_warps(dev, D, K, dtype):
    """A warp a token, past the number of warps a grid has (at most 4 a CTA, 3 rounds of 4
    CTAs an SM): tokens follow one another in a warp, in several passes for K > 8."""
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    if (K + 1) * D * torch.finfo(DT[dtype]).bits // 8 >= 35 * 1024:
        pytest.skip("a CTA a token")
    check_gate_grad(sms * 48 + 1203, D, K, dtype, dev)


@pytest.mark.parametrize("T,D,K,dtype", [
    (64, 2040, 8, "bf16"), (64, 1000, 8, "f32"), (64, 1000, 20, "bf16"), (64, 504, 32, "f32"),
    (2, 1000, 9, "f32"), (2, 4104, 1, "bf16"), (2, 2056, 2, "f32"), (2, 4088, 4, "bf16"),
    (2, 2056, 3, "f32")])
def test_gate_grad_by_ctas(dev, T, D, K, dtype):
    """A CTA a token, T tokens an SM and some: 64 is past the number of CTAs a grid has."""
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    check_gate_grad(sms * T + 101, D, K, dtype, dev, bad=K > 1)
