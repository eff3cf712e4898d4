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


# -- norm: the forms of large blocks -----------------------------------------------
def norm_of(x, res, w, eps):
    """h, rstd and y in 64 bits."""
    h = x.double() if res is None else x.double() + res.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    return h, rstd, h * rstd[:, None] * w.double()


def within(got, want, lim, name):
    off = (got.double() - want).abs() > lim
    assert not off.any(), (name, int(off.sum()), (got.double() - want).abs().max().item())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [264, 1000, 1032, 2040, 4088, 8184, 8200])
def test_norm_forward_of_large_blocks(dev, D, dtype, residual):
    """More than 16384 values an SM, where several units a thread (and for bfloat16 rows
    without a residual other threads a row) take over: every output, each width of the
    8-bit groups."""
    from demand_side_expert_gb300 import AddRMSNorm

    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    T, eps = sms * 16384 // D + 3, 1e-5
    gen = torch.Generator(device=dev).manual_seed(D)
    dt = DT[dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    x, w = randn(T, D).to(dt), (1 + 0.2 * randn(D)).to(dt)
    res = (3 * randn(T, D)).to(dt) if residual else None
    h, rstd, y = norm_of(x, res, w, eps)
    out = 2.0 ** -8 if dtype == "bf16" else 0.0  # the rounding of a stored value
    rs = (D + 8) * U  # D squares and sums, a division, a root
    mag = y.abs()
    h_lim = U * (x.double().abs() + (0 if res is None else res.double().abs()))
    if residual:  # the rounding of the sum reaches y times rstd w
        mag = mag + h_lim / U * rstd[:, None] * w.double().abs()
    y_lim = (rs + 4 * U) * mag
    for q_cols in (None, 0, 32, 64, 128, 256):
        n = AddRMSNorm(T, D, dtype, eps=eps, q_cols=q_cols, store_y=q_cols in (None, 64))
        n.forward(x, w, residual=res)
        within(n.rstd, rstd, rs * rstd, "rstd")
        if residual:
            within(n.h, h, out * h.abs() + 2 * h_lim, "h")
        if n.y is not None:
            within(n.y, y, out * y.abs() + y_lim, "y")
        if q_cols is None:
            continue
        cols = q_cols or D
        groups = -(-D // cols)
        pad = (0, groups * cols - D)
        top = torch.nn.functional.pad(y.abs(), pad).view(T, groups, cols).amax(2) / 448
        slack = torch.nn.functional.pad(y_lim, pad).view(T, groups, cols).amax(2) / 448
        within(n.q_scale, top, slack + 4 * U * top, "q_scale")
        scale = n.q_scale.double().repeat_interleave(cols, 1)[:, :D]
        # half a step of the code: 2^-4 of a normal value, 2^-10 below
        half = torch.maximum(y.abs() * 2.0 ** -4, scale * 2.0 ** -10)
        within(n.q.double() * scale, y, half * (1 + 1e-3) + 4 * y_lim, "q")


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,rows_per_sm", [(16384, 4), (8200, 7), (8192, 9), (1032, 40), (72, 300)])
def test_norm_backward_of_many_rows(dev, D, rows_per_sm, dtype, grad):
    """More rows a CTA than its ring has places, at every depth of the ring: the places are
    used again and again. With the residual stream's gradient."""
    from demand_side_expert_gb300 import AddRMSNorm

    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    T = rows_per_sm * sms + 5
    gen = torch.Generator(device=dev).manual_seed(D)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    x, w = randn(T, D).to(DT[dtype]), (1 + 0.2 * randn(D)).to(DT[dtype])
    dy, dh = randn(T, D).to(DT[grad]), randn(T, D).to(DT[grad])
    n = AddRMSNorm(T, D, dtype, eps=1e-5, grad_dtype=grad)
    n.forward(x, w)
    n.backward(dy, w, dh=dh, h=x)
    rstd, d64, w64 = n.rstd.double()[:, None], dy.double(), w.double()
    xhat, wdy = x.double() * rstd, dy.double() * w64
    dx = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True)) + dh.double()
    # D products and sums of the row's mean, and 8 roundings of what it is taken from
    mag = rstd * (wdy.abs() * 8 + xhat.abs() * (wdy * xhat).abs().mean(1, keepdim=True) * (D + 8))
    lim = U * (mag + 2 * dh.double().abs())
    if grad == "bf16":
        lim = lim + 2.0 ** -8 * dx.abs()
    within(n.dx, dx, lim, "dx")
    within(n.dw, (d64 * xhat).sum(0), (T + 3) * U * (d64 * xhat).abs().sum(0), "dw")


# -- router: rounds and shared memory of many tokens ----------------------------------
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,K,dtype", [(20, 3, "f32"), (32, 12, "bf16"), (64, 8, "bf16"),
                                       (100, 8, "f32"), (128, 16, "bf16"), (250, 8, "bf16"),
                                       (250, 20, "f32")])
def test_route_gradient_of_many_tokens(dev, E, K, dtype, renorm):
    """More tokens than a grid takes at once (8 CTAs an SM of 8 warps, up to 4 tokens each):
    the choices of the second round are read during the first."""
    from demand_side_expert_gb300 import Router

    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    T = sms * 8 * 32 + 2003
    gen = torch.Generator(device=dev).manual_seed(E)
    x = (2 * torch.randn(T, E, generator=gen, device=dev)).to(DT[dtype])
    mask = torch.rand(T, generator=gen, device=dev) < 0.9
    da = torch.randn(T, K, generator=gen, device=dev)
    dl = torch.tensor([1.5, -0.5], device=dev)
    c_b, c_z = 50.0, 200.0
    r = Router(T, E, K, dtype, renorm=renorm, balance_coef=c_b, z_coef=c_z)
    r.route(x, mask=mask)
    r.backward(x, da, mask=mask, dloss=dl)
    x64 = x.double()
    idx = x64.sort(dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(r.topk_idx.long(), idx)
    lse = x64.logsumexp(1)
    p = (x64 - lse[:, None]).exp()
    n = int(mask.sum())
    counts = torch.zeros(E, dtype=torch.int64, device=dev)
    counts.scatter_add_(0, idx[mask].reshape(-1), torch.ones(n * K, dtype=torch.int64, device=dev))
    assert torch.equal(r.counts.long(), counts)
    cost = 1.5 * c_b * E * counts.double() / (n * n * K)
    chosen, d64 = p.gather(1, idx), da.double()
    want = p * (cost - (p * cost).sum(1, keepdim=True)) - (p * c_z * lse[:, None] / n)
    a = torch.zeros_like(p)
    if renorm:
        w = chosen / chosen.sum(1, keepdim=True)
        own = w * (d64 - (w * d64).sum(1, keepdim=True))
        a.scatter_(1, idx, w)
    else:
        dp = torch.zeros_like(p).scatter_(1, idx, d64)
        want, own = want + p * (dp - (p * dp).sum(1, keepdim=True)), torch.zeros_like(d64)
    want = want.scatter_add(1, idx, own) * mask[:, None]
    # p and the weights: their exponential at a distance of up to `span` (2 span u), E terms
    # of the sum; they multiply dalpha, its mean, the cost, its mean and lse
    span = (x64.max() - x64.min()).item()
    tol = (2 * span + E + 16) * U
    scale = 2 * d64.abs().amax(1) + 2 * cost.max() + c_z / n * (lse.abs() + 1)
    lim = (3 * tol + (K + E + 16) * U) * torch.maximum(a, p) * scale[:, None]
    if dtype == "bf16":
        lim = lim + 2.0 ** -8 * want.abs()
    within(r.dlogits, want, lim + 1e-37, "dlogits")


@pytest.mark.parametrize("T,E,K,dtype", [(9001, 400, 6, "bf16"), (9001, 512, 4, "bf16"),
                                         (5003, 320, 8, "bf16"), (9001, 512, 4, "f32"),
                                         (9001, 1000, 8, "bf16")])
def test_route_statistics_in_much_shared_memory(dev, T, E, K, dtype):
    """Statistics of 311 to 512 experts and thousands of bfloat16 tokens are the ones whose
    sums take more shared memory than a kernel has unasked; and those beside them."""
    from demand_side_expert_gb300 import Router

    gen = torch.Generator(device=dev).manual_seed(E)
    x = torch.randn(T, E, generator=gen, device=dev).to(DT[dtype])
    r = Router(T, E, K, dtype, balance_coef=0.3, z_coef=0.2)
    r.route(x)
    x64 = x.double()
    idx = x64.sort(dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(r.topk_idx.long(), idx)
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    assert torch.equal(r.counts.long(), counts)
    lse = x64.logsumexp(1)
    p = (x64 - lse[:, None]).exp()
    tol = (2 * (x64.max() - x64.min()).item() + E + 16) * U
    within(r.alpha, p.gather(1, idx), 2 * tol * p.gather(1, idx), "alpha")
    prob = p.sum(0)
    within(r.prob_sum, prob, (tol + (T + 8) * U) * prob, "prob_sum")
    loss = torch.stack([0.3 * E / (T * T * K) * (counts * prob).sum(), 0.2 * lse.square().mean()])
    within(r.loss, loss, (2 * tol + (T + E + 16) * U) * loss, "loss")


def test_router_through_the_c_names(dev):
    """lrm_route and lrm_route_bwd of the binding on the caller's buffers give Router's."""
    from demand_side_expert_gb300 import Router, lrm

    T, E, K = 300, 24, 3
    x = torch.randn(T, E, device=dev)
    mask = (torch.arange(T, device=dev) % 5 != 0).to(torch.uint8)
    da = torch.randn(T, K, device=dev)
    r = Router(T, E, K, "f32", renorm=True, balance_coef=0.5, z_coef=0.25)
    r.route(x, mask=mask)
    r.backward(x, da, mask=mask)
    desc = lrm.lrm_router(T, E, K, lrm.LRM_F32, E, 1, 0.5, 0.25)
    size = lrm.lrm_router_workspace_bytes(desc)
    ws = torch.zeros(size, dtype=torch.uint8, device=dev)
    idx, counts = (torch.empty(n, dtype=torch.int32, device=dev) for n in ((T, K), (E,)))
    alpha, prob, loss, dx = (torch.empty(n, device=dev) for n in ((T, K), (E,), (2,), (T, E)))
    lrm.lrm_route(desc, x, mask, idx, alpha, counts, prob, loss, ws, size)
    lrm.lrm_route_bwd(desc, x, mask, idx, counts, da, None, dx, ws, size)
    for got, name in ((idx, "topk_idx"), (alpha, "alpha"), (counts, "counts"),
                      (prob, "prob_sum"), (loss, "loss"), (dx, "dlogits")):
        assert torch.equal(got, getattr(r, name)), name
    assert lrm.lrm_get_device_error(ws, size) == 0


# -- AdamW: more tensors than a launch describes ---------------------------------------
@pytest.mark.parametrize("state", ["f32", "f8"])
def test_adamw_of_many_tensors_of_mixed_kinds(dev, state):
    """600 tensors of one kind are three launches; with another 40 of other types between
    them each is stepped once, from its own place, like the same tensor alone."""
    from demand_side_expert_gb300 import AdamW

    gen = torch.Generator(device=dev).manual_seed(0)
    params, grads = [], []
    for i in range(640):
        n = int(torch.randint(1, 700, (1,), generator=gen, device=dev))
        p = torch.randn(n, generator=gen, device=dev)
        g = torch.randn(n, generator=gen, device=dev)
        if i % 16 == 7:
            p, g = p.to(torch.bfloat16), (g if i % 32 == 7 else g.to(torch.bfloat16))
        params.append(p)
        grads.append(g)
    alone = [p.clone() for p in params]
    decay = [0.1 * (i % 3) for i in range(640)]
    kw = dict(lr=1e-2, betas=(0.9, 0.95), state=state, master=True)
    opt = AdamW(params, grads, weight_decay=decay, **kw)
    for _ in range(2):
        opt.step()
    for i, (p, g) in enumerate(zip(alone, grads)):
        one = AdamW([p], [g], weight_decay=decay[i], **kw)
        for _ in range(2):
            one.step()
        assert torch.equal(p, params[i]), i
        for name in ("m", "v"):
            got, want = getattr(opt, name), getattr(one, name)[:p.numel()]
            got = got[opt.starts[i]:opt.starts[i] + p.numel()]
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), (i, name)
