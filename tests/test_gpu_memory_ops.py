"""GPU tests of the operators for training under tight memory (grouped router, saved
state in 8 bits, norms around a block) against the float64 oracle.

u = 2^-24 is the unit rounding of float32; every tolerance below counts the roundings of
the longest chain that the operation needs, whatever order a kernel takes: a sum of n
terms is off by at most n u times the sum of their magnitudes. A bfloat16 result is off
by half a step more, 2^-8 of its value.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import memory_oracle as mo
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 1e-37  # below float32's normal numbers


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    from demand_side_expert_gb300 import lrm  # noqa: F401  (liblrm.so must load)
    return torch.device("cuda:0")


def to64(t):
    return t.detach().cpu().double().numpy()


def codes(t):
    return t.view(torch.uint8)


def close(got, ref, lim, name):
    """|got - ref| <= lim elementwise, NaN and infinities at the same places."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), name
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), name
    fine = np.isfinite(ref)
    err = np.abs(got[fine] - ref[fine])
    over = err > np.broadcast_to(lim, ref.shape)[fine]
    assert not over.any(), f"{name}: {int(over.sum())} values off, worst {err.max():.3e}"


# -- router -------------------------------------------------------------------
def make_logits(T, E, dtype, seed, off=0.0, kind="normal"):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=gen) * 1.5
    if kind == "equal":
        x = (x * 2).round() / 2  # many ties
    if kind == "near":
        x = 1 + torch.randint(0, 300, (T, E), generator=gen) * 2.0 ** -23
        x = torch.where(torch.rand(T, E, generator=gen) < 0.3, x, -x)
    if kind == "one":
        x = torch.full((T, E), 0.25)
    if kind == "low":
        x = x * 4 - 95
    if kind == "high":
        x = x * 4 + 30
    if off:
        x = x.masked_fill(torch.rand(T, E, generator=gen) < off, -math.inf)
    return x.to(DT[dtype])


def make_bias(E, kind, seed=0):
    if kind is None:
        return None
    gen = torch.Generator().manual_seed(seed)
    if kind == "zero":
        return torch.zeros(E)
    if kind == "steps":  # what steps of one size add up to
        return torch.randint(-60, 61, (E,), generator=gen) * 1e-3
    return torch.randn(E, generator=gen) * 0.3


def score_tol(x):
    """Relative error of a score or a share: exp of a difference of size s is off by 2 s u
    (its rounding and the base's) and a few ulp, the sum of E positive terms by E u."""
    x = np.where(np.isfinite(x), x, 0.0)
    span = np.abs(x).max() + x.max() - x.min() if x.size else 0.0
    return (2 * span + x.shape[1] + 24) * U


def router(T, E, K, dtype, **kw):
    from demand_side_expert_gb300 import GroupRouter

    return GroupRouter(T, E, K, dtype, **kw)


def check_router(dev, x, K, fn, bias, groups, top, gt, renorm, mask=None, seed=0, balance=0.3):
    """Choices, weights, statistics and gradient of one router against the oracle."""
    T, E = x.shape
    dtype = "bf16" if x.dtype is torch.bfloat16 else "f32"
    r = router(T, E, K, dtype, score=fn, groups=groups, top_groups=top, group_top=gt,
               renorm=renorm, scale=1.7, balance_coef=balance)
    b = None if bias is None else bias.to(dev)
    m = None if mask is None else torch.as_tensor(mask, dtype=torch.uint8, device=dev)
    r.route(x.to(dev), bias=b, mask=m)
    x64 = to64(x)
    kw = dict(fn=fn, renorm=renorm, scale=1.7, balance_coef=balance, mask=mask)
    ref = mo.group_route(x64, K, bias=None if bias is None else to64(bias), groups=groups,
                         top_groups=top, group_top=gt, **kw)
    assert np.array_equal(r.topk_idx.cpu().numpy(), ref["topk_idx"])
    tol = score_tol(x64)
    close(to64(r.alpha), ref["alpha"], (2 * tol + K * U) * np.abs(ref["alpha"]) + TINY, "alpha")
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    close(to64(r.prob_sum), ref["prob_sum"], (tol + (T + 8) * U) * ref["prob_sum"] + TINY,
          "prob_sum")
    close(to64(r.loss), ref["loss"], (2 * tol + (T + E + 16) * U) * ref["loss"], "loss")
    serve = router(T, E, K, dtype, score=fn, groups=groups, top_groups=top, group_top=gt,
                   renorm=renorm, scale=1.7)
    serve.route(x.to(dev), bias=b, mask=m, stats=False)
    assert torch.equal(serve.topk_idx, r.topk_idx) and torch.equal(serve.alpha, r.alpha)

    rng = np.random.default_rng(seed)
    da = rng.standard_normal((T, K)).astype(np.float32)
    r.backward(x.to(dev), torch.from_numpy(da).to(dev), mask=m,
               dloss=torch.tensor([1.5], device=dev))
    assert r.device_error() == 0
    want = mo.group_route_bwd(x64, ref["topk_idx"], ref["counts"], da, 1.5, **kw)
    # scores, shares and 1 - s carry tol; they multiply dalpha, its mean (K terms), the
    # balance cost and its mean (E terms)
    n = max(1, int(ref["use"].sum()))
    cost = 1.5 * balance * E * ref["counts"].max() / (n * n * K) if T else 0
    own = np.zeros((T, E))
    np.put_along_axis(own, ref["topk_idx"].astype(np.int64), np.abs(ref["alpha"]), 1)
    if fn == "softmax" and not renorm:
        own = np.maximum(own, 1.7 * ref["s"])
    mag = own * 2 * np.abs(da).max(1)[:, None] * (1.7 if renorm else 1) + ref["share"] * 2 * cost
    lim = (4 * tol + (K + E + 24) * U) * mag
    if dtype == "bf16":
        lim = lim + BF16 * np.abs(want)
    close(to64(r.dlogits), want, lim + TINY, "dlogits")
    return r, ref


SHAPES = [  # T, E, K, groups, top_groups, group_top, dtype
    (1, 1, 1, 1, 1, 2, "f32"), (1, 256, 8, 8, 4, 2, "bf16"), (5, 8, 3, 4, 2, 2, "f32"),
    (33, 31, 5, 1, 1, 1, "bf16"), (70, 60, 8, 5, 2, 2, "f32"), (130, 64, 8, 16, 5, 1, "bf16"),
    (257, 128, 8, 4, 2, 2, "f32"), (100, 100, 7, 4, 3, 2, "bf16"), (600, 256, 8, 8, 4, 2, "f32"),
    (65, 320, 6, 8, 3, 2, "f32"), (40, 512, 16, 32, 7, 2, "bf16"), (37, 992, 32, 31, 4, 2, "f32"),
    (50, 1024, 8, 8, 2, 1, "bf16"), (90, 96, 4, 2, 1, 2, "f32")]


@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [None, "zero", "steps", "random"])
@pytest.mark.parametrize("T,E,K,groups,top,gt,dtype", SHAPES)
def test_router(dev, T, E, K, groups, top, gt, dtype, bias, fn):
    x = make_logits(T, E, dtype, T + E, off=0.2 if E % 3 == 0 else 0.0,
                    kind="equal" if E % 2 == 0 else "normal")
    rng = np.random.default_rng(E)
    mask = (rng.random(T) < 0.8).astype(np.uint8) if T > 2 else None
    if T > 4:
        x[2] = -math.inf  # nothing to choose from
        x[3, 1:] = -math.inf  # one open expert
    check_router(dev, x, K, fn, make_bias(E, bias, E), groups, top, gt, bias != "steps", mask)


# not: a bias on sigmoids of 1 but for 64 bits' last place, where the larger one of two is a
# matter of the formula's own rounding
HARD = [(b, k, f) for b in (None, "zero", "steps")
        for k in ("equal", "near", "one", "low", "high") for f in ("sigmoid", "softmax")
        if not (b and k == "high" and f == "sigmoid")]


@pytest.mark.parametrize("bias,kind,fn", HARD)
def test_router_hard_choices(dev, bias, kind, fn):
    """Logits that 32 bits cannot rank: equal ones, ones that differ in the last bits, one
    value everywhere, scores near 0 and near 1."""
    for dtype in ("f32", "bf16"):
        x = make_logits(200, 256, dtype, 3, kind=kind)
        check_router(dev, x, 8, fn, make_bias(256, bias), 8, 4, 2, True)


MANY = [(5000, 256, 8, 8, 4, "f32"), (4099, 128, 6, 4, 2, "bf16"), (6001, 64, 2, 8, 3, "f32"),
        (5000, 32, 4, 4, 4, "bf16"), (3500, 160, 8, 5, 3, "f32"), (5000, 16, 1, 2, 1, "bf16"),
        (4000, 256, 8, 1, 1, "bf16"), (4001, 200, 4, 8, 4, "f32"), (3100, 256, 8, 16, 8, "f32")]


@pytest.mark.parametrize("kind", ["normal", "equal", "near", "closed"])
@pytest.mark.parametrize("T,E,K,groups,top,dtype", MANY)
def test_router_many_tokens(dev, T, E, K, groups, top, dtype, kind):
    """Enough tokens that they share warps."""
    x = make_logits(T, E, dtype, E, off=0.9 if kind == "closed" else 0.0, kind=kind)
    bias = make_bias(E, "steps" if T % 2 else "zero")
    check_router(dev, x, K, "sigmoid" if E > 100 else "softmax", bias, groups, top, 2, True)


def test_router_gradient_matches_differences(dev):
    """The kernel's own gradient against central differences of the float64 loss."""
    T, E, K = 4, 12, 3
    x = make_logits(T, E, "f32", 5)
    da = np.random.default_rng(0).standard_normal((T, K))
    for fn in ("sigmoid", "softmax"):
        for renorm in (False, True):
            r = router(T, E, K, "f32", score=fn, groups=3, top_groups=2, renorm=renorm, scale=2.0,
                       balance_coef=0.4)
            r.route(x.to(dev))
            r.backward(x.to(dev), torch.from_numpy(da).float().to(dev))
            idx, x64 = r.topk_idx.cpu().numpy(), to64(x)
            da32 = da.astype(np.float32).astype(np.float64)

            def total(v):
                q = mo.group_route(v, K, fn, renorm=renorm, scale=2.0, balance_coef=0.4, idx=idx)
                return (q["alpha"] * da32).sum() + q["loss"].sum()

            for t in range(T):
                for e in range(E):
                    d = np.zeros_like(x64)
                    d[t, e] = 1e-5
                    fd = (total(x64 + d) - total(x64 - d)) / 2e-5
                    assert abs(fd - r.dlogits[t, e].item()) < 1e-5


def test_router_nan_and_inf(dev):
    """NaN and +inf reach the outputs of the tokens that take part, and only those; every
    row's ids are valid, distinct and of the kept groups."""
    clean = make_logits(6, 16, "f32", 3)
    dirty = clean.clone()
    dirty[1, 3], dirty[4] = math.nan, math.nan
    mask = torch.tensor([1, 0, 1, 1, 0, 1], dtype=torch.uint8, device=dev)
    for fn in ("sigmoid", "softmax"):
        got = []
        for x in (clean, dirty):
            r = router(6, 16, 3, "f32", score=fn, groups=4, top_groups=2, balance_coef=1.0)
            r.route(x.to(dev), mask=mask)
            da = torch.ones(6, 3, device=dev)
            da[1] = math.nan
            r.backward(x.to(dev), da, mask=mask)
            assert torch.isfinite(r.dlogits).all() and (r.dlogits[[1, 4]] == 0).all()
            got.append(r)
            idx = r.topk_idx.cpu().numpy()
            assert all(len(set(row)) == 3 and row.min() >= 0 and row.max() < 16 and
                       len({e // 4 for e in row}) <= 2 for row in idx)
        for name in ("alpha", "counts", "prob_sum", "loss"):
            assert torch.equal(getattr(got[0], name), getattr(got[1], name)), (fn, name)
        r.route(dirty.to(dev))
        assert torch.isnan(r.prob_sum).any() and torch.isnan(r.loss).all()
        assert torch.isfinite(r.alpha[[0, 2, 3, 5]]).all()
        if fn == "softmax":
            assert torch.isnan(r.alpha[[1, 4]]).all()
        else:  # NaN comes last: three numbers are there to choose, its own token has none
            assert torch.isfinite(r.alpha[1]).all() and 3 not in r.topk_idx[1].tolist()
            assert torch.isnan(r.alpha[4]).all()
    x = clean.clone()
    x[0, 5] = math.inf
    r = router(6, 16, 3, "f32", score="sigmoid", renorm=False)
    r.route(x.to(dev))
    assert r.topk_idx[0, 0].item() == 5 and r.alpha[0, 0].item() == 1.0
    assert torch.isfinite(r.prob_sum).all()


def test_router_no_tokens_all_masked_and_bad_ids(dev):
    from demand_side_expert_gb300 import lrm

    r = router(0, 8, 2, "f32", balance_coef=1.0)
    r.counts.fill_(7)
    x = torch.empty(0, 8, device=dev)
    r.route(x)
    assert (r.counts == 0).all() and (r.prob_sum == 0).all() and (r.loss == 0).all()
    r.route(x, stats=False)
    r.backward(x)
    x = make_logits(300, 8, "f32", 0).to(dev)
    s = router(300, 8, 2, "f32", balance_coef=1.0)
    mask = torch.zeros(300, dtype=torch.bool, device=dev)
    s.route(x, mask=mask)
    assert (s.alpha == 0).all() and (s.counts == 0).all() and (s.loss == 0).all()
    s.backward(x, torch.ones(300, 2, device=dev), mask=mask)
    assert (s.dlogits == 0).all()
    s.route(x)
    s.topk_idx[1, 0], s.topk_idx[3, 1] = 8, -1
    s.backward(x, torch.ones(300, 2, device=dev))
    assert s.device_error() == lrm.LRM_DEVERR_EXPERT_ID
    assert torch.isfinite(s.dlogits).all()


def test_router_strides_and_mask_types(dev):
    T, E, K = 70, 40, 4
    wide = make_logits(T, 3 * E + 1, "bf16", 1).to(dev)
    x = wide[:, 16:16 + E]
    mask = torch.arange(T, device=dev) % 3 != 0
    bias = make_bias(E, "steps").to(dev)
    a, b = (router(T, E, K, "bf16", groups=4, top_groups=2, balance_coef=0.1) for _ in range(2))
    a.route(x, bias=bias, mask=mask)
    b.route(x.contiguous(), bias=bias, mask=mask.to(torch.uint8))
    a.backward(x, a.alpha, mask=mask)
    b.backward(x.contiguous(), b.alpha, mask=mask)
    for name in ("topk_idx", "alpha", "counts", "prob_sum", "loss", "dlogits"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("E,groups", [(256, 8), (128, 4), (64, 4), (200, 5)])
def test_router_strided_rows_of_many_tokens(dev, E, groups):
    """Odd strides and offsets where tokens share warps: the contiguous rows' bits."""
    T, K = 17001, 8
    wide = make_logits(T, E + 9, "f32", E).to(dev)
    x = wide[:, 4:4 + E]
    bias = make_bias(E, "steps").to(dev)
    a, b = (router(T, E, K, "f32", groups=groups, top_groups=2, balance_coef=0.1)
            for _ in range(2))
    for r, v in ((a, x), (b, x.contiguous())):
        r.route(v, bias=bias)
        r.backward(v, r.alpha)
    for name in ("topk_idx", "alpha", "counts", "prob_sum", "loss", "dlogits"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_router_weights_do_not_depend_on_the_block(dev):
    """The same tokens alone, among a few and among many (three kernels): the same choices,
    weights to the last bits, also where scores are below float32's normal numbers."""
    E, K = 256, 8
    for renorm in (False, True):
        for kind in ("normal", "low"):
            x = make_logits(20000, E, "f32", 2, kind=kind).to(dev)
            bias = make_bias(E, "steps").to(dev)
            got = []
            for T in (20000, 5000, 200, 1):
                r = router(T, E, K, "f32", groups=8, top_groups=4, renorm=renorm)
                r.route(x[:T], bias=bias, stats=False)
                got.append(r)
            for r in got[1:]:
                n = r.T
                assert torch.equal(r.topk_idx, got[0].topk_idx[:n])
                a, b = to64(r.alpha), to64(got[0].alpha[:n])
                # a dozen roundings, or two steps of the smallest number
                close(a, b, 32 * U * np.abs(b) + 2 ** -147.0, "alpha")


def test_bias_steps_even_the_loads(dev):
    """The step is the formula's, bit for bit, in place as well; many of them even out
    what the experts get."""
    T, E, K = 4096, 64, 4
    x = make_logits(T, E, "f32", 1)
    x[:, :8] += 2  # eight experts that every token likes
    x = x.to(dev)
    r = router(T, E, K, "f32")
    bias = make_bias(E, "random").to(dev)
    r.route(x, bias=bias)
    want = mo.bias_step(to64(bias), r.counts.cpu().numpy(), 1e-3)
    got = r.next_bias(bias, 1e-3)
    close(to64(got), want, 2 * U * (np.abs(want) + 1e-3), "bias")
    r.next_bias(bias, 1e-3, out=bias)
    assert torch.equal(bias, got)
    bias.zero_()
    r.route(x, bias=bias)
    first = r.counts.max().item()
    for _ in range(200):
        r.next_bias(bias, 2e-3, out=bias)
        r.route(x, bias=bias)
    assert r.counts.max().item() < 0.5 * first and r.counts.sum().item() == T * K


def test_router_repeats_and_in_a_graph(dev):
    """Statistics do not depend on the order in which CTAs arrive; captured calls replay on
    new logits, beside an eager router's; calls on a stream of their own."""
    T, E, K = 20000, 256, 8
    x = make_logits(T, E, "f32", 0).to(dev)
    bias = make_bias(E, "steps").to(dev)
    r = router(T, E, K, "f32", groups=8, top_groups=4, balance_coef=0.1)
    names = ("topk_idx", "alpha", "counts", "prob_sum", "loss", "dlogits")

    def once(q, v, stream=None):
        q.route(v, bias=bias, stream=stream)
        q.backward(v, q.alpha, stream=stream)

    once(r, x)
    first = [getattr(r, n).clone() for n in names]
    for _ in range(5):
        once(r, x)
        assert all(torch.equal(a, getattr(r, n)) for a, n in zip(first, names))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        s = router(T, E, K, "f32", groups=8, top_groups=4, balance_coef=0.1)
        torch.cuda.synchronize()
        once(s, x, stream)
        side.synchronize()
        assert all(torch.equal(a, getattr(s, n)) for a, n in zip(first, names))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            once(r, held)
            r.next_bias(bias, 1e-3)
    held.copy_(make_logits(T, E, "f32", 1))
    graph.replay()
    torch.cuda.synchronize()
    got = [getattr(r, n).clone() for n in names]
    once(r, held)
    assert all(torch.equal(a, getattr(r, n)) for a, n in zip(got, names))
    assert not torch.equal(got[3], first[3])


def test_router_past_2_31_elements(dev):
    """Rows of logits whose offsets need 64 bits, forward and backward."""
    T, E, K = (1 << 21) + 77, 1024, 4
    x = torch.empty(T, E, dtype=torch.bfloat16, device=dev).normal_()
    r = router(T, E, K, "bf16", groups=8, top_groups=4)
    r.route(x)
    da = torch.ones(T, K, device=dev)
    da[:, 1] = -1
    r.backward(x, da)
    assert r.counts.sum().item() == T * K
    tail = to64(x[-5:])
    ref = mo.group_route(tail, K, groups=8, top_groups=4)
    assert np.array_equal(r.topk_idx[-5:].cpu().numpy(), ref["topk_idx"])
    tol = score_tol(tail)
    close(to64(r.alpha[-5:]), ref["alpha"], 2 * tol * ref["alpha"], "alpha")
    want = mo.group_route_bwd(tail, ref["topk_idx"], ref["counts"], to64(da[-5:]))
    close(to64(r.dlogits[-5:]), want, 4 * tol * 2 + BF16 * np.abs(want), "dlogits")


# -- saved state in 8 bits --------------------------------------------------------
def make_ab(N, H, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + H)
    ab = torch.randn(N, 2 * H, generator=gen) * torch.exp(torch.randn(N, 1, generator=gen))
    return ab.to(DT[dtype])


def phi_tol(a):
    """Relative error of SiLU(a) b: exp and reciprocal on the hardware, 2 |a| u for the
    exponent's rounding, and a few ulp."""
    return (2 * np.abs(a) + 12) * U


STATES = [  # T, K, H, cols, dtype
    (1, 1, 8, 32, "f32"), (1, 8, 64, 64, "bf16"), (5, 2, 72, 32, "bf16"), (33, 3, 192, 128, "bf16"),
    (130, 8, 512, 64, "bf16"), (77, 4, 768, 128, "bf16"), (20, 8, 1408, 128, "bf16"),
    (9, 1, 1544, 32, "f32"), (65, 2, 264, 128, "f32"), (3, 2, 2056, 64, "bf16"),
    (1000, 8, 256, 128, "bf16"), (65, 2, 24, 128, "bf16"), (9, 3, 128, 32, "bf16"),
    (7, 5, 40, 64, "f32"), (11, 3, 64, 128, "f32"), (50, 1, 120, 64, "bf16"), (6, 2, 904, 64, "bf16")]


@pytest.mark.parametrize("T,K,H,cols,dtype", STATES)
def test_pack(dev, T, K, H, cols, dtype):
    from demand_side_expert_gb300 import PackedState

    ab = make_ab(T * K, H, dtype)
    p = PackedState(T, K, H, dtype, cols=cols)
    p.pack(ab.to(dev))
    q, scale, sq = mo.pack(to64(ab), cols)
    # amax / 448, one rounding and the inverse's
    close(to64(p.scale), scale, 2 * U * scale, "scale")
    got = to64(p.q.float())
    if dtype == "bf16":  # quotients of 8-bit values: no rounding but the code's own
        assert np.array_equal(got, q)
    else:
        G = scale.shape[1] // 2
        wide = np.concatenate([np.repeat(scale[:, :G], cols, 1)[:, :H],
                               np.repeat(scale[:, G:], cols, 1)[:, :H]], 1)
        ratio = to64(ab) / wide
        # half a step of the code, with what the quotient itself may be off by
        half = np.maximum(np.abs(ratio) * 2.0 ** -4, 2.0 ** -10)
        close(got, ratio, half + 4 * U * np.abs(ratio), "q")
    a, b = to64(ab)[:, :H], to64(ab)[:, H:]
    f = mo.phi(a, b) ** 2
    close(to64(p.phi_sq), sq, (f * 2 * phi_tol(a)).sum(1) + (H + 4) * U * sq + TINY, "phi_sq")


def test_pack_zero_nan_inf_and_lowest(dev):
    """Zero rows, NaN and infinities stay in their group; the type's largest and smallest
    values neither overflow a quotient nor lose their scale."""
    from demand_side_expert_gb300 import PackedState

    H = 128
    for dtype in ("f32", "bf16"):
        ab = make_ab(8, H, dtype)
        ab[0] = 0
        ab[1, 3] = math.nan
        ab[2, 70] = math.inf
        big = torch.finfo(DT[dtype]).max
        ab[3, :64] = torch.linspace(-1, 1, 64).to(DT[dtype]) * big
        ab[4] = ab[4].float().mul(1e-38).to(DT[dtype])
        p = PackedState(4, 2, H, dtype, cols=64)
        p.pack(ab.to(dev))
        q, scale = to64(p.q.float()), to64(p.scale)
        assert (q[0] == 0).all() and (scale[0] > 0).all() and p.phi_sq[0].item() == 0
        assert np.isnan(q[1, 3]) and np.isfinite(np.delete(q[1], 3)).all()
        assert np.isfinite(scale[1]).all() and math.isnan(p.phi_sq[1].item())
        assert np.isinf(scale[2, 1]) and np.isfinite(scale[2, [0, 2, 3]]).all()
        assert np.isfinite(q[2, :64]).all() and np.isfinite(q[2, 128:]).all()
        want, ws, _ = mo.pack(to64(ab[[3, 4]]), 64)
        close(scale[[3, 4]], ws, 2 * U * ws, "scale")
        half = np.maximum(np.abs(want) * 2.0 ** -3, 2.0 ** -9)  # a step: a tie may go either way
        close(q[[3, 4]], want, half, "q")
        clean = make_ab(8, H, dtype)
        p2 = PackedState(4, 2, H, dtype, cols=64)
        p2.pack(clean.to(dev))
        assert torch.equal(codes(p.q)[5:], codes(p2.q)[5:]) and torch.equal(p.phi_sq[5:],
                                                                            p2.phi_sq[5:])


def layer_case(T, D, H, E, K, dtype, seed=0):
    from workloads import generate, get_config

    cfg = get_config("qwen3-30b-a3b-t4k", T=T, D=D, H=H, E=E, K=K, dtype=dtype)
    return generate(cfg, device="cpu", seed=seed)


def norm8(x, cols):
    """8-bit rows with their scales, as the norms write them."""
    q, s = mo.quantise_rows(to64(x), cols)
    return torch.from_numpy(q).to(torch.float8_e4m3fn), torch.from_numpy(s).float()


@pytest.mark.parametrize("x8", [None, 0, 64, 128])
@pytest.mark.parametrize("T,D,H,E,K,dtype,rate", [
    (256, 256, 192, 8, 2, "bf16", (1, 2)), (130, 320, 64, 24, 3, "bf16", (1, 1)),
    (64, 32, 16, 8, 2, "f32", (3, 5)), (1, 64, 64, 4, 1, "bf16", (1, 1)),
    (200, 128, 128, 16, 8, "bf16", (1, 4)), (65, 64, 64, 8, 2, "bf16", (0, 1))])
def test_step_from_packed_state(dev, T, D, H, E, K, dtype, rate, x8):
    """The whole backward from the 8-bit state: scores of the exact state, rows rebuilt from
    the codes, gradients of the rebuilt rows."""
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward

    import parity_util as pu

    inp = layer_case(T, D, H, E, K, dtype)
    d = {k: (v.to(dev) if torch.is_tensor(v) else v) for k, v in inp.items()}
    pipe = RecalibratedExpertBackward(T, D, H, E, K, dtype, dev)
    pipe.dispatch(d["topk_idx"])
    perm, inv, counts, off = oracle.dispatch_permute(inp["topk_idx"].numpy(), E)
    ab = pipe.to_dispatch_order(d["ab_pair"])
    cols = 64 if H % 128 else 128
    state = PackedState(T, K, H, dtype, cols=cols)
    state.pack(ab)
    x, x_np = d["x"], to64(inp["x"])
    if x8 is not None:
        q, s = norm8(inp["x"], x8)
        x, x_np = (q.to(dev), s.to(dev)), mo.decode(to64(q.float()), to64(s), x8)
    args = (d["topk_idx"], d["alpha"], x, d["g"], state, None, d["w_gate"], d["w_up"], d["w_down"])
    N, fill = T * K, 7.0
    for name in ("dy_c", "ab_c", "phi_c", "x_c"):
        getattr(pipe, name).fill_(fill)
    pipe.step(*args, rate=rate)
    torch.cuda.synchronize()
    assert pipe.device_error() == 0

    a64, g64, alpha = to64(ab), to64(inp["g"]), to64(inp["alpha"]).reshape(-1)
    f = mo.phi(a64[:, :H], a64[:, H:])
    score = alpha[perm] ** 2 * (g64 ** 2).sum(1)[perm // K] * (f ** 2).sum(1)
    pu.check_scores(pu.to_np(pipe.score)[:N], score)
    quota = oracle.quota_from_rate(counts, *rate)
    keep, sel_off, sel_pos = pu.check_selection(pipe, perm, off, quota)
    M = int(sel_off[-1])
    state_ab, state_phi = mo.unpack(to64(state.q.float()), to64(state.scale), cols)
    c = oracle.compact(perm, sel_off, sel_pos, to64(inp["alpha"]), x_np, g64, state_ab, state_phi, K)
    assert np.array_equal(pu.to_np(pipe.tok_c)[:M], c["tok_c"])
    assert np.array_equal(pu.to_np(pipe.row_of_pos)[:N], c["row_of_pos"])
    # one product (or the chain of phi) in float32 and one rounding to the layer's type
    half = BF16 if dtype == "bf16" else 0.0
    fa = np.abs(state_ab[sel_pos][:, :H])
    for name, tol in (("dy_c", 2 * U), ("ab_c", 2 * U), ("x_c", 2 * U), ("phi_c", phi_tol(fa))):
        close(to64(getattr(pipe, name))[:M], c[name], (half + tol) * np.abs(c[name]) + TINY, name)
    # rows behind the retained ones are left as they were, but for the zeros behind dy_c
    pad = min(M + 64, N)
    assert (pipe.dy_c[M:pad] == 0).all() and (pipe.dy_c[pad:] == fill).all()
    for name in ("ab_c", "phi_c", "x_c"):
        assert (getattr(pipe, name)[M:] == fill).all(), name
    inp_np = {k: pu.to_np(v) if torch.is_tensor(v) else v for k, v in inp.items()}
    pu.check_backward(pipe, inp_np, c, sel_off, inv, T, K, dtype)
    if x8 is None:  # x read in place: the same rows in the same order
        first = [getattr(pipe, n).clone() for n in ("dw_gate", "dw_up", "dw_down", "dx")]
        pipe.x_c.fill_(fill)
        pipe.step(*args, rate=rate, gathered=True)
        torch.cuda.synchronize()
        for a, n in zip(first, ("dw_gate", "dw_up", "dw_down", "dx")):
            assert torch.equal(a, getattr(pipe, n)), n
        assert (pipe.x_c == fill).all()


@pytest.mark.parametrize("rounds,more", [(1, 0), (1, 1), (2, -1), (2, 0), (3, 0), (3, 7)])
def test_packed_rows_of_many_experts(dev, rounds, more):
    """As many retained rows as the kernel's warps take in whole rounds, a few more or less,
    from many experts of uneven size: every row comes out, whatever its round."""
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward

    warps = torch.cuda.get_device_properties(dev).multi_processor_count * 32
    N, D, H, E = rounds * warps + more, 16, 8, 251
    gen = torch.Generator().manual_seed(rounds)
    ids = (torch.rand(N, 1, generator=gen) ** 2 * E).to(torch.int32).clamp_(max=E - 1)
    pipe = RecalibratedExpertBackward(N, D, H, E, 1, "f32", dev)
    pipe.dispatch(ids.to(dev))
    state = PackedState(N, 1, H, "f32", cols=32)
    state.pack(torch.randn(N, 2 * H, generator=gen).to(dev))
    alpha = torch.rand(N, 1, generator=gen).to(dev)
    g, x = torch.randn(N, D, generator=gen).to(dev), torch.randn(N, D, generator=gen).to(dev)
    pipe.score_pairs(alpha, g, state)
    for rate in ((1, 1), (2, 3)):
        pipe.select_rate(*rate)
        for t in (pipe.dy_c, pipe.x_c, pipe.ab_c, pipe.phi_c):
            t.fill_(math.nan)
        pipe.tok_c.fill_(-5)
        pipe.compact(alpha, x, g, state, None)
        assert pipe.device_error() == 0
        M = pipe.retained_rows
        pos = pipe.sel_pos[:M].long()
        pair = pipe.perm[pos].long()
        assert torch.equal(pipe.tok_c[:M].long(), pair)
        assert torch.equal(pipe.row_of_pos[pos].long(), torch.arange(M, device=dev))
        assert torch.equal(pipe.x_c[:M], x[pair])
        assert torch.equal(pipe.dy_c[:M], alpha[pair] * g[pair])
        wide = state.scale.repeat_interleave(H, 1)
        assert torch.equal(pipe.ab_c[:M], (state.q.float() * wide)[pos])
        assert torch.isfinite(pipe.phi_c[:M]).all()


def _every_row_comes_out(dev, T, K, D, H, E, dtype, seed):
    """compact of random pairs of uneven experts: each retained row is its pair's, bit for bit
    (dy is one rounded product, a and b another)."""
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward

    tdtype = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator().manual_seed(seed)
    ids = (torch.rand(T, E, generator=gen) ** torch.arange(1, E + 1)).topk(K, dim=1)[1]
    pipe = RecalibratedExpertBackward(T, D, H, E, K, dtype, dev)
    pipe.dispatch(ids.to(torch.int32).to(dev))
    state = PackedState(T, K, H, dtype, cols=32)
    state.pack(torch.randn(T * K, 2 * H, generator=gen).to(tdtype).to(dev))
    alpha = torch.rand(T, K, generator=gen).to(dev)
    g = torch.randn(T, D, generator=gen).to(tdtype).to(dev)
    x = torch.randn(T, D, generator=gen).to(tdtype).to(dev)
    pipe.score_pairs(alpha, g, state)
    for rate in ((1, 1), (2, 3)):
        pipe.select_rate(*rate)
        for t in (pipe.dy_c, pipe.x_c, pipe.ab_c, pipe.phi_c):
            t.fill_(math.nan)
        pipe.tok_c.fill_(-5)
        pipe.compact(alpha, x, g, state, None)
        assert pipe.device_error() == 0
        M = pipe.retained_rows
        pos = pipe.sel_pos[:M].long()
        pair = pipe.perm[pos].long()
        tok = pair // K
        assert torch.equal(pipe.tok_c[:M].long(), tok)
        assert torch.equal(pipe.row_of_pos[pos].long(), torch.arange(M, device=dev))
        assert int((pipe.row_of_pos[:T * K] >= 0).sum()) == M
        assert torch.equal(pipe.x_c[:M], x[tok])
        dy = alpha.view(-1)[pair][:, None] * g[tok].float()
        assert torch.equal(pipe.dy_c[:M], dy.to(tdtype))
        wide = state.scale.view(T * K, 2, -1).repeat_interleave(32, 2)[:, :, :H].reshape(T * K, -1)
        assert torch.equal(pipe.ab_c[:M], (state.q.float() * wide)[pos].to(tdtype))
        assert torch.isfinite(pipe.phi_c[:M].float()).all()


@pytest.mark.parametrize("rounds,more", [(2, -1), (2, 0), (2, 1), (3, 0), (3, 7)])
def test_packed_rows_of_wide_tokens(dev, rounds, more):
    """The rows that are met by segments (32 MB of cotangents at least), as many as the warps take
    in whole rounds, a few more or less."""
    warps = torch.cuda.get_device_properties(dev).multi_processor_count * 32
    _every_row_comes_out(dev, rounds * warps + more, 1, 1024, 8, 251, "f32", rounds)
    _every_row_comes_out(dev, rounds * (warps - 60 - 8) + more, 1, 2048, 8, 60, "bf16", rounds)


@pytest.mark.parametrize("T,K,D,H,E,dtype", [
    (1, 1, 8, 8, 1, "bf16"), (5, 3, 24, 40, 7, "f32"),
    (20000, 2, 80, 48, 28, "f32"), (20001, 2, 256, 64, 28, "bf16"),  # eight lanes a row
    (7261, 4, 320, 136, 130, "bf16"), (10001, 2, 256, 256, 9, "f32"),  # sixteen
    (3001, 4, 80, 48, 28, "bf16"), (1200, 4, 80, 48, 28, "f32"),  # more lanes for fewer rows
    (8001, 4, 1032, 264, 17, "bf16"), (3001, 4, 264, 520, 64, "f32"),  # a warp, several rounds
])
def test_packed_rows_of_every_width(dev, T, K, D, H, E, dtype):
    _every_row_comes_out(dev, T, K, D, H, E, dtype, T)


def test_forward_packs_its_state(dev):
    """forward(packed=...) leaves what pack makes of the saved [a | b]; the backward from it
    is near the one from the 16-bit state (e4m3 has 2^-4 of a value, random ones add in
    squares: the gradients of the same rows differ by a few 2^-5)."""
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward

    T, D, H, E, K = 512, 256, 192, 8, 2
    inp = layer_case(T, D, H, E, K, "bf16")
    d = {k: (v.to(dev) if torch.is_tensor(v) else v) for k, v in inp.items()}
    pipe = RecalibratedExpertBackward(T, D, H, E, K, "bf16", dev)
    state, other = PackedState(T, K, H, "bf16"), PackedState(T, K, H, "bf16")
    w = (d["w_gate"], d["w_up"], d["w_down"])
    pipe.forward(d["topk_idx"], d["alpha"], d["x"], *w, packed=state)
    other.pack(pipe.ab)
    assert torch.equal(codes(state.q), codes(other.q)) and torch.equal(state.phi_sq, other.phi_sq)
    args = (d["topk_idx"], d["alpha"], d["x"], d["g"])
    pipe.step(*args, pipe.ab, pipe.phi, *w, rate=(1, 1))
    want = [getattr(pipe, n).clone() for n in ("dw_gate", "dw_up", "dw_down", "dx")]
    pipe.ab.fill_(math.nan)  # the next layer's
    pipe.phi.fill_(math.nan)
    pipe.step(*args, state, None, *w, rate=(1, 1))
    for a, n in zip(want, ("dw_gate", "dw_up", "dw_down", "dx")):
        b = getattr(pipe, n)
        assert ((a - b).norm() / a.norm()).item() < 2.0 ** -3, n


def test_packed_bad_indices_and_no_pairs(dev):
    """Bad indices are skipped and flagged; a layer without tokens does nothing."""
    from demand_side_expert_gb300 import PackedState, lrm

    T, D, H, E, K = 4, 64, 64, 4, 2
    N = T * K
    s = lrm.make_shape(T, D, H, E, K, lrm.LRM_BF16)
    n = lrm.lrm_workspace_bytes(s)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    p = PackedState(T, K, H, "bf16")
    p.pack(make_ab(N, H, "bf16").to(dev))
    g = torch.ones(T, D, dtype=torch.bfloat16, device=dev)
    alpha = torch.ones(T, K, device=dev)
    inv = torch.arange(N, dtype=torch.int32, device=dev)
    score = torch.full((N,), -1.0, device=dev)
    inv[3], inv[5] = N, -7
    lrm.lrm_score_packed(s, p.desc, g, alpha, inv, score, ws, n)
    assert lrm.lrm_get_device_error(ws, n) == lrm.LRM_DEVERR_INDEX
    assert (score[[3, 5]] == -1).all() and (score[[0, 1, 2, 4, 6, 7]] >= 0).all()

    def buffers():
        e = lambda c: torch.full((N, c), 5.0, dtype=torch.bfloat16, device=dev)  # noqa: E731
        i = lambda: torch.full((N,), -9, dtype=torch.int32, device=dev)  # noqa: E731
        return e(D), None, e(2 * H), e(H), i(), i()

    perm = torch.arange(N, dtype=torch.int32, device=dev)
    keep = torch.ones(N, dtype=torch.uint8, device=dev)
    sel_off = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32, device=dev)
    for change in ("pos", "perm", "count"):
        sp, pm, so_ = perm.clone(), perm.clone(), sel_off.clone()
        if change == "pos":
            sp[2] = N + 3
        if change == "perm":
            pm[2] = -1
        if change == "count":
            so_[-1] = 3 * N
        out = buffers()
        lrm.lrm_clear_device_error(ws, n)
        lrm.lrm_compact_packed(s, p.desc, pm, keep, so_, sp, alpha, None, None, 0, g, *out, ws, n)
        assert lrm.lrm_get_device_error(ws, n) == lrm.LRM_DEVERR_INDEX
        if change != "count":
            assert (out[0][2] == 5).all() and (out[4][2] == -9).all() and (out[0][3] == 1).all()
    zero = lrm.make_shape(0, D, H, E, K, lrm.LRM_BF16)
    e = PackedState(0, K, H, "bf16")
    e.pack(torch.empty(0, 2 * H, dtype=torch.bfloat16, device=dev))
    lrm.lrm_score_packed(zero, e.desc, None, None, None, None, ws, n)
    lrm.lrm_compact_packed(zero, e.desc, *[None] * 7, 0, *[None] * 7, ws, n)


def test_pack_past_2_31_elements(dev):
    from demand_side_expert_gb300 import PackedState

    T, K, H = 160000, 8, 1024
    p = PackedState(T, K, H, "bf16")
    ab = torch.empty(T * K, 2 * H, dtype=torch.bfloat16, device=dev).normal_()
    p.pack(ab)
    tail = ab[-3:].cpu()
    q, scale, sq = mo.pack(to64(tail), 128)
    assert np.array_equal(to64(p.q[-3:].float()), q)
    close(to64(p.phi_sq[-3:]), sq, (H + 40) * U * sq, "phi_sq")


def test_packed_calls_on_streams_and_in_a_graph(dev):
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward

    T, D, H, E, K = 256, 128, 64, 8, 2
    inp = layer_case(T, D, H, E, K, "bf16")
    d = {k: (v.to(dev) if torch.is_tensor(v) else v) for k, v in inp.items()}
    w = (d["w_gate"], d["w_up"], d["w_down"])
    names = ("dw_gate", "dw_up", "dw_down", "dx")
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side.cuda_stream):
        pipe = RecalibratedExpertBackward(T, D, H, E, K, "bf16", dev)
        state = PackedState(T, K, H, "bf16")
        torch.cuda.synchronize()
        pipe.forward(d["topk_idx"], d["alpha"], d["x"], *w, stream=stream, packed=state)
        pipe.step(d["topk_idx"], d["alpha"], d["x"], d["g"], state, None, *w, rate=(1, 2),
                  stream=stream, gathered=True)
        torch.cuda.synchronize()
        got.append([getattr(pipe, n).clone() for n in names])
    assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph, held = torch.cuda.CUDAGraph(), d["x"].clone()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            pipe.forward(d["topk_idx"], d["alpha"], held, *w, packed=state)
            pipe.step(d["topk_idx"], d["alpha"], held, d["g"], state, None, *w, rate=(1, 2),
                      gathered=True)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, getattr(pipe, n)) for a, n in zip(got[0], names))
    held.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got[0][0], pipe.dw_gate)


# -- norms around a block ---------------------------------------------------------
NORMS = [  # T, D, dtype, block dtype
    (1, 8, "f32", "f32"), (1, 4096, "bf16", "f32"), (3, 40, "bf16", "bf16"),
    (5, 256, "f32", "f32"), (9, 264, "bf16", "f32"), (130, 512, "f32", "f32"),
    (700, 776, "bf16", "bf16"), (31, 1024, "f32", "f32"), (333, 1032, "bf16", "f32"),
    (64, 2048, "bf16", "f32"), (21, 2056, "f32", "f32"), (11, 4104, "f32", "f32"),
    (6, 8192, "bf16", "f32"), (4, 8192, "f32", "f32"), (2000, 64, "bf16", "bf16"),
    (3000, 1024, "bf16", "f32"), (1500, 2048, "bf16", "bf16"), (900, 4096, "bf16", "f32"),
    (400, 8184, "bf16", "f32")]


def norm_case(T, D, dtype, block, post, kind, seed=0):
    gen = torch.Generator().manual_seed(seed + D)
    dt = DT[dtype]
    v = {"block": (torch.randn(T, D, generator=gen) * 0.5).to(DT[block]),
         "res": (torch.randn(T, D, generator=gen) * 2).to(dt),
         "w": (1 + 0.2 * torch.randn(D, generator=gen)).to(dt), "w_post": None, "gate": None}
    if post:
        v["w_post"] = (1 + 0.2 * torch.randn(D, generator=gen)).to(dt)
    if kind:
        v["gate"] = (0.5 + 0.3 * torch.randn(D if kind == "column" else T, generator=gen)).to(dt)
    return v, gen


def on(dev, v):
    return {k: None if t is None else t.to(dev) for k, t in v.items()}


def run_norm(n, d, **kw):
    n.forward(d["block"], d["res"], d["w"], w_post=d["w_post"], gate=d["gate"], **kw)


def arrays(v):
    return {k: None if t is None else to64(t) for k, t in v.items()}


def check_norm(n, v, kind, q_cols, dtype, scale, eps):
    a = arrays(v)
    D = a["w"].shape[0]
    ref = mo.block_norm(a["block"], a["res"], a["w"], a["w_post"], a["gate"], kind, scale, eps,
                        q_cols)
    # a sum of D squares, a division, a root
    rs = (D + 8) * U
    out = BF16 if dtype == "bf16" else 0.0
    u = np.abs(ref["h"] - scale * a["res"])
    h_lim = (rs + 6 * U) * u + 3 * U * np.abs(scale * a["res"])
    if a["w_post"] is not None:
        close(to64(n.block_rstd), ref["block_rstd"], rs * ref["block_rstd"], "block_rstd")
    # the norm of a row whose values are off by h_lim
    h_rel = np.sqrt((h_lim ** 2).sum(1)) * ref["rstd"] / math.sqrt(D)
    close(to64(n.rstd), ref["rstd"], (rs + h_rel) * ref["rstd"], "rstd")
    close(to64(n.h), ref["h"], out * np.abs(ref["h"]) + h_lim, "h")
    y_lim = (rs + 4 * U + h_rel[:, None]) * np.abs(ref["y"]) + \
        h_lim * ref["rstd"][:, None] * np.abs(a["w"])
    if n.y is not None:
        close(to64(n.y), ref["y"], out * np.abs(ref["y"]) + y_lim, "y")
    if q_cols is not None:
        cols = q_cols or D
        s = to64(n.q_scale)
        top = np.stack([y_lim[:, c:c + cols].max(1) for c in range(0, D, cols)], 1) / so.F8_MAX
        close(s, ref["q_scale"], top + 4 * U * ref["q_scale"], "q_scale")
        wide = np.repeat(s, cols, axis=1)[:, :D]
        # half a step of the code: 2^-4 of a normal value, 2^-10 below
        half = np.maximum(np.abs(ref["y"]) * 2.0 ** -4, wide * 2.0 ** -10)
        close(to64(n.q.float()) * wide, ref["y"], half * (1 + 1e-3) + 4 * y_lim, "q")
    return ref


@pytest.mark.parametrize("kind", [None, "column", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,D,dtype,block", NORMS)
def test_block_norm_forward(dev, T, D, dtype, block, post, kind):
    from demand_side_expert_gb300 import BlockNorm

    v, _ = norm_case(T, D, dtype, block, post, kind)
    for q_cols in (None, 0, 32, 64, 128, 256):
        n = BlockNorm(T, D, dtype, block, gate=kind, post=post, residual_scale=0.7, eps=1e-5,
                      q_cols=q_cols, store_y=q_cols in (None, 64))
        run_norm(n, on(dev, v))
        check_norm(n, v, kind, q_cols, dtype, 0.7, 1e-5)


def check_norm_bwd(n, v, dy, dh, h, kind, dtype, grad, scale):
    a = arrays(v)
    T, D = a["block"].shape
    post = a["w_post"] is not None
    rstd = to64(n.rstd)
    rb = to64(n.block_rstd) if post else None
    d64, e64 = to64(dy), None if dh is None else to64(dh)
    ref = mo.block_norm_bwd(d64, e64, to64(h), a["block"], a["w"], rstd, a["w_post"], a["gate"],
                            kind, rb, scale)
    rs = rstd[:, None]
    xhat, wdy = np.abs(to64(h) * rs), np.abs(d64 * a["w"])
    mean = (wdy * xhat).mean(1, keepdims=True)
    stream = 0 if e64 is None else np.abs(e64)
    # the terms of dhs, and what their roundings and the mean's sum of D add up to
    terms = rs * (wdy + xhat * mean) + stream
    err = U * (8 * (rs * wdy + stream) + (D + 8) * rs * xhat * mean)
    g = 1.0
    if kind:
        g = np.abs(a["gate"])
        g = g[:, None] if kind == "token" else g[None, :]
    ohat = np.abs(a["block"]) * (rb[:, None] if post else 1.0)
    k = np.abs(a["w_post"]) if post else 1.0
    half = BF16 if grad == "bf16" else 0.0
    close(to64(n.dres), ref["dres"], half * np.abs(ref["dres"]) + abs(scale) * (err + 2 * U * terms),
          "dres")
    close(to64(n.dw), ref["dw"], (T + 4) * U * (np.abs(d64) * xhat).sum(0) + TINY, "dw")
    # a row's sum of k ohat dhs (the gate's of a column inside, a token's outside)
    inner = k * ohat * (g if kind == "column" else 1.0)
    p_err = (inner * err).sum(1) + (D + 12) * U * (inner * terms).sum(1)
    p_mag = (inner * terms).sum(1)
    if kind == "token":
        close(to64(n.dgate), ref["dgate"], p_err + TINY, "dgate")
    if kind == "column":
        lim = (k * ohat * err).sum(0) + (T + 8) * U * (k * ohat * terms).sum(0)
        close(to64(n.dgate), ref["dgate"], lim + TINY, "dgate")
    lim = k * g * (err + 6 * U * terms)
    if post:
        gt = g if kind == "token" else 1.0
        lim = rb[:, None] * (lim + ohat * gt * ((p_err + 6 * U * p_mag) / D)[:, None])
        col = (g * ohat * err).sum(0) + (T + 8) * U * (g * ohat * terms).sum(0)
        close(to64(n.dw_post), ref["dw_post"], col + TINY, "dw_post")
    half = BF16 if dtype == "bf16" else 0.0
    close(to64(n.dblock), ref["dblock"], half * np.abs(ref["dblock"]) + lim + TINY, "dblock")


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [None, "column", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,D,dtype,block", NORMS)
def test_block_norm_backward(dev, T, D, dtype, block, post, kind, grad):
    from demand_side_expert_gb300 import BlockNorm

    v, gen = norm_case(T, D, dtype, block, post, kind)
    dy = torch.randn(T, D, generator=gen).to(DT[grad])
    dh = torch.randn(T, D, generator=gen).to(DT[grad]) if T % 2 else None
    n = BlockNorm(T, D, dtype, block, gate=kind, post=post, residual_scale=0.7, eps=1e-5,
                  grad_dtype=grad)
    d = on(dev, v)
    run_norm(n, d)
    n.backward(dy.to(dev), d["block"], d["w"], d["w_post"], d["gate"],
               dh=None if dh is None else dh.to(dev))
    check_norm_bwd(n, v, dy, dh, n.h, kind, dtype, grad, 0.7)


def test_block_norm_gradient_matches_differences(dev):
    from demand_side_expert_gb300 import BlockNorm

    T, D = 3, 16
    for kind in (None, "column", "token"):
        for post in (False, True):
            v, gen = norm_case(T, D, "f32", "f32", post, kind)
            dy, dh = torch.randn(T, D, generator=gen), torch.randn(T, D, generator=gen)
            n = BlockNorm(T, D, "f32", gate=kind, post=post, residual_scale=0.7, eps=1e-5)
            d = on(dev, v)
            run_norm(n, d)
            n.backward(dy.to(dev), d["block"], d["w"], d["w_post"], d["gate"], dh=dh.to(dev))
            a = arrays(v)

            def total(**change):
                b = {**a, **change}
                r = mo.block_norm(b["block"], b["res"], b["w"], b["w_post"], b["gate"], kind, 0.7,
                                  1e-5)
                return (r["y"] * to64(dy)).sum() + (r["h"] * to64(dh)).sum()

            for name, grad in (("block", n.dblock), ("res", n.dres), ("w", n.dw),
                               ("w_post", n.dw_post), ("gate", n.dgate)):
                if a[name] is None:
                    assert grad is None
                    continue
                for at in np.ndindex(a[name].shape):
                    e = np.zeros_like(a[name])
                    e[at] = 1e-5
                    fd = (total(**{name: a[name] + e}) - total(**{name: a[name] - e})) / 2e-5
                    assert abs(fd - grad[at].item()) < 3e-5, (kind, post, name, at)


@pytest.mark.parametrize("D", [72, 2048, 8192])
def test_block_norm_strides_aliases_and_repeats(dev, D):
    """Strided rows give the contiguous rows' bits, h may be the residual; the backward pass
    repeats bit for bit, and may write over its own gradients."""
    from demand_side_expert_gb300 import BlockNorm, lrm

    T = 300
    v, gen = norm_case(T, D, "bf16", "f32", True, "column")
    d = on(dev, v)
    make = lambda: BlockNorm(T, D, "bf16", gate="column", residual_scale=0.9, q_cols=128,  # noqa: E731
                             store_y=True)
    a, b, c = make(), make(), make()
    run_norm(a, d)
    wide = torch.zeros(T, D + 40, device=dev)
    wide[:, 8:8 + D] = d["block"]
    wider = torch.zeros(T, 2 * D, dtype=torch.bfloat16, device=dev)
    wider[:, D:] = d["res"]
    run_norm(b, {**d, "block": wide[:, 8:8 + D], "res": wider[:, D:]})
    c.h.copy_(d["res"])
    run_norm(c, {**d, "res": c.h})
    for o in (b, c):
        for name in ("h", "y", "q_scale", "rstd", "block_rstd"):
            assert torch.equal(getattr(a, name), getattr(o, name)), name
        assert torch.equal(codes(a.q), codes(o.q))
    dy = torch.randn(T, D, generator=gen).to(dev)
    names = ("dres", "dblock", "dw", "dw_post", "dgate")
    args = (d["block"], d["w"], d["w_post"], d["gate"])
    a.backward(dy, *args, dh=dy)
    first = [getattr(a, n).clone() for n in names]
    for _ in range(3):
        a.backward(dy, *args, dh=dy)
        assert all(torch.equal(x, getattr(a, n)) for x, n in zip(first, names))
    over = dy.clone()
    lrm.lrm_block_norm_bwd(a.desc, over, dy, a.h, d["block"], d["w"], d["w_post"], d["gate"],
                           a.rstd, a.block_rstd, over, a.dblock, a.dw, a.dw_post, a.dgate, a._ws,
                           a.ws_bytes)
    assert torch.equal(over, first[0])
    over = dy.clone()
    lrm.lrm_block_norm_bwd(a.desc, dy, over, a.h, d["block"], d["w"], d["w_post"], d["gate"],
                           a.rstd, a.block_rstd, over, a.dblock, a.dw, a.dw_post, a.dgate, a._ws,
                           a.ws_bytes)
    assert torch.equal(over, first[0])


def test_block_norm_zero_rows_nan_and_inf(dev):
    """NaN and infinities stay in their rows, and reach the column sums as the formula says;
    a block of zeros leaves the scaled residual."""
    from demand_side_expert_gb300 import BlockNorm

    T, D = 6, 256
    v, gen = norm_case(T, D, "f32", "f32", True, "token")
    v["block"][1] = 0
    v["block"][2, 5] = math.nan
    v["res"][3, 7] = math.inf
    n = BlockNorm(T, D, "f32", gate="token", residual_scale=0.5, q_cols=128, store_y=True)
    d = on(dev, v)
    run_norm(n, d)
    assert torch.equal(n.h[1], 0.5 * d["res"][1])
    assert torch.isnan(n.y[2]).all() and torch.isnan(n.y[3, 7])
    good = [0, 1, 4, 5]
    assert torch.isfinite(n.y[good]).all() and torch.isfinite(n.q_scale[good]).all()
    dy = torch.randn(T, D, generator=gen).to(dev)
    n.backward(dy, d["block"], d["w"], d["w_post"], d["gate"])
    assert torch.isfinite(n.dres[good]).all() and torch.isfinite(n.dblock[good]).all()
    assert torch.isnan(n.dblock[2]).all() and torch.isnan(n.dw).all()


def test_block_norm_no_rows(dev):
    from demand_side_expert_gb300 import BlockNorm

    D = 64
    w = torch.ones(D, dtype=torch.bfloat16, device=dev)
    e, f = torch.empty(0, D, dtype=torch.bfloat16, device=dev), torch.empty(0, D, device=dev)
    for kind in (None, "column", "token"):
        n = BlockNorm(0, D, "bf16", gate=kind)
        gate = None if kind is None else w if kind == "column" else w[:0]
        n.forward(f, e, w, w, gate)
        n.dw.fill_(3)
        n.dw_post.fill_(3)
        n.backward(f, f, w, w, gate)
        assert (n.dw == 0).all() and (n.dw_post == 0).all()
        if kind == "column":
            assert (n.dgate == 0).all()


def test_block_norm_past_2_31_elements(dev):
    from demand_side_expert_gb300 import BlockNorm

    T, D = (1 << 18) + 3, 8192
    n = BlockNorm(T, D, "bf16", "bf16", gate="token", residual_scale=0.5, grad_dtype="bf16")
    w = torch.ones(D, dtype=torch.bfloat16, device=dev)
    b = torch.empty(T, D, dtype=torch.bfloat16, device=dev).normal_()
    r = torch.empty(T, D, dtype=torch.bfloat16, device=dev).normal_()
    gate = torch.empty(T, dtype=torch.bfloat16, device=dev).normal_()
    n.forward(b, r, w, w, gate)
    n.backward(r, b, w, w, gate, dh=b)
    tail = slice(T - 3, T)
    ref = mo.block_norm(to64(b[tail]), to64(r[tail]), to64(w), to64(w), to64(gate[tail]), "token",
                        0.5, 1e-6)
    lim = BF16 * np.abs(ref["h"]) + (D + 16) * U * (np.abs(ref["h"]) + np.abs(to64(r[tail])))
    close(to64(n.h[tail]), ref["h"], lim, "h")
    back = mo.block_norm_bwd(to64(r[tail]), to64(b[tail]), to64(n.h[tail]), to64(b[tail]), to64(w),
                             to64(n.rstd[tail]), to64(w), to64(gate[tail]), "token",
                             to64(n.block_rstd[tail]), 0.5)
    for name in ("dres", "dblock"):
        got = to64(getattr(n, name)[tail])
        # values near 1 and their sums of D terms
        close(got, back[name], BF16 * np.abs(back[name]) + 4 * (D + 16) * U * 8, name)


def test_block_norm_on_streams_and_in_a_graph(dev):
    from demand_side_expert_gb300 import BlockNorm

    T, D = 700, 512
    v, gen = norm_case(T, D, "bf16", "f32", True, "column")
    d = on(dev, v)
    dy = torch.randn(T, D, generator=gen).to(dev)
    side = torch.cuda.Stream()
    names = ("h", "y", "dres", "dblock", "dw", "dw_post", "dgate")
    got = []

    def once(n, stream=None):
        run_norm(n, d, stream=stream)
        n.backward(dy, d["block"], d["w"], d["w_post"], d["gate"], dh=dy, stream=stream)

    for stream in (None, side, side.cuda_stream):
        n = BlockNorm(T, D, "bf16", gate="column")
        torch.cuda.synchronize()
        once(n, stream)
        torch.cuda.synchronize()
        got.append([getattr(n, k).clone() for k in names])
    assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            once(n)
    d["block"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [getattr(n, k).clone() for k in names]
    once(n)
    assert all(torch.equal(a, getattr(n, k)) for a, k in zip(replayed, names))
    d["block"].mul_(0.5)
