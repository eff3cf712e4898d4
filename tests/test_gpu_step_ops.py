"""GPU tests of the operators around the expert passes (router, routing weights'
gradient, RMS norm, AdamW) against the float64 oracle.

u = 2^-24 is the unit rounding of float32; every tolerance below counts the
roundings of the longest chain that the operation needs, whatever order a kernel
takes: a sum of n terms is off by at most n u times the sum of their magnitudes.
"""

import math

import numpy as np
import pytest
import torch

from oracle import step_oracle as so

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8  # one rounding to bfloat16, with room for a float32 value at a tie
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    from demand_side_expert_gb300 import lrm  # noqa: F401  (liblrm.so must load)
    return torch.device("cuda:0")


def to64(t):
    return t.detach().cpu().double().numpy()


def close(got, ref, lim, name):
    """|got - ref| <= lim elementwise, NaN and infinities at the same places (a value
    past float32 is the infinity that float32 holds for it)."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    ref = np.where(np.abs(ref) > np.finfo(np.float32).max, np.copysign(np.inf, ref), ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), name
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), name
    fine = np.isfinite(ref)
    err = np.abs(got[fine] - ref[fine])
    over = err > np.broadcast_to(lim, ref.shape)[fine]
    assert not over.any(), f"{name}: {int(over.sum())} values off, worst {err.max():.3e}"


# -- router -------------------------------------------------------------------
def make_logits(T, E, dtype, seed, off=0.0, equal=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=gen) * 2 - 1.2 * torch.log(torch.arange(E) + 1.0)
    if equal:
        x = (x * 2).round() / 2  # many ties
    if off:
        x = x.masked_fill(torch.rand(T, E, generator=gen) < off, -math.inf)
    return x.to(DT[dtype])


def route_on(dev, x, K, renorm, mask=None, stats=True, balance=0.3, z=0.2):
    from demand_side_expert_gb300 import Router

    dtype = "bf16" if x.dtype is torch.bfloat16 else "f32"
    r = Router(x.shape[0], x.shape[1], K, dtype, renorm=renorm, balance_coef=balance, z_coef=z)
    m = None if mask is None else torch.as_tensor(mask, dtype=torch.uint8, device=dev)
    r.route(x.to(dev), mask=m, stats=stats)
    assert r.device_error() == 0
    return r, m


def router_tol(x):
    """Relative error of a softmax value: exp of a difference of size s is off by s u
    (its rounding) and 2 ulp, the sum of E positive terms by E u, the division by u."""
    x = np.where(np.isfinite(x), x, 0.0)
    span = x.max() - x.min() if x.size else 0.0
    return (2 * span + x.shape[1] + 16) * U


def check_route(r, x, K, renorm, mask, stats, balance=0.3, z=0.2):
    x64 = to64(x)
    ref = so.route(x64, K, renorm, balance, z, mask)
    assert np.array_equal(r.topk_idx.cpu().numpy(), ref["topk_idx"])
    tol = router_tol(x64)
    close(to64(r.alpha), ref["alpha"], (2 * tol) * np.nan_to_num(ref["alpha"]) + 1e-37, "alpha")
    if stats:
        T = x64.shape[0]
        assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
        close(to64(r.prob_sum), ref["prob_sum"],
              (tol + (T + 8) * U) * np.nan_to_num(ref["prob_sum"]) + 1e-37, "prob_sum")
        big = np.nan_to_num(np.abs(ref["lse"])).max() if T else 0.0
        slack = np.array([0.0, z * 2 * big * (tol + U * big)])
        close(to64(r.loss), ref["loss"],
              (2 * tol + (T + x64.shape[1] + 16) * U) * np.nan_to_num(np.abs(ref["loss"])) + slack,
              "loss")
    return ref


ROUTES = [  # T, E, K, dtype, off
    (1, 1, 1, "f32", 0), (1, 128, 8, "bf16", 0), (3, 31, 5, "f32", 0.5), (33, 32, 32, "bf16", 0),
    (257, 33, 1, "bf16", 0.2), (100, 64, 7, "f32", 0), (513, 100, 8, "f32", 0.3),
    (4099, 128, 8, "bf16", 0), (5003, 256, 8, "f32", 0.1), (65, 300, 6, "bf16", 0.9),
    (130, 512, 8, "f32", 0), (37, 1000, 32, "bf16", 0.1), (600, 1024, 4, "f32", 0)]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K,dtype,off", ROUTES)
def test_route_and_gradient(dev, T, E, K, dtype, off, renorm):
    x = make_logits(T, E, dtype, T + E, off, equal=E % 2 == 0)
    rng = np.random.default_rng(E)
    mask = (rng.random(T) < 0.8).astype(np.uint8) if T > 2 else None
    if T > 4:
        x[2] = -math.inf  # nothing to choose from
    r, m = route_on(dev, x, K, renorm, mask)
    ref = check_route(r, x, K, renorm, mask, True)
    serve, _ = route_on(dev, x, K, renorm, mask, stats=False)
    assert torch.equal(serve.topk_idx, r.topk_idx) and torch.equal(serve.alpha, r.alpha)

    da, dl = rng.standard_normal((T, K)).astype(np.float32), np.array([1.5, -0.5], np.float32)
    r.backward(x.to(dev), torch.from_numpy(da).to(dev), mask=m,
               dloss=torch.from_numpy(dl).to(dev))
    assert r.device_error() == 0
    want = so.route_bwd(to64(x), ref["topk_idx"], ref["counts"], da, dl, renorm, 0.3, 0.2, mask)
    # p and alpha carry router_tol; they multiply dalpha, its mean (K terms), the
    # balance cost, its mean (E terms) and lse
    n = max(1, int(ref["use"].sum()))
    cost = abs(dl[0]) * 0.3 * E * ref["counts"].max() / (n * n * K) if T else 0
    zt = abs(dl[1]) * 2 * 0.2 * (np.abs(ref["lse"]).max() + 1) / n
    mag = 2 * np.abs(da).max(1) + 2 * cost + zt
    a = np.zeros((T, E))
    np.put_along_axis(a, ref["topk_idx"].astype(np.int64), ref["alpha"], 1)
    lim = (3 * router_tol(to64(x)) + (K + E + 16) * U) * np.maximum(a, ref["p"]) * mag[:, None]
    if dtype == "bf16":
        lim = lim + BF16 * np.abs(want)
    close(to64(r.dlogits), want, lim + 1e-37, "dlogits")


MANY = [(5000, 20, 1, "f32"), (6001, 32, 5, "bf16"), (5000, 60, 2, "bf16"), (5000, 64, 8, "f32"),
        (7003, 100, 3, "bf16"), (9000, 128, 8, "f32"), (5000, 200, 4, "f32"), (5001, 256, 8, "bf16"),
        (5000, 256, 12, "f32"), (5000, 130, 1, "f32"), (5000, 5, 5, "f32"), (5000, 8, 8, "bf16"),
        (5000, 1, 1, "f32")]


@pytest.mark.parametrize("kind", ["normal", "equal", "near", "zeros", "closed", "nan"])
@pytest.mark.parametrize("T,E,K,dtype", MANY)
def test_route_many_tokens(dev, T, E, K, dtype, kind):
    """Enough tokens that they share warps, and logits that are hard to rank: equal
    ones, ones that differ in the last bits only, zeros of both signs, mostly closed
    experts, NaN. The choices have to be those of a stable sort, bit for bit."""
    gen = torch.Generator().manual_seed(E)
    x = torch.randn(T, E, generator=gen)
    if kind == "equal":
        x = (x * 2).round() / 2
    if kind == "near":
        x = 1 + torch.randint(0, 300, (T, E), generator=gen) * 2.0 ** -23
        x = torch.where(torch.rand(T, E, generator=gen) < 0.3, x, -x)
    if kind == "zeros":
        x = torch.where(torch.rand(T, E, generator=gen) < 0.5, 0.0, -0.0)
    if kind == "closed":
        x = x.masked_fill(torch.rand(T, E, generator=gen) < 0.95, -math.inf)
    if kind == "nan":
        x = x.masked_fill(torch.rand(T, E, generator=gen) < 0.01, math.nan)
    x = x.to(DT[dtype])
    r, _ = route_on(dev, x, K, K > 2)
    x64 = to64(x)
    idx = so.topk(x64, K)
    assert np.array_equal(r.topk_idx.cpu().numpy(), idx)
    use = so.takes_part(x64)
    counts = np.bincount(idx[use].reshape(-1), minlength=E)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    good = use & ~np.isnan(x64).any(1)
    top = np.where(good, np.max(np.where(np.isnan(x64), -np.inf, x64), 1), 0.0)
    with np.errstate(invalid="ignore"):
        p = np.where(good[:, None], np.exp(x64 - top[:, None]), 0.0)
    p /= np.where(good, p.sum(1), 1.0)[:, None]
    want = np.take_along_axis(p, idx.astype(np.int64), 1)
    if K > 2:
        want = want / np.where(good, want.sum(1), 1.0)[:, None]
    got = to64(r.alpha)
    close(got[good], want[good], 2 * router_tol(x64) * want[good] + 1e-37, "alpha")
    assert np.isnan(got[use & ~good]).all() and (got[~use] == 0).all()
    if kind != "nan":
        close(to64(r.prob_sum), p.sum(0), (router_tol(x64) + (T + 8) * U) * p.sum(0) + 1e-37,
              "prob_sum")


def test_route_gradient_matches_differences(dev):
    """The kernel's own gradient against central differences of the float64 loss."""
    T, E, K = 4, 9, 3
    x = make_logits(T, E, "f32", 5)
    rng = np.random.default_rng(0)
    da = rng.standard_normal((T, K))
    for renorm in (False, True):
        r, _ = route_on(dev, x, K, renorm)
        r.backward(x.to(dev), torch.from_numpy(da).float().to(dev))
        idx = r.topk_idx.cpu().numpy()
        x64, da32 = to64(x), da.astype(np.float32).astype(np.float64)

        def total(v):
            q = so.route(v, K, renorm, 0.3, 0.2, idx=idx)
            return (q["alpha"] * da32).sum() + q["loss"].sum()

        for t in range(T):
            for e in range(E):
                d = np.zeros_like(x64)
                d[t, e] = 1e-5
                fd = (total(x64 + d) - total(x64 - d)) / 2e-5
                assert abs(fd - r.dlogits[t, e].item()) < 1e-5


def test_route_strided_rows_and_mask_types(dev):
    T, E, K = 70, 20, 4
    wide = make_logits(T, 3 * E + 1, "bf16", 1).to(dev)
    x = wide[:, 16:16 + E]
    mask = torch.arange(T, device=dev) % 3 != 0
    from demand_side_expert_gb300 import Router
    r, s = Router(T, E, K, "bf16"), Router(T, E, K, "bf16")
    r.route(x, mask=mask)
    s.route(x.contiguous(), mask=mask.to(torch.uint8))
    for name in ("topk_idx", "alpha", "counts", "prob_sum", "loss"):
        assert torch.equal(getattr(r, name), getattr(s, name)), name
    r.backward(x, r.alpha, mask=mask)
    s.backward(x.contiguous(), s.alpha, mask=mask)
    assert torch.equal(r.dlogits, s.dlogits)


def test_route_extreme_logits(dev):
    lowest = torch.finfo(torch.float32).min
    x = torch.tensor([
        [lowest, lowest, lowest, lowest],          # the type's lowest value everywhere: uniform
        [lowest, 3.0, lowest, -1.0],
        [0.0, -0.0, -0.0, 0.0],                    # one value: the lower ids win
        [3.4e38, lowest, 0.0, 3.4e38],
        [-math.inf, -math.inf, 2.0, -math.inf],    # fewer open experts than choices
        [1e-40, 2e-40, -1e-40, 0.0],               # subnormal
    ])
    for renorm in (False, True):
        r, _ = route_on(dev, x, 2, renorm)
        check_route(r, x, 2, renorm, None, True)
        assert torch.isfinite(r.alpha).all() and torch.isfinite(r.prob_sum).all()


def test_route_nan_and_inf(dev):
    """NaN and +inf reach the outputs of the tokens that take part, and only those:
    a masked row with them changes nothing."""
    clean = make_logits(6, 8, "f32", 3)
    dirty = clean.clone()
    dirty[1, 3], dirty[4] = math.nan, math.inf
    mask = np.array([1, 0, 1, 1, 0, 1], np.uint8)
    a, m = route_on(dev, clean, 3, True, mask)
    b, _ = route_on(dev, dirty, 3, True, mask)
    for name in ("alpha", "counts", "prob_sum", "loss"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    da = torch.ones(6, 3, device=dev)
    da[1] = math.nan
    b.backward(dirty.to(dev), da, mask=m)
    assert torch.isfinite(b.dlogits).all()
    assert (b.dlogits[[1, 4]] == 0).all()
    # ids of every row are valid and distinct; NaN is not chosen before a number
    idx = b.topk_idx.cpu().numpy()
    assert all(len(set(row)) == 3 and row.min() >= 0 and row.max() < 8 for row in idx)
    assert 3 not in idx[1]
    for renorm in (False, True):
        c, _ = route_on(dev, dirty, 3, renorm)
        assert torch.isnan(c.alpha[[1, 4]]).all() and torch.isfinite(c.alpha[[0, 2, 3, 5]]).all()
        assert torch.isnan(c.prob_sum).any() and torch.isnan(c.loss).all()
        c.backward(dirty.to(dev), torch.ones(6, 3, device=dev))


def test_route_no_tokens_and_all_masked(dev):
    from demand_side_expert_gb300 import Router

    r = Router(0, 8, 2, "f32", balance_coef=1.0, z_coef=1.0)
    r.counts.fill_(7)
    x = torch.empty(0, 8, device=dev)
    r.route(x)
    assert (r.counts == 0).all() and (r.prob_sum == 0).all() and (r.loss == 0).all()
    r.route(x, stats=False)
    r.backward(x)
    x = make_logits(300, 8, "f32", 0).to(dev)
    s = Router(300, 8, 2, "f32", balance_coef=1.0, z_coef=1.0)
    mask = torch.zeros(300, dtype=torch.bool, device=dev)
    s.route(x, mask=mask)
    assert (s.alpha == 0).all() and (s.counts == 0).all() and (s.loss == 0).all()
    s.backward(x, torch.ones(300, 2, device=dev), mask=mask)
    assert (s.dlogits == 0).all()


def test_route_bad_ids_are_flagged(dev):
    from demand_side_expert_gb300 import lrm

    x = make_logits(5, 8, "f32", 0).to(dev)
    r, _ = route_on(dev, x.cpu(), 2, False)
    r.topk_idx[1, 0], r.topk_idx[3, 1] = 8, -1
    r.backward(x, torch.ones(5, 2, device=dev))
    assert r.device_error() == lrm.LRM_DEVERR_EXPERT_ID
    assert torch.isfinite(r.dlogits).all()


def test_route_repeats_bit_for_bit_and_in_a_graph(dev):
    """Statistics do not depend on the order in which CTAs arrive; a captured call
    replays on new logits; calls on a stream of their own."""
    x = make_logits(20000, 128, "bf16", 0).to(dev)
    r, _ = route_on(dev, x.cpu(), 8, False)
    first = [t.clone() for t in (r.alpha, r.counts, r.prob_sum, r.loss)]
    for _ in range(5):
        r.route(x)
        assert all(torch.equal(a, b) for a, b in
                   zip(first, (r.alpha, r.counts, r.prob_sum, r.loss)))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            r.route(held)
    held.copy_(make_logits(20000, 128, "bf16", 1))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (r.alpha, r.counts, r.prob_sum, r.loss)]
    r.route(held)
    assert all(torch.equal(a, b) for a, b in zip(got, (r.alpha, r.counts, r.prob_sum, r.loss)))
    assert not torch.equal(got[3], first[3])


def test_route_past_2_31_elements(dev):
    """Rows of logits whose offsets need 64 bits, forward and backward."""
    from demand_side_expert_gb300 import Router

    T, E, K = (1 << 21) + 77, 1024, 4
    x = torch.empty(T, E, dtype=torch.bfloat16, device=dev).normal_()
    r = Router(T, E, K, "bf16", renorm=True, balance_coef=0.0)
    r.route(x)
    da = torch.ones(T, K, device=dev)
    da[:, 1] = -1
    r.backward(x, da)
    assert r.counts.sum().item() == T * K
    tail = x[-5:].cpu()
    ref = so.route(to64(tail), K, True)
    assert np.array_equal(r.topk_idx[-5:].cpu().numpy(), ref["topk_idx"])
    tol = router_tol(to64(tail))
    close(to64(r.alpha[-5:]), ref["alpha"], 2 * tol * ref["alpha"], "alpha")
    want = so.route_bwd(to64(tail), ref["topk_idx"], ref["counts"], to64(da[-5:]), (0, 0), True)
    a = np.zeros((5, E))
    np.put_along_axis(a, ref["topk_idx"].astype(np.int64), ref["alpha"], 1)
    lim = (3 * tol + (K + 16) * U) * a * 2 * np.abs(to64(da[-5:])).max() + BF16 * np.abs(want)
    close(to64(r.dlogits[-5:]), want, lim + 1e-37, "dlogits")


def test_calls_on_a_stream_of_their_own(dev):
    """The stream argument: work ordered on it alone gives the current stream's bits."""
    from demand_side_expert_gb300 import AddRMSNorm, AdamW, Router

    gen = torch.Generator().manual_seed(4)
    x = torch.randn(700, 64, generator=gen).to(dev)
    w = torch.ones(64, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for stream in (None, side, side.cuda_stream):
        norm, router = AddRMSNorm(700, 64, "f32"), Router(700, 64, 4, "f32")
        p, g = torch.ones(5000, device=dev), torch.full((5000,), 0.5, device=dev)
        opt = AdamW([p], [g], state="f8")
        torch.cuda.synchronize()
        norm.forward(x, w, residual=x, stream=stream)
        router.route(norm.y, stream=stream)
        router.backward(norm.y, router.alpha, stream=stream)
        norm.backward(router.dlogits, w, stream=stream)
        opt.step(stream=stream)
        side.synchronize()
        torch.cuda.synchronize()
        got.append([t.clone() for t in (norm.y, router.alpha, router.loss, router.dlogits,
                                        norm.dx, norm.dw, p)])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# -- routing weights' gradient ----------------------------------------------------
@pytest.mark.parametrize("T,D,K,dtype", [
    (1, 8, 1, "f32"), (5, 64, 2, "bf16"), (33, 1000, 8, "bf16"), (17, 2048, 9, "f32"),
    (130, 4096, 8, "bf16"), (7, 72, 32, "f32"), (3, 8200, 3, "bf16")])
def test_gate_grad(dev, T, D, K, dtype):
    from demand_side_expert_gb300 import lrm

    gen = torch.Generator().manual_seed(D)
    E = max(K, 4)
    g = torch.randn(T, D, generator=gen).to(DT[dtype])
    y = torch.randn(T * K, D, generator=gen).to(DT[dtype])
    inv = torch.randperm(T * K, generator=gen).to(torch.int32)
    shape = lrm.make_shape(T, D, 8, E, K, lrm.LRM_BF16 if dtype == "bf16" else lrm.LRM_F32)
    n = lrm.lrm_workspace_bytes(shape)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    out = torch.full((T, K), math.nan, device=dev)
    lrm.lrm_gate_grad(shape, g.to(dev), y.to(dev), inv.to(dev), out, ws, n)
    want = so.gate_grad(to64(g), to64(y), inv.numpy(), K)
    mag = so.gate_grad(np.abs(to64(g)), np.abs(to64(y)), inv.numpy(), K)
    close(to64(out), want, (D + 1) * U * mag, "dalpha")
    bad = inv.clone()
    bad[0] = T * K
    lrm.lrm_gate_grad(shape, g.to(dev), y.to(dev), bad.to(dev), out, ws, n)
    assert out[0, 0].item() == 0
    assert lrm.lrm_get_device_error(ws, n) == lrm.LRM_DEVERR_INDEX


def test_gate_grad_past_2_31_elements(dev):
    """Rows of y whose offsets need 64 bits."""
    from demand_side_expert_gb300 import lrm

    T, D, K = 34000, 8192, 8
    g = torch.empty(T, D, dtype=torch.bfloat16, device=dev).normal_()
    y = torch.empty(T * K, D, dtype=torch.bfloat16, device=dev).normal_()
    inv = torch.arange(T * K, dtype=torch.int32, device=dev).flip(0)
    shape = lrm.make_shape(T, D, 8, 8, K, lrm.LRM_BF16)
    n = lrm.lrm_workspace_bytes(shape)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    out = torch.empty(T, K, device=dev)
    lrm.lrm_gate_grad(shape, g, y, inv, out, ws, n)
    for t in (0, 1, T - 2, T - 1):
        rows = y[inv[t * K:(t + 1) * K].long()]
        want = (rows.double() * g[t].double()).sum(1).cpu().numpy()
        mag = (rows.double().abs() * g[t].double().abs()).sum(1).cpu().numpy()
        close(to64(out[t]), want, (D + 1) * U * mag, "dalpha")


# -- norm -------------------------------------------------------------------------
NORMS = [  # T, D, dtype
    (1, 8, "f32"), (1, 4096, "bf16"), (3, 40, "bf16"), (5, 256, "f32"), (9, 264, "bf16"),
    (130, 512, "f32"), (700, 776, "bf16"), (31, 1024, "f32"), (333, 1032, "bf16"),
    (64, 2048, "bf16"), (21, 2056, "f32"), (11, 4104, "f32"), (6, 8192, "bf16"),
    (4, 8200, "bf16"), (2, 16384, "f32"), (3, 16384, "bf16")]


def norm_inputs(T, D, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + D)
    dt = DT[dtype]
    x, res = torch.randn(T, D, generator=gen).to(dt), (torch.randn(T, D, generator=gen) * 3).to(dt)
    return x, res, (1 + 0.2 * torch.randn(D, generator=gen)).to(dt), gen


def check_norm(n, x, res, w, eps, q_cols, dtype):
    D = x.shape[1]
    ref = so.add_rmsnorm(to64(x), None if res is None else to64(res), to64(w), eps, q_cols)
    # a sum of D squares (each with the rounding of h twice), a division, a root
    rs = (D + 8) * U
    close(to64(n.rstd), ref["rstd"], rs * ref["rstd"], "rstd")
    out = BF16 if dtype == "bf16" else 0.0
    mag = np.abs(ref["y"])
    if res is not None:
        h_lim = U * (np.abs(to64(x)) + np.abs(to64(res)))
        close(to64(n.h), ref["h"], out * np.abs(ref["h"]) + 2 * h_lim, "h")
        # the rounding of the sum reaches y times rstd w
        mag = mag + h_lim / U * ref["rstd"][:, None] * np.abs(to64(w))
    y_lim = (rs + 4 * U) * mag
    if n.y is not None:
        close(to64(n.y), ref["y"], out * np.abs(ref["y"]) + y_lim, "y")
    if q_cols is not None:
        cols = q_cols or D
        s = to64(n.q_scale)
        assert s.shape == ref["q_scale"].shape
        top = np.stack([y_lim[:, c:c + cols].max(1) for c in range(0, D, cols)], 1) / so.F8_MAX
        close(s, ref["q_scale"], top + 4 * U * ref["q_scale"], "q_scale")
        scale = np.repeat(s, cols, axis=1)[:, :D]
        # half a step of the code: 2^-4 of a normal value, 2^-10 below
        got = to64(n.q.float()) * scale
        half = np.maximum(np.abs(ref["y"]) * 2.0 ** -4, scale * 2.0 ** -10)
        close(got, ref["y"], half * (1 + 1e-3) + 4 * y_lim, "q")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,D,dtype", NORMS)
def test_norm_forward(dev, T, D, dtype, residual):
    from demand_side_expert_gb300 import AddRMSNorm

    x, res, w, _ = norm_inputs(T, D, dtype)
    res = res if residual else None
    for q_cols in (None, 0, 32, 64, 128, 256):
        n = AddRMSNorm(T, D, dtype, eps=1e-5, q_cols=q_cols, store_y=q_cols in (None, 64))
        n.forward(x.to(dev), w.to(dev), residual=None if res is None else res.to(dev))
        check_norm(n, x, res, w, 1e-5, q_cols, dtype)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,dtype", NORMS + [(1500, 264, "bf16"), (2500, 1032, "f32")])
def test_norm_backward(dev, T, D, dtype, grad):
    from demand_side_expert_gb300 import AddRMSNorm

    x, _, w, gen = norm_inputs(T, D, dtype)
    dy = torch.randn(T, D, generator=gen).to(DT[grad])
    dh = torch.randn(T, D, generator=gen).to(DT[grad]) if T % 2 else None
    n = AddRMSNorm(T, D, dtype, eps=1e-5, grad_dtype=grad)
    n.forward(x.to(dev), w.to(dev))
    rstd = to64(n.rstd)
    n.backward(dy.to(dev), w.to(dev), dh=None if dh is None else dh.to(dev), h=x.to(dev))
    dx, dw = so.add_rmsnorm_bwd(to64(dy), None if dh is None else to64(dh), to64(x), to64(w), rstd)
    h, d64, w64 = to64(x), to64(dy), to64(w)
    xhat = np.abs(h * rstd[:, None])
    wdy = np.abs(d64 * w64)
    mag = rstd[:, None] * (wdy * 8 + xhat * (wdy * xhat).mean(1, keepdims=True) * (D + 8))
    lim = U * (mag + (0 if dh is None else 2 * np.abs(to64(dh))))
    if grad == "bf16":
        lim = lim + BF16 * np.abs(dx)
    close(to64(n.dx), dx, lim, "dx")
    close(to64(n.dw), dw, (T + 3) * U * (np.abs(d64) * xhat).sum(0) + 1e-37, "dw")


def test_norm_gradient_matches_differences(dev):
    from demand_side_expert_gb300 import AddRMSNorm

    T, D = 3, 16
    x, res, w, gen = norm_inputs(T, D, "f32")
    dy, dh = torch.randn(T, D, generator=gen), torch.randn(T, D, generator=gen)
    n = AddRMSNorm(T, D, "f32", eps=1e-5)
    n.forward(x.to(dev), w.to(dev), residual=res.to(dev))
    n.backward(dy.to(dev), w.to(dev), dh=dh.to(dev))

    def total(x_, w_):
        r = so.add_rmsnorm(x_, to64(res), w_, 1e-5)
        return (r["y"] * to64(dy)).sum() + (r["h"] * to64(dh)).sum()

    for i in range(T):
        for j in range(D):
            e = np.zeros((T, D))
            e[i, j] = 1e-5
            fd = (total(to64(x) + e, to64(w)) - total(to64(x) - e, to64(w))) / 2e-5
            assert abs(fd - n.dx[i, j].item()) < 2e-5
    for j in range(D):
        e = np.zeros(D)
        e[j] = 1e-5
        fd = (total(to64(x), to64(w) + e) - total(to64(x), to64(w) - e)) / 2e-5
        assert abs(fd - n.dw[j].item()) < 2e-5


@pytest.mark.parametrize("D", [72, 2048, 8192])
def test_norm_strides_aliases_and_repeats(dev, D):
    """Strided rows give the contiguous rows' bits, in place as well; the backward
    pass repeats bit for bit, and may write over its own gradients."""
    from demand_side_expert_gb300 import AddRMSNorm, lrm

    T = 300
    x, res, w, gen = norm_inputs(T, D, "bf16")
    x, res, w = x.to(dev), res.to(dev), w.to(dev)
    a = AddRMSNorm(T, D, "bf16", q_cols=128, store_y=True)
    a.forward(x, w, residual=res)
    wide = torch.zeros(T, D + 40, dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + D] = x
    wider = torch.zeros(T, 2 * D, dtype=torch.bfloat16, device=dev)
    wider[:, D:] = res
    b = AddRMSNorm(T, D, "bf16", q_cols=128, store_y=True)
    b.forward(wide[:, 8:8 + D], w, residual=wider[:, D:])
    for name in ("h", "y", "q_scale", "rstd"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
    # the sum over the residual, the norm over x
    c = AddRMSNorm(T, D, "bf16")
    hx, hr = x.clone(), res.clone()
    lrm.lrm_add_rmsnorm(c.desc, hx, hr, w, hr, hx, None, None, c.rstd)
    assert torch.equal(hr, a.h) and torch.equal(hx, a.y) and torch.equal(c.rstd, a.rstd)
    dy = torch.randn(T, D, generator=gen).to(dev)
    a.backward(dy, w, dh=dy)
    dx, dw = a.dx.clone(), a.dw.clone()
    for _ in range(3):
        a.backward(dy, w, dh=dy)
        assert torch.equal(a.dx, dx) and torch.equal(a.dw, dw)
    over = dy.clone()
    lrm.lrm_add_rmsnorm_bwd(a.desc, over, dy, a.h, w, a.rstd, over, a.dw, a._ws, a.ws_bytes)
    assert torch.equal(over, dx)


def test_norm_zero_rows_nan_and_inf(dev):
    from demand_side_expert_gb300 import AddRMSNorm

    T, D = 6, 256
    x, _, w, _ = norm_inputs(T, D, "f32")
    x[1] = 0
    x[2, 5] = math.nan
    x[3, 7] = math.inf
    x[4] *= 1e-25  # squares below the smallest float32: eps alone is left
    n = AddRMSNorm(T, D, "f32", eps=1e-6, q_cols=128, store_y=True)
    n.forward(x.to(dev), w.to(dev))
    assert (n.y[1] == 0).all() and (n.q[1].float() == 0).all()
    assert torch.isfinite(n.q_scale[[0, 1, 4, 5]]).all() and (n.q_scale[1] > 0).all()
    assert torch.isnan(n.y[2]).all() and torch.isnan(n.q[2].float()).all()
    assert torch.isnan(n.y[3, 7])
    good = [0, 1, 4, 5]
    ref = so.add_rmsnorm(to64(x[good]), None, to64(w), 1e-6)
    close(to64(n.y[good]), ref["y"], (D + 12) * U * np.abs(ref["y"]) + 1e-37, "y")
    # eps = 0 and a zero row: 0 / 0, as the formula says
    z = AddRMSNorm(1, 8, "f32", eps=0.0)
    z.forward(torch.zeros(1, 8, device=dev), torch.ones(8, device=dev))
    assert torch.isnan(z.y).all()


def test_norm_backward_keeps_infinities_apart(dev):
    """A row whose 1/rms is infinite (zeros and eps = 0) leaves the other rows' gradients
    alone, and reaches dw as its formula says: 0 * inf in every column."""
    from demand_side_expert_gb300 import AddRMSNorm

    T, D = 5, 64
    x, _, w, gen = norm_inputs(T, D, "f32")
    x[0] = 0
    n = AddRMSNorm(T, D, "f32", eps=0.0)
    n.forward(x.to(dev), w.to(dev))
    assert torch.isinf(n.rstd[0])
    dy = torch.randn(T, D, generator=gen)
    n.backward(dy.to(dev), w.to(dev), h=x.to(dev))
    dx, _ = so.add_rmsnorm_bwd(to64(dy[1:]), None, to64(x[1:]), to64(w), to64(n.rstd[1:]))
    close(to64(n.dx[1:]), dx, 64 * U * (np.abs(dx) + 8), "dx")
    assert torch.isnan(n.dx[0]).all() and torch.isnan(n.dw).all()


def test_norm_no_rows(dev):
    from demand_side_expert_gb300 import AddRMSNorm

    n = AddRMSNorm(0, 64, "bf16")
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    n.forward(e, w)
    n.dw.fill_(3)
    n.backward(torch.empty(0, 64, device=dev), w, h=e)
    assert (n.dw == 0).all()


def test_norm_past_2_31_elements(dev):
    """Row offsets that need 64 bits: the last rows of 2.2e9 elements."""
    from demand_side_expert_gb300 import AddRMSNorm

    D, T = 2048, (1 << 20) + 50021
    x = torch.empty(T, D, dtype=torch.bfloat16, device=dev).normal_()
    w = torch.ones(D, dtype=torch.bfloat16, device=dev)
    n = AddRMSNorm(T, D, "bf16", grad_dtype="bf16")
    n.forward(x, w)
    n.backward(x, w, h=x)
    tail = x[-3:].cpu()
    ref = so.add_rmsnorm(to64(tail), None, np.ones(D), 1e-6)
    lim = (D + 12) * U * np.abs(ref["y"])
    close(to64(n.y[-3:]), ref["y"], BF16 * np.abs(ref["y"]) + lim, "y")
    dx, _ = so.add_rmsnorm_bwd(to64(tail), None, to64(tail), np.ones(D), to64(n.rstd[-3:]))
    lim = U * (8 * np.abs(to64(tail)) + np.abs(ref["y"]) * 2 * (D + 8))
    close(to64(n.dx[-3:]), dx, BF16 * np.abs(dx) + lim, "dx")
    # x . xhat summed over rows is sum x^2 rstd: one column in 64 bits on the device
    col = (x[:, 77].double().square() * n.rstd.double()).sum().item()
    assert abs(n.dw[77].item() - col) <= (T // 600 + 700) * U * col


def test_norm_refuses_tensors(dev):
    from demand_side_expert_gb300 import AddRMSNorm

    n = AddRMSNorm(4, 64, "bf16")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    for bad in (x.float(), x.cpu(), x[:3], torch.zeros(64, 4, dtype=x.dtype, device=dev).t(),
                x[:1].expand(4, 64)):
        with pytest.raises(ValueError):
            n.forward(bad, w)
    with pytest.raises(ValueError):
        n.forward(x, w.float())
    with pytest.raises(ValueError):
        n.forward(x, w, residual=x[:, :32])
    with pytest.raises(ValueError):
        n.backward(x, w, h=x)  # float32 gradients are expected
    n.forward(x, w)
    with pytest.raises(ValueError):
        n.backward(x.float(), w)  # no residual, no sum of one
    with pytest.raises(AttributeError):
        n.rstd = torch.zeros(4, device=dev)


# -- AdamW --------------------------------------------------------------------------
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("param,master", [("f32", False), ("bf16", False), ("bf16", True)])
def test_adamw_matches_the_formula(dev, param, master, state, grad):
    """Several steps over tensors of odd lengths; each step is checked from the state
    that the one before it left."""
    from demand_side_expert_gb300 import AdamW

    rng = np.random.default_rng(1)
    sizes = [1, 7, 8, 255, 256, 257, 2048, 2049, 5000, 70001] + [3] * 150
    decay = [0.0 if n < 300 else 0.1 for n in sizes]
    params = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(DT[param]).to(dev)
              for n in sizes]
    grads = [torch.zeros(n, dtype=DT[grad], device=dev) for n in sizes]
    opt = AdamW(params, grads, weight_decay=decay, state=state, master=master, **HYPER)
    scale = torch.tensor([0.5], device=dev)
    for step in range(1, 4):
        for g in grads:
            g.copy_(torch.from_numpy(rng.standard_normal(g.numel()) * 10.0 ** rng.uniform(-6, 1)))
        old = []
        for i, n in enumerate(sizes):
            sl = slice(opt.starts[i], opt.starts[i] + n)
            m, v = to64(opt.m[sl].float()), to64(opt.v[sl].float())
            if state == "f8":
                b = slice(opt.starts[i] // 256, opt.starts[i] // 256 + -(-n // 256))
                m = m * np.repeat(to64(opt.m_scale[b]), 256)[:n]
                v = (v * np.repeat(to64(opt.v_scale[b]), 256)[:n]) ** 2
            old.append((to64(opt.master[sl] if master else params[i]), m, v))
        opt.step(grad_scale=scale if step == 2 else None)
        for i, n in enumerate(sizes):
            sl = slice(opt.starts[i], opt.starts[i] + n)
            p0, m0, v0 = old[i]
            g = to64(grads[i])
            s = 0.5 if step == 2 else 1.0
            p, m, v = so.adamw(p0, g, m0, v0, step, HYPER["lr"], *HYPER["betas"], HYPER["eps"],
                               decay[i], s)
            # sums of two products; the dequantised values carry one rounding each
            m_lim = 6 * U * (np.abs(m0) + 0.1 * np.abs(g) * s)
            v_lim = 8 * U * v
            den = np.sqrt(v) / math.sqrt(1 - 0.95 ** step) + 1e-8
            lr = HYPER["lr"] / (1 - 0.9 ** step)
            p_lim = 4 * U * np.abs(p0) + lr * (m_lim / den + np.abs(m) / den * 12 * U)
            if master:
                close(to64(opt.master[sl]), p, p_lim, "master")
            out = BF16 if param == "bf16" else 0.0
            close(to64(params[i]), p, p_lim + out * np.abs(p), "param")
            if state == "f32":
                close(to64(opt.m[sl]), m, m_lim, "m")
                close(to64(opt.v[sl]), v, v_lim + 1e-45, "v")
                continue
            b = slice(opt.starts[i] // 256, opt.starts[i] // 256 + -(-n // 256))
            for name, w, lim, root in (("m", m, m_lim, False),
                                       ("v", np.sqrt(v), 8 * U * np.sqrt(v), True)):
                sc = np.repeat(to64(getattr(opt, name + "_scale")[b]), 256)[:n]
                _, want = so.quantise_blocks(w, root)
                top = np.repeat(want, 256)[:n]
                # a block's scale follows its largest value, wherever that is
                worst = max(lim.max(initial=0.0) / so.F8_MAX, 0)
                close(sc, top, 4 * U * top + worst, name + "_scale")
                got = to64(getattr(opt, name)[sl].float()) * sc
                half = np.maximum(np.abs(w) * 2.0 ** -4, sc * 2.0 ** (-9 if root else -10))
                close(got, w, half * (1 + 1e-3) + 2 * lim, name)
                if root:
                    assert ((got > 0) == (w > 0)).all()


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_adamw_leaves_padding_and_neighbours(dev, state):
    from demand_side_expert_gb300 import AdamW

    flat = torch.full((4096,), 7.0, device=dev)
    params = [flat[16:16 + 33], flat[256:256 + 1000]]
    grads = [torch.ones(33, device=dev), torch.ones(1000, device=dev)]
    opt = AdamW(params, grads, state=state)
    opt.step()
    keep = torch.ones(4096, dtype=torch.bool)
    keep[16:49] = False
    keep[256:1256] = False
    assert (flat.cpu()[keep] == 7).all() and (flat.cpu()[~keep] != 7).all()
    assert (opt.m[33:256].float() == 0).all() and (opt.v[1256:].float() == 0).all()


def test_adamw_state_round_trip_and_repeats(dev):
    from demand_side_expert_gb300 import AdamW

    def make(state):
        gen = torch.Generator().manual_seed(2)
        ps = [torch.randn(n, generator=gen).to(torch.bfloat16).to(dev) for n in (300, 4000)]
        gs = [torch.randn(n, generator=gen).to(dev) for n in (300, 4000)]
        return AdamW(ps, gs, state=state, master=True), ps

    for state in ("f32", "f8"):
        a, pa = make(state)
        a.step()
        a.step()
        saved = {k: v.clone() if torch.is_tensor(v) else v for k, v in a.state_dict().items()}
        held = [p.clone() for p in pa]
        a.step(lr=0.5)
        b, pb = make(state)
        b.load_state_dict(saved)
        for p, h in zip(pb, held):
            p.copy_(h)
        b.step(lr=0.5)
        assert a.t == b.t == 3
        for x, y in zip(pa, pb):
            assert torch.equal(x, y)
        assert torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))
        assert torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8))
        assert torch.equal(a.master, b.master)
        with pytest.raises(ValueError):
            b.load_state_dict({**saved, "master": None})
        with pytest.raises(ValueError):
            b.load_state_dict({**saved, "m": saved["m"][:-256]})


def test_adamw_nan_and_inf(dev):
    """A NaN gradient stays in its own value, an infinite one in its block of 256."""
    from demand_side_expert_gb300 import AdamW

    for state in ("f32", "f8"):
        p = torch.ones(1024, device=dev)
        g = torch.ones(1024, device=dev)
        g[3], g[600] = math.nan, math.inf
        opt = AdamW([p], [g], state=state)
        opt.step()
        assert torch.isnan(p[3]) and torch.isnan(p[600])
        assert torch.isfinite(p).sum() == 1022
        m = opt.m.float()
        assert torch.isnan(m[3]) and torch.isfinite(m[4:256]).all()
        assert torch.isfinite(m[768:]).all() and torch.isfinite(m[256:512]).all()


def test_adamw_refuses_tensors(dev):
    from demand_side_expert_gb300 import AdamW

    p, g = torch.zeros(64, device=dev), torch.zeros(64, device=dev)
    for ps, gs, kw in (([p], [], {}), ([p.half()], [g], {}), ([p], [g.half()], {}),
                       ([p], [g[:32]], {}), ([p[::2]], [g[::2]], {}), ([p], [g.cpu()], {}),
                       ([p], [g], dict(state="f4")), ([p], [g], dict(betas=(1.0, 0.9))),
                       ([p], [g], dict(weight_decay=[0.1, 0.2]))):
        with pytest.raises(ValueError):
            AdamW(ps, gs, **kw)
    from demand_side_expert_gb300 import lrm
    with pytest.raises(lrm.LrmError):  # 16-byte alignment
        AdamW([torch.zeros(65, device=dev)[1:]], [g]).step()
    with pytest.raises(ValueError):
        AdamW([p], [g]).step(grad_scale=torch.zeros(2, device=dev))


def test_adamw_past_2_31_elements(dev):
    from demand_side_expert_gb300 import AdamW

    n = (1 << 31) + 4099
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g[-300:] = 1.0
    g[5] = -1.0
    opt = AdamW([p], [g], lr=0.25, weight_decay=0.0, state="f8")
    opt.step()
    assert (p[-300:] == -0.25).all() and p[5] == 0.25
    assert p[6:-300].count_nonzero() == 0
    assert (opt.m[n - 300:n].float() == 448).all()
