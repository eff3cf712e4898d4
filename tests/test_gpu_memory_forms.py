"""GPU tests of the operators for training under tight memory in the forms that only large
blocks take, against the float64 oracle. Sizes are counted from the device's SMs, as the
choice of a form is; tolerances are those of test_gpu_memory_ops.
"""

import math

import numpy as np
import pytest
import torch

from oracle import memory_oracle as mo
from test_gpu_memory_ops import (BF16, DT, TINY, U, close, dev, make_bias,  # noqa: F401
                                 make_logits, router, score_tol, to64)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# -- router -------------------------------------------------------------------
def check_routed(dev, x, K, fn, bias, groups, top, gt, renorm, mask=None):
    """Choices, weights and statistics of a block of tokens; those without statistics too."""
    T, E = x.shape
    dtype = "bf16" if x.dtype is torch.bfloat16 else "f32"
    kw = dict(score=fn, groups=groups, top_groups=top, group_top=gt, renorm=renorm, scale=1.7)
    r = router(T, E, K, dtype, balance_coef=0.3, **kw)
    b = None if bias is None else bias.to(dev)
    m = None if mask is None else torch.as_tensor(mask, dtype=torch.uint8, device=dev)
    r.route(x.to(dev), bias=b, mask=m)
    serve = router(T, E, K, dtype, **kw)
    serve.route(x.to(dev), bias=b, mask=m, stats=False)
    x64 = to64(x)
    args = (K, fn, None if bias is None else to64(bias), groups, top, gt)
    ids = mo.choose_rows(x64, *args)
    ends = np.r_[:40, T - 40:T]
    assert np.array_equal(ids[ends], mo.choose(x64[ends], *args))
    ref = mo.group_route(x64, K, fn, renorm=renorm, scale=1.7, balance_coef=0.3, mask=mask, idx=ids)
    assert np.array_equal(r.topk_idx.cpu().numpy(), ids)
    tol = score_tol(x64)
    close(to64(r.alpha), ref["alpha"], (2 * tol + K * U) * np.abs(ref["alpha"]) + TINY, "alpha")
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    close(to64(r.prob_sum), ref["prob_sum"], (tol + (T + 8) * U) * ref["prob_sum"] + TINY,
          "prob_sum")
    close(to64(r.loss), ref["loss"], (2 * tol + (T + E + 16) * U) * ref["loss"], "loss")
    assert torch.equal(serve.topk_idx, r.topk_idx) and torch.equal(serve.alpha, r.alpha)
    assert r.device_error() == 0


def large_block(E):
    """Tokens from which on lists of experts are merged across tokens, and a few more."""
    return 50 * sms() + 3 if E > 128 else 100 * sms() + 5


def routed_rows(E, dtype, kind, off):
    T = large_block(E)
    x = make_logits(T, E, dtype, E + len(kind), off=off, kind=kind)
    x[2] = -math.inf  # nothing to choose from
    x[3, 1:] = -math.inf  # one open expert
    x[T - 1] = -math.inf
    return x, (np.random.default_rng(E).random(T) < 0.8).astype(np.uint8)


@pytest.mark.parametrize("E,groups,dtype,fn", [
    (256, 32, "f32", "sigmoid"), (200, 25, "bf16", "softmax"), (128, 16, "f32", "softmax"),
    (100, 10, "bf16", "sigmoid")])
def test_router_keeps_all_groups(dev, E, groups, dtype, fn):  # noqa: F811
    """top_groups is groups, of fewer experts than a lane holds: one group of all."""
    x, mask = routed_rows(E, dtype, "equal", 0.1)
    check_routed(dev, x, 8, fn, make_bias(E, "steps"), groups, groups, 2, True, mask)


# E, K, groups, top, group_top, dtype, fn, bias, kind, renorm, off. Not a bias on sigmoids of
# 1 but for 64 bits' last place, where the larger of two is a matter of the formula's rounding.
MERGED = [
    (256, 8, 8, 4, 2, "f32", "sigmoid", "steps", "normal", True, 0.0),
    (256, 8, 8, 4, 2, "bf16", "softmax", None, "equal", False, 0.1),
    (256, 5, 8, 4, 1, "f32", "softmax", "zero", "near", True, 0.0),
    (256, 8, 16, 5, 2, "bf16", "sigmoid", None, "equal", True, 0.0),
    (256, 1, 4, 1, 2, "f32", "sigmoid", None, "low", True, 0.0),
    (256, 8, 8, 3, 2, "f32", "sigmoid", None, "high", False, 0.0),
    (256, 7, 2, 1, 1, "f32", "softmax", None, "one", True, 0.0),
    (256, 8, 1, 1, 2, "bf16", "softmax", "steps", "low", False, 0.0),
    (200, 8, 1, 1, 2, "bf16", "sigmoid", "steps", "normal", True, 0.9),
    (200, 3, 1, 1, 1, "f32", "softmax", None, "near", False, 0.0),
    (192, 6, 12, 5, 2, "f32", "sigmoid", "zero", "equal", False, 0.2),
    (192, 8, 3, 2, 2, "bf16", "softmax", "random", "low", True, 0.0),
    (240, 8, 15, 7, 1, "f32", "sigmoid", "steps", "near", True, 0.0),
    (128, 8, 8, 3, 2, "f32", "sigmoid", None, "low", False, 0.1),
    (128, 8, 4, 2, 1, "bf16", "softmax", None, "normal", False, 0.1),
    (128, 4, 2, 1, 2, "f32", "softmax", "steps", "equal", True, 0.0),
    (128, 8, 8, 4, 1, "f32", "sigmoid", "random", "near", True, 0.9),
    (100, 5, 1, 1, 2, "bf16", "sigmoid", None, "equal", True, 0.0),
    (100, 8, 1, 1, 1, "f32", "softmax", "zero", "low", False, 0.0),
    (96, 2, 6, 3, 1, "bf16", "sigmoid", "steps", "normal", False, 0.9),
    (96, 8, 3, 2, 2, "f32", "softmax", None, "one", True, 0.0),
    (80, 1, 5, 2, 2, "f32", "sigmoid", "random", "normal", True, 0.0),
]


@pytest.mark.parametrize("E,K,groups,top,gt,dtype,fn,bias,kind,renorm,off", MERGED)
def test_router_merges_lists_across_tokens(dev, E, K, groups, top, gt, dtype, fn,  # noqa: F811
                                           bias, kind, renorm, off):
    x, mask = routed_rows(E, dtype, kind, off)
    check_routed(dev, x, K, fn, make_bias(E, bias, E), groups, top, gt, renorm, mask)


FORMS = [  # tokens a SM (0: 6 in all), E, K, groups, top
    (0, 16, 3, 4, 2), (0, 256, 8, 8, 4),  # a warp a token, lists of 8
    (25, 32, 3, 4, 2), (25, 64, 8, 4, 2), (25, 256, 8, 8, 4),  # tokens that share a warp
    (50, 256, 8, 8, 4), (50, 200, 3, 1, 1), (100, 128, 8, 4, 2),  # and merge their lists
    (0, 64, 12, 4, 2), (3, 320, 6, 8, 3), (3, 200, 8, 25, 5),  # a warp a token, one maximum each
]


@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [None, "steps"])
@pytest.mark.parametrize("per_sm,E,K,groups,top", FORMS)
def test_router_nan_and_inf_in_every_form(dev, per_sm, E, K, groups, top, bias, fn):  # noqa: F811
    """NaN and infinities reach the outputs of their own tokens, and of masked ones nothing;
    every row's ids are valid, distinct and of the kept groups."""
    T = per_sm * sms() + 6
    clean = make_logits(T, E, "f32", E)
    hit = torch.arange(T) % 5 == 1  # a lane group's neighbours are clean
    nan_rows, all_nan = torch.nonzero(hit)[:, 0], torch.nonzero(torch.arange(T) % 5 == 4)[:, 0]
    dirty = clean.clone()
    dirty[nan_rows, 1] = math.nan
    dirty[all_nan] = math.nan
    out = torch.zeros(T, dtype=torch.bool)
    out[nan_rows] = out[all_nan] = True
    mask = (~out).to(dev)
    b = None if bias is None else make_bias(E, bias).to(dev)
    da = torch.ones(T, K, device=dev)
    da[out.to(dev)] = math.nan
    size = E // groups

    def routed(x, m, **kw):
        r = router(T, E, K, "f32", score=fn, groups=groups, top_groups=top, balance_coef=1.0, **kw)
        r.route(x.to(dev), bias=b, mask=m)
        ids = r.topk_idx.cpu().long()
        assert ids.min() >= 0 and ids.max() < E
        assert (ids.sort(1)[0].diff(dim=1) > 0).all()
        kept = (ids // size).sort(1)[0]
        assert ((kept.diff(dim=1) > 0).sum(1) < top).all()
        return r

    got = [routed(x, mask) for x in (clean, dirty)]
    for r, x in zip(got, (clean, dirty)):
        r.backward(x.to(dev), da, mask=mask)
        assert torch.isfinite(r.dlogits).all() and (r.dlogits[out.to(dev)] == 0).all()
    for name in ("alpha", "counts", "prob_sum", "loss", "dlogits"):
        assert torch.equal(getattr(got[0], name), getattr(got[1], name)), name
    assert torch.equal(got[0].topk_idx[mask], got[1].topk_idx[mask])
    r = routed(dirty, None)
    alone = routed(clean, None)
    assert torch.isnan(r.prob_sum).all() and torch.isnan(r.loss).all()
    assert torch.equal(r.alpha[mask], alone.alpha[mask])
    assert torch.equal(r.topk_idx[mask], alone.topk_idx[mask])
    if fn == "softmax":
        assert torch.isnan(r.alpha[out.to(dev)]).all()
    else:  # NaN comes last: numbers are there to choose, and a row of NaN alone has none
        assert torch.isfinite(r.alpha[nan_rows.to(dev)]).all()
        assert (r.topk_idx[nan_rows.to(dev)] != 1).all()
        assert torch.isnan(r.alpha[all_nan.to(dev)]).all()
        x = clean.clone()
        x[nan_rows, E - 1] = math.inf  # a score of 1, and without a bias the largest key
        r = routed(x, None, renorm=False)
        assert torch.isfinite(r.prob_sum).all() and torch.isfinite(r.alpha).all()
        ids = mo.choose(to64(x[:12]), K, fn, None if b is None else to64(b), groups, top, 2)
        assert np.array_equal(r.topk_idx[:12].cpu().numpy(), ids[:T])


# -- rows rebuilt from 8 bits ---------------------------------------------------
def compacted(dev, T, K, D, H, E, dtype, x_cols, seed):
    """compact of random pairs of uneven experts, all and two thirds of them: each retained row
    is its pair's. dy, a, b and the rows of an 8-bit x are one rounded product each, bit for bit;
    phi is within the formula's own roundings."""
    from demand_side_expert_gb300 import PackedState, RecalibratedExpertBackward

    tdtype, N = DT[dtype], T * K
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    ids = torch.rand(T, E, generator=gen, device=dev)
    ids = (ids ** torch.arange(1, E + 1, device=dev)).topk(K, dim=1)[1].to(torch.int32)
    pipe = RecalibratedExpertBackward(T, D, H, E, K, dtype, dev)
    pipe.dispatch(ids)
    state = PackedState(T, K, H, dtype, cols=32)
    state.pack(randn(N, 2 * H).to(tdtype))
    alpha, g, x = torch.rand(T, K, generator=gen, device=dev), randn(T, D).to(tdtype), randn(T, D)
    if x_cols is None:
        x = x_rows = x.to(tdtype)
    else:
        groups = -(-D // x_cols) if x_cols else 1
        scale = torch.rand(T, groups, generator=gen, device=dev) + 0.5
        q = x.to(torch.float8_e4m3fn)
        x_rows = (q.float() * scale.repeat_interleave(x_cols or D, 1)[:, :D]).to(tdtype)
        x = (q, scale)
    wide = state.scale.view(N, 2, -1).repeat_interleave(32, 2)[:, :, :H].reshape(N, 2 * H)
    ab = state.q.float() * wide
    a, b = ab[:, :H].double(), ab[:, H:].double()
    phi = a / (1 + torch.exp(-a)) * b
    half = BF16 if dtype == "bf16" else 0.0
    lim = (half + (2 * a.abs() + 12) * U) * phi.abs() + TINY
    pipe.score_pairs(alpha, g, state)
    for rate in ((1, 1), (2, 3)):
        pipe.select_rate(*rate)
        for t in (pipe.dy_c, pipe.x_c, pipe.ab_c, pipe.phi_c):
            t.fill_(math.nan)
        pipe.tok_c.fill_(-5)
        pipe.compact(alpha, x, g, state, None)
        assert pipe.device_error() == 0
        M = pipe.retained_rows
        assert M == N or rate != (1, 1)
        pos = pipe.sel_pos[:M].long()
        pair = pipe.perm[pos].long()
        tok = pair // K
        assert torch.equal(pipe.tok_c[:M].long(), tok)
        assert torch.equal(pipe.row_of_pos[pos].long(), torch.arange(M, device=dev))
        assert int((pipe.row_of_pos[:N] >= 0).sum()) == M
        assert torch.equal(pipe.x_c[:M], x_rows[tok])
        assert torch.equal(pipe.dy_c[:M], (alpha.view(-1)[pair][:, None] * g[tok].float()).to(tdtype))
        assert torch.equal(pipe.ab_c[:M], ab[pos].to(tdtype))
        assert ((pipe.phi_c[:M].double() - phi[pos]).abs() <= lim[pos]).all()


@pytest.mark.parametrize("more", [-1, 0, 1, 7])
@pytest.mark.parametrize("rounds", [2, 3])
@pytest.mark.parametrize("lanes,D,H,dtype", [(8, 16, 8, "f32"), (8, 256, 64, "bf16"),
                                             (16, 256, 72, "f32"), (16, 24, 256, "bf16"),
                                             (32, 264, 8, "f32"), (32, 64, 264, "bf16")])
def test_packed_rows_in_whole_rounds(dev, lanes, D, H, dtype, rounds, more):  # noqa: F811
    """As many rows as the teams of lanes take in whole rounds, a few more or less."""
    teams = sms() * 4 * (256 // lanes)
    compacted(dev, rounds * teams + more, 1, D, H, 61, dtype, None, rounds)


@pytest.mark.parametrize("more", [-1, 0, 1])
@pytest.mark.parametrize("K,E,x_cols", [(4, 60, None), (8, 60, 128), (4, 28, 0), (2, 121, 32)])
def test_packed_rows_met_by_segments(dev, K, E, x_cols, more):  # noqa: F811
    """32 MB of cotangents whose tokens' rows are shared by K pairs: about as many rows as are
    dealt out in whole rounds, x in the layer's type or in 8 bits."""
    deal = sms() * 32 - E - 8
    tokens = -(-8192 * K // deal) * deal // K + more  # 32 MB of rows of 4096 bytes at least
    compacted(dev, tokens, K, 2048, 40, E, "bf16", x_cols, K)
    compacted(dev, -(-2048 * K // deal) * deal // K + more, K, 4096, 8, E, "f32", x_cols, K)


@pytest.mark.parametrize("T,K,D,H,E,dtype,x_cols", [
    (20001, 2, 64, 48, 28, "bf16", 0), (10001, 2, 256, 256, 9, "f32", 64),
    (3001, 4, 264, 520, 64, "f32", 256), (33, 3, 1032, 264, 17, "bf16", 128)])
def test_packed_rows_beside_8_bit_rows(dev, T, K, D, H, E, dtype, x_cols):  # noqa: F811
    compacted(dev, T, K, D, H, E, dtype, x_cols, T)


@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_sm,E,K", [(0, 16, 2), (0, 64, 8), (25, 64, 4), (25, 128, 8),
                                        (25, 256, 8), (50, 256, 8), (100, 128, 2), (0, 600, 20)])
def test_router_shares_of_low_rows(dev, per_sm, E, K, dtype, fn):  # noqa: F811
    """Rows whose largest logit is -21 to -69 and whose others are up to 60 below: every share
    keeps its own accuracy, in the statistics and in the gradient, however small its score."""
    T = per_sm * sms() + 100
    gen = torch.Generator().manual_seed(E)
    top = -21 - 48 * torch.rand(T, 1, generator=gen)
    below = 60 * torch.rand(1, E, generator=gen) + 0.5 * torch.rand(T, E, generator=gen)
    x = (top - below).to(DT[dtype])
    r = router(T, E, K, dtype, score=fn, balance_coef=1.0)
    r.route(x.to(dev))
    x64 = to64(x)
    kw = dict(fn=fn, balance_coef=1.0)
    ref = mo.group_route(x64, K, idx=mo.choose_rows(x64, K, fn), **kw)
    assert np.array_equal(r.topk_idx.cpu().numpy(), ref["topk_idx"])
    tol = score_tol(x64)
    close(to64(r.prob_sum), ref["prob_sum"], (tol + (T + 8) * U) * ref["prob_sum"] + TINY,
          "prob_sum")
    r.backward(x.to(dev))
    assert r.device_error() == 0
    some = np.r_[:60, T - 60:T] if T > 120 else np.arange(T)
    want = mo.group_route_bwd(x64[some], ref["topk_idx"][some], ref["counts"], None, **kw)
    cost = E * ref["counts"] / (float(T) * T * K)
    mag = ref["share"][some] * (cost + ref["share"][some] @ cost[:, None])
    lim = (4 * tol + (E + 24) * U) * mag + (BF16 * np.abs(want) if dtype == "bf16" else 0)
    close(to64(r.dlogits)[some], want, lim + TINY, "dlogits")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_sm,E,K", [(0, 64, 8), (25, 128, 8), (50, 256, 8), (100, 128, 3),
                                        (0, 600, 20)])
def test_router_weights_of_low_rows(dev, per_sm, E, K, dtype):  # noqa: F811
    """One choice of a score of 1e-9 to 1e-26, the others 40 to 45 below it: each weight keeps
    its own accuracy."""
    T = per_sm * sms() + 100
    gen = torch.Generator().manual_seed(E)
    top = -21 - 39 * torch.rand(T, 1, generator=gen)
    x = top - 40 - 5 * torch.rand(T, E, generator=gen)
    x.scatter_(1, torch.randint(0, E, (T, 1), generator=gen), top)
    x = x.to(DT[dtype])
    r = router(T, E, K, dtype, score="sigmoid", renorm=True)
    r.route(x.to(dev), stats=False)
    x64 = to64(x)
    ids = mo.choose_rows(x64, K)
    ref = mo.group_route(x64, K, idx=ids)
    assert np.array_equal(r.topk_idx.cpu().numpy(), ids)
    lim = (2 * score_tol(x64) + K * U) * ref["alpha"]
    close(to64(r.alpha), ref["alpha"], lim + TINY, "alpha")
