"""The float64 oracle of the operators for training under tight memory against central
differences, closed forms and hand-worked rows; and the library's refusals, which return
before any launch (no GPU)."""

import ctypes
import os

import numpy as np
import pytest

from oracle import memory_oracle as mo

# central differences in float64 with step 1e-6: truncation ~1e-12 times the third
# derivative, rounding ~1e-16 / 1e-6 = 1e-10 times the value
FD_STEP, FD_TOL = 1e-6, 1e-7


@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K,off", [(1, 1, 1, 0), (3, 4, 2, 0), (6, 12, 5, 0.3)])
def test_router_gradient_matches_differences(T, E, K, off, renorm, fn):
    rng = np.random.default_rng(T * 100 + E)
    x = rng.standard_normal((T, E)) * 1.5
    x[rng.random((T, E)) < off] = -np.inf
    mask = np.ones(T, dtype=np.uint8)
    if T > 3:
        mask[1] = 0
        x[2] = -np.inf
    dalpha, bias = rng.standard_normal((T, K)), rng.standard_normal(E) * 0.1
    kw = dict(fn=fn, renorm=renorm, scale=1.7, balance_coef=0.5, mask=mask)
    ref = mo.group_route(x, K, bias=bias, groups=1, **kw)
    got = mo.group_route_bwd(x, ref["topk_idx"], ref["counts"], dalpha, 1.3, **kw)

    def total(z):
        r = mo.group_route(z, K, idx=ref["topk_idx"], **kw)
        return (r["alpha"] * dalpha).sum() + 1.3 * r["loss"][0]

    for t in range(T):
        for e in range(E):
            if not np.isfinite(x[t, e]):
                assert got[t, e] == 0
                continue
            d = np.zeros_like(x)
            d[t, e] = FD_STEP
            fd = (total(x + d) - total(x - d)) / (2 * FD_STEP)
            assert abs(fd - got[t, e]) <= FD_TOL * (1 + abs(fd)), (t, e)


def test_choices_by_hand():
    # 2 groups of 3; scores are sigmoid(0) = 1/2 but for the named ones
    x = np.array([[2.0, 0.0, 0.0, 1.0, 1.0, -5.0]])
    # pairs: sigma(2) + sigma(0) = 1.38, sigma(1) + sigma(1) = 1.46: the second group
    assert mo.choose(x, 2, groups=2, top_groups=1, group_top=2).tolist() == [[3, 4]]
    assert mo.choose(x, 2, groups=2, top_groups=1, group_top=1).tolist() == [[0, 1]]
    assert mo.choose(x, 3, groups=2, top_groups=2).tolist() == [[0, 3, 4]]
    # a bias moves the choice and not the weight
    bias = np.array([0.0, 0.0, 0.5, 0.0, 0.0, 0.0])
    r = mo.group_route(x, 1, bias=bias, groups=2, top_groups=1, renorm=False)
    assert r["topk_idx"].tolist() == [[2]] and r["alpha"][0, 0] == 0.5
    # closed experts: the first group has one open expert left, 0.88 against 1.46
    x[0, 1:3] = -np.inf
    assert mo.choose(x, 2, groups=2, top_groups=2).tolist() == [[0, 3]]
    assert mo.choose(x, 3, groups=2, top_groups=1, group_top=1).tolist() == [[0, 1, 2]]
    # nothing open: ids stay valid and distinct, weights and counts are 0
    r = mo.group_route(np.full((2, 4), -np.inf), 2, groups=2, top_groups=1, balance_coef=1.0)
    assert r["topk_idx"].tolist() == [[0, 1], [0, 1]] and (r["alpha"] == 0).all()
    assert (r["counts"] == 0).all() and (r["loss"] == 0).all()


def test_router_closed_forms():
    T, E, K = 6, 8, 2
    r = mo.group_route(np.zeros((T, E)), K, balance_coef=3.0, scale=2.0)
    assert np.allclose(r["alpha"], 1.0) and np.isclose(r["loss"][0], 3.0)
    assert np.allclose(r["share"], 1 / E) and (r["s"] == 0.5).all()
    # very low logits: the shares and the renormalised weights are a softmax's
    x = np.array([[-900.0, -901.0, -902.0]])
    r = mo.group_route(x, 2)
    p = np.exp([0.0, -1.0, -2.0])
    assert np.allclose(r["share"], p / p.sum()) and np.allclose(r["alpha"], p[:2] / p[:2].sum())
    assert mo.bias_step([0.0, 0.0, 0.5], [1, 2, 3], 0.1).tolist() == [0.1, 0.0, 0.4]


def test_pack_by_hand():
    ab = np.zeros((1, 16))
    ab[0, :3] = [448.0, 1.0, -0.3]
    ab[0, 8:10] = [0.0, 2.0 ** -10 * 448]
    q, scale, sq = mo.pack(ab, 32)
    assert scale[0, 0] == 1.0 and q[0, 0] == 448 and q[0, 1] == 1 and q[0, 2] == -0.3125
    assert scale[0, 1] == 2.0 ** -10 and q[0, 9] == 448
    phi = ab[0, 1] / (1 + np.exp(-1.0)) * ab[0, 9]
    assert np.isclose(sq[0], phi ** 2)
    back, f = mo.unpack(q, scale, 32)
    assert np.array_equal(back[0, [0, 1, 9]], ab[0, [0, 1, 9]]) and np.isclose(f[0, 1], phi)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind", [None, "column", "token"])
def test_block_norm_gradient_matches_differences(kind, post):
    rng = np.random.default_rng(4)
    T, D = 3, 16
    v = {"block": rng.standard_normal((T, D)), "res": rng.standard_normal((T, D)),
         "w": rng.standard_normal(D)}
    if post:
        v["w_post"] = rng.standard_normal(D)
    if kind:
        v["gate"] = rng.standard_normal(D if kind == "column" else T)
    dy, dh = rng.standard_normal((T, D)), rng.standard_normal((T, D))
    kw = dict(gate_kind=kind, res_scale=0.7, eps=1e-5)
    f = mo.block_norm(**v, **kw)
    g = mo.block_norm_bwd(dy, dh, f["h"], v["block"], v["w"], f["rstd"], v.get("w_post"),
                          v.get("gate"), kind, f.get("block_rstd"), 0.7)

    def total(**change):
        r = mo.block_norm(**{**v, **change}, **kw)
        return (r["y"] * dy).sum() + (r["h"] * dh).sum()

    for name, grad in (("block", "dblock"), ("res", "dres"), ("w", "dw"), ("w_post", "dw_post"),
                       ("gate", "dgate")):
        if name not in v:
            assert grad not in g
            continue
        for at in np.ndindex(v[name].shape):
            e = np.zeros_like(v[name])
            e[at] = FD_STEP
            fd = (total(**{name: v[name] + e}) - total(**{name: v[name] - e})) / (2 * FD_STEP)
            assert abs(fd - g[grad][at]) <= 10 * FD_TOL * (1 + abs(fd)), (name, at)


# -- refusals -----------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from demand_side_expert_gb300 import build as b

    if not os.path.exists(b.LIB):
        b.build()
    from demand_side_expert_gb300 import lrm

    return lrm


def _router(lib, **kw):
    v = dict(T=4, E=16, K=2, dtype=lib.LRM_F32, stride=16, score_fn=0, groups=4, top_groups=2,
             group_top=2, renorm=1, scale=1.0, balance_coef=0.1)
    v.update(kw)
    return lib.lrm_group_router(*v.values())


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), "bad"), (dict(E=0), "bad"), (dict(K=0), "bad"), (dict(groups=0), "bad"),
    (dict(top_groups=0), "bad"), (dict(group_top=0), "bad"), (dict(dtype=7), "bad"),
    (dict(score_fn=2), "bad"), (dict(stride=15), "bad"), (dict(group_top=3), "no"),
    (dict(groups=3), "no"), (dict(top_groups=5), "no"), (dict(K=9), "no"),
    (dict(E=2048, stride=2048), "no"), (dict(E=128, stride=128, groups=64), "no"),
    (dict(E=128, stride=128, K=33, groups=1, top_groups=1), "no"), (dict(T=1 << 30), "no")])
def test_router_refuses(lib, bad, want):
    want = lib.LRM_ERR_INVALID_ARG if want == "bad" else lib.LRM_ERR_UNSUPPORTED
    r = _router(lib, **bad)
    assert lib.lrm_group_router_workspace_bytes(r) == 0
    b = ctypes.byref(r)
    assert lib._lib.lrm_group_route(b, *[256] * 9, 1 << 30, None) == want
    assert lib._lib.lrm_group_route_bwd(b, *[256] * 8, 1 << 30, None) == want


def test_router_refuses_pointers(lib):
    r = _router(lib)
    b, n = ctypes.byref(r), lib.lrm_group_router_workspace_bytes(r)
    f, g = lib._lib.lrm_group_route, lib._lib.lrm_group_route_bwd
    bad, no, short = lib.LRM_ERR_INVALID_ARG, lib.LRM_ERR_UNSUPPORTED, lib.LRM_ERR_WORKSPACE
    # logits, bias, mask, topk_idx, alpha, counts, prob_sum, loss, ws
    assert f(b, 256, None, None, 256, 256, None, None, None, None, n, None) == short
    assert f(b, 256, None, None, 256, 256, None, None, None, 256, n - 1, None) == short
    assert f(b, 256, None, None, 256, 256, None, None, None, 264, n, None) == no
    assert f(b, 256, None, None, 256, 256, 256, None, 256, 256, n, None) == bad
    assert f(b, None, None, None, 256, 256, None, None, None, 256, n, None) == bad
    assert f(b, 264, None, None, 256, 256, None, None, None, 256, n, None) == no
    assert f(b, 256, 258, None, 256, 256, None, None, None, 256, n, None) == no
    # logits, mask, topk_idx, counts, dalpha, dloss, dlogits, ws
    assert g(b, 256, None, None, 256, 256, None, 256, 256, n, None) == bad
    assert g(b, 256, None, 256, 256, 264, None, 256, 256, n, None) == no
    assert g(b, 256, None, 256, 256, 256, 257, 256, 256, n, None) == no
    s = lib.lrm_bias(16, 0.1)
    step = lib._lib.lrm_bias_step
    assert step(None, 256, 256, 256, None) == bad
    assert step(ctypes.byref(s), 256, None, 256, None) == bad
    assert step(ctypes.byref(s), 256, 256, 258, None) == no
    assert step(ctypes.byref(lib.lrm_bias(0, 0.1)), 256, 256, 256, None) == bad
    assert step(ctypes.byref(lib.lrm_bias(2000, 0.1)), 256, 256, 256, None) == no


def _packed(lib, **kw):
    v = dict(q=256, scale=256, phi_sq=256, rows=8, H=64, cols=64, dtype=lib.LRM_BF16, reserved=0)
    v.update(kw)
    return lib.lrm_packed(*v.values())


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), "bad"), (dict(H=0), "bad"), (dict(dtype=3), "bad"), (dict(q=None), "bad"),
    (dict(scale=None), "bad"), (dict(phi_sq=None), "bad"), (dict(H=60), "no"),
    (dict(cols=256), "no"), (dict(cols=0), "no"), (dict(q=264), "no"), (dict(rows=1 << 31), "no")])
def test_packed_state_refuses(lib, bad, want):
    want = lib.LRM_ERR_INVALID_ARG if want == "bad" else lib.LRM_ERR_UNSUPPORTED
    p = ctypes.byref(_packed(lib, **bad))
    assert lib._lib.lrm_pack_state(p, 256, None) == want
    s = lib.make_shape(4, 64, 64, 8, 2, lib.LRM_BF16)
    n = lib.lrm_workspace_bytes(s)
    assert lib._lib.lrm_score_packed(ctypes.byref(s), p, *[256] * 5, n, None) == want
    assert lib._lib.lrm_compact_packed(ctypes.byref(s), p, *[256] * 7, 0, *[256] * 8, n,
                                       None) == want


def test_packed_state_refuses_other_layers_and_pointers(lib):
    bad, no, short = lib.LRM_ERR_INVALID_ARG, lib.LRM_ERR_UNSUPPORTED, lib.LRM_ERR_WORKSPACE
    s = lib.make_shape(4, 64, 64, 8, 2, lib.LRM_BF16)
    b, n = ctypes.byref(s), lib.lrm_workspace_bytes(s)
    score, compact = lib._lib.lrm_score_packed, lib._lib.lrm_compact_packed
    for other in (dict(rows=6), dict(H=128), dict(dtype=lib.LRM_F32)):
        p = ctypes.byref(_packed(lib, **other))
        assert score(b, p, *[256] * 5, n, None) == bad
        assert compact(b, p, *[256] * 7, 0, *[256] * 8, n, None) == bad
    p = ctypes.byref(_packed(lib))
    assert lib._lib.lrm_pack_state(p, None, None) == bad
    assert lib._lib.lrm_pack_state(p, 264, None) == no
    assert lib._lib.lrm_pack_state(None, 256, None) == bad
    assert score(b, p, 256, 256, 256, 256, None, n, None) == short
    assert score(b, p, 256, 256, 256, None, 256, n, None) == bad
    assert score(b, p, 264, 256, 256, 256, 256, n, None) == no
    # perm, keep, sel_off, sel_pos, alpha, x, x_scale, x_cols, g, dy_c, x_c, ab_c, phi_c, ..
    args = [256] * 7 + [48] + [256] * 8
    assert compact(b, p, *args, n, None) == no  # x_cols
    args[7], args[5] = 0, None
    assert compact(b, p, *args, n, None) == bad  # x_c without x
    args[5], args[11] = 256, None
    assert compact(b, p, *args, n, None) == bad  # ab_c
    args[11], args[8] = 256, 264
    assert compact(b, p, *args, n, None) == no  # g
    f = lib._lib.lrm_expert_bwd_compacted
    assert f(b, *[256] * 17, None, n, None) == short
    assert f(b, 256, None, *[256] * 16, n, None) == bad  # tok_c


def _block(lib, **kw):
    v = dict(T=4, D=64, dtype=lib.LRM_BF16, block_dtype=lib.LRM_F32, grad_dtype=lib.LRM_F32,
             gate=0, q_cols=0, eps=1e-6, residual_scale=1.0, block_stride=64, res_stride=64)
    v.update(kw)
    return lib.lrm_block(*v.values())


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), "bad"), (dict(D=0), "bad"), (dict(dtype=5), "bad"), (dict(gate=3), "bad"),
    (dict(eps=-1.0), "bad"), (dict(eps=float("nan")), "bad"), (dict(block_stride=56), "bad"),
    (dict(res_stride=32), "bad"), (dict(q_cols=-1), "bad"), (dict(grad_dtype=4), "bad"),
    (dict(D=60, block_stride=60, res_stride=60), "no"), (dict(q_cols=48), "no"),
    (dict(D=8200, block_stride=8200, res_stride=8200), "no"), (dict(block_stride=68), "no"),
    (dict(dtype=0, block_dtype=1), "no")])
def test_block_norm_refuses(lib, bad, want):
    want = lib.LRM_ERR_INVALID_ARG if want == "bad" else lib.LRM_ERR_UNSUPPORTED
    d = _block(lib, **bad)
    assert lib.lrm_block_workspace_bytes(d) == 0
    b = ctypes.byref(d)
    assert lib._lib.lrm_block_norm(b, *[256] * 11, None) == want
    assert lib._lib.lrm_block_norm_bwd(b, *[256] * 15, 1 << 30, None) == want


def test_block_norm_refuses_pointers(lib):
    bad, no, short = lib.LRM_ERR_INVALID_ARG, lib.LRM_ERR_UNSUPPORTED, lib.LRM_ERR_WORKSPACE
    d = _block(lib)
    b, n = ctypes.byref(d), lib.lrm_block_workspace_bytes(d)
    f, g = lib._lib.lrm_block_norm, lib._lib.lrm_block_norm_bwd
    # block, res, w, w_post, gate, h, y, q, q_scale, rstd, block_rstd
    ok = [256, 512, 256, 256, None, 256, 256, None, None, 256, 256]

    def fwd(desc=b, **change):
        a = list(ok)
        for i, v in change.items():
            a[int(i[1:])] = v
        return f(desc, *a, None)

    assert fwd(_0=None) == bad and fwd(_1=None) == bad and fwd(_2=None) == bad
    assert fwd(_5=None) == bad and fwd(_6=None) == bad  # h; no output
    assert fwd(_7=256) == bad  # q without scales
    assert fwd(_4=256) == bad  # a gate where there is none
    assert fwd(ctypes.byref(_block(lib, gate=1))) == bad  # none where there is one
    assert fwd(ctypes.byref(_block(lib, gate=1)), _4=260) == no
    assert fwd(_0=264) == no and fwd(_3=264) == no
    wide = ctypes.byref(_block(lib, res_stride=128))
    assert fwd(wide, _5=512) == bad  # h over rows that are not contiguous
    # dy, dh, h, block, w, w_post, gate, rstd, block_rstd, dres, dblock, dw, dw_post, dgate, ws
    back = [256] * 6 + [None] + [256] * 6 + [None, 256]

    def bwd(desc=b, size=n, **change):
        a = list(back)
        for i, v in change.items():
            a[int(i[1:])] = v
        return g(desc, *a, size, None)

    assert bwd(_14=None) == short and bwd(size=n - 1) == short
    for i in (0, 2, 3, 4, 7, 8, 9, 10, 11, 12):
        assert bwd(**{f"_{i}": None}) == bad, i
    assert bwd(_0=264) == no and bwd(_14=264) == no
    assert bwd(ctypes.byref(_block(lib, gate=2)), _6=256) == bad  # no dgate


def test_python_classes_refuse_on_the_host():
    from demand_side_expert_gb300 import BlockNorm, GroupRouter, PackedState

    for kw in (dict(E=2048), dict(groups=3), dict(K=20), dict(score="relu"), dict(group_top=3),
               dict(groups=8, top_groups=9), dict(groups=8, top_groups=0), dict(device="cpu")):
        with pytest.raises(ValueError):
            GroupRouter(**{**dict(T=4, E=16, K=2), **kw})
    for kw in (dict(H=60), dict(cols=100), dict(K=0), dict(device="cpu"), dict(T=-1)):
        with pytest.raises(ValueError):
            PackedState(**{**dict(T=4, K=2, H=64), **kw})
    for kw in (dict(D=30), dict(D=8200), dict(gate="row"), dict(q_cols=48), dict(eps=-1.0),
               dict(dtype="f32", block_dtype="bf16"), dict(store_y=False), dict(device="cpu")):
        with pytest.raises(ValueError):
            BlockNorm(**{**dict(T=4, D=64), **kw})
