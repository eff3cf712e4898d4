"""The float64 oracle of the training-step operators against central differences of
its own losses, closed forms and brute force; and the host side of the operators:
refused arguments return before any launch (no GPU)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import step_oracle as so


def _logits(rng, T, E, off=0.0):
    x = rng.standard_normal((T, E)) * 1.5
    if off:
        x[rng.random((T, E)) < off] = -np.inf
    return x


# central differences of a smooth function in float64 with step 1e-6: truncation
# ~1e-12 times the third derivative, rounding ~1e-16 / 1e-6 = 1e-10 times the value
FD_STEP, FD_TOL = 1e-6, 1e-7


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K,off", [(1, 1, 1, 0), (3, 4, 2, 0), (7, 12, 5, 0.3), (5, 6, 6, 0)])
def test_router_gradient_matches_differences(T, E, K, off, renorm):
    rng = np.random.default_rng(T * 100 + E)
    x = _logits(rng, T, E, off)
    mask = np.ones(T, dtype=np.uint8)
    if T > 3:
        mask[1] = 0
        x[2] = -np.inf
    dalpha, dloss = rng.standard_normal((T, K)), (1.3, 0.7)
    kw = dict(renorm=renorm, balance_coef=0.5, z_coef=0.25, mask=mask)
    ref = so.route(x, K, **kw)
    got = so.route_bwd(x, ref["topk_idx"], ref["counts"], dalpha, dloss, **kw)

    def total(z):
        r = so.route(z, K, idx=ref["topk_idx"], **kw)
        return (r["alpha"] * dalpha).sum() + dloss[0] * r["loss"][0] + dloss[1] * r["loss"][1]

    for t in range(T):
        for e in range(E):
            if not np.isfinite(x[t, e]):
                assert got[t, e] == 0
                continue
            d = np.zeros_like(x)
            d[t, e] = FD_STEP
            fd = (total(x + d) - total(x - d)) / (2 * FD_STEP)
            assert abs(fd - got[t, e]) <= FD_TOL * (1 + abs(fd)), (t, e)


def test_router_closed_forms():
    # uniform logits: every p is 1/E, the lowest K experts win, balance = c_b E K/(E K) ...
    T, E, K = 6, 8, 2
    r = so.route(np.zeros((T, E)), K, balance_coef=3.0, z_coef=1.0)
    assert (r["topk_idx"] == np.arange(K)).all()
    assert np.allclose(r["alpha"], 1 / E)
    # counts are T for two experts, P is T/E each: E/(T^2 K) * 2 T * T/E = 1
    assert np.isclose(r["loss"][0], 3.0) and np.isclose(r["loss"][1], np.log(E) ** 2)
    # nothing usable: everything is zero, ids stay valid
    r = so.route(np.full((2, 3), -np.inf), 2, renorm=True, balance_coef=1.0, z_coef=1.0)
    assert (r["alpha"] == 0).all() and (r["counts"] == 0).all() and (r["loss"] == 0).all()
    assert (r["topk_idx"] == [[0, 1], [0, 1]]).all()


def test_topk_ties_zero_and_nan():
    x = np.array([[0.0, -0.0, 1.0, np.nan], [-np.inf, np.nan, -np.inf, -5.0]])
    assert so.topk(x, 4).tolist() == [[2, 0, 1, 3], [3, 0, 1, 2]]


@pytest.mark.parametrize("T,D", [(1, 8), (3, 16), (5, 40)])
def test_norm_gradient_matches_differences(T, D):
    rng = np.random.default_rng(D)
    x, res, w = rng.standard_normal((T, D)), rng.standard_normal((T, D)), rng.standard_normal(D)
    dy, dh = rng.standard_normal((T, D)), rng.standard_normal((T, D))
    f = so.add_rmsnorm(x, res, w, 1e-5)
    dx, dw = so.add_rmsnorm_bwd(dy, dh, f["h"], w, f["rstd"])

    def total(x_, w_):
        r = so.add_rmsnorm(x_, res, w_, 1e-5)
        return (r["y"] * dy).sum() + (r["h"] * dh).sum()

    for t in range(T):
        for d in range(D):
            e = np.zeros_like(x)
            e[t, d] = FD_STEP
            fd = (total(x + e, w) - total(x - e, w)) / (2 * FD_STEP)
            assert abs(fd - dx[t, d]) <= 10 * FD_TOL * (1 + abs(fd))
    for d in range(D):
        e = np.zeros(D)
        e[d] = FD_STEP
        fd = (total(x, w + e) - total(x, w - e)) / (2 * FD_STEP)
        assert abs(fd - dw[d]) <= 10 * FD_TOL * (1 + abs(fd))


def test_e4m3_is_the_format():
    # the whole grid against torch's own decoding of the 127 non-negative codes
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(so.e4m3_grid(), codes)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 2, 4000), codes,
                        (codes[1:] + codes[:-1]) / 2])
    v = np.clip(v, -448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(so.e4m3(v), want)


def test_adamw_first_step_closed_form():
    # at step 1 from zero moments mhat = g and vhat = g^2: the step is lr sign(g)
    g = np.array([2.0, -3.0, 0.0])
    p, m, v = so.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 1, 0.1, 0.9, 0.99, 0.0 + 1e-30,
                       0.5)
    assert np.allclose(p, 1 * (1 - 0.05) - 0.1 * np.sign(g))


def test_gate_grad_is_the_combine_gradient():
    rng = np.random.default_rng(3)
    T, K, D = 4, 3, 5
    y, g = rng.standard_normal((T * K, D)), rng.standard_normal((T, D))
    inv = rng.permutation(T * K)
    a = rng.standard_normal((T, K))

    def out(alpha):
        return sum(g[t] @ (alpha[t, k] * y[inv[t * K + k]]) for t in range(T) for k in range(K))

    got = so.gate_grad(g, y, inv, K)
    for t in range(T):
        for k in range(K):
            d = np.zeros_like(a)
            d[t, k] = 1.0
            assert np.isclose(out(a + d) - out(a), got[t, k])


# -- refusals -----------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    from demand_side_expert_gb300 import build as b

    if not os.path.exists(b.LIB):
        b.build()
    from demand_side_expert_gb300 import lrm

    return lrm


def _router(lib, **kw):
    f = dict(T=4, E=8, K=2, dtype=lib.LRM_F32, stride=8, renorm=0, balance_coef=0.0, z_coef=0.0)
    f.update(kw)
    return lib.lrm_router(*[f[k] for k, _ in lib.lrm_router._fields_])


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(K=0), 1), (dict(K=9), 1), (dict(dtype=7), 1),
    (dict(stride=7), 1), (dict(E=2048, stride=2048), 2), (dict(E=64, K=40, stride=64), 2),
    (dict(T=1 << 30, K=2), 2)])
def test_router_refuses_shapes(lib, bad, want):
    r = _router(lib, **bad)
    assert lib.lrm_router_workspace_bytes(r) == 0
    args = [ctypes.byref(r)] + [256] * 9 + [1 << 30, None]
    assert lib._lib.lrm_route(*args) == want
    assert lib._lib.lrm_route_bwd(*args) == want


def test_router_refuses_pointers(lib):
    r = _router(lib)
    n = lib.lrm_router_workspace_bytes(r)
    ok = dict(logits=256, mask=None, idx=512, alpha=768, counts=1024, psum=1280, loss=1536)

    def call(ws=4096, nb=n, **kw):
        a = {**ok, **kw}
        return lib._lib.lrm_route(ctypes.byref(r), *a.values(), ws, nb, None)

    assert call(ws=None) == lib.LRM_ERR_WORKSPACE
    assert call(nb=n - 1) == lib.LRM_ERR_WORKSPACE
    assert call(ws=4096 + 128) == lib.LRM_ERR_UNSUPPORTED
    assert call(loss=None) == lib.LRM_ERR_INVALID_ARG  # all three statistics or none
    assert call(logits=None) == lib.LRM_ERR_INVALID_ARG
    assert call(alpha=None) == lib.LRM_ERR_INVALID_ARG
    assert call(logits=264) == lib.LRM_ERR_UNSUPPORTED
    assert lib._lib.lrm_route(None, *ok.values(), 4096, n, None) == lib.LRM_ERR_INVALID_ARG


def _norm(lib, **kw):
    f = dict(T=4, D=64, dtype=lib.LRM_BF16, grad_dtype=lib.LRM_F32, q_cols=0, eps=1e-6,
             x_stride=64, res_stride=64)
    f.update(kw)
    return lib.lrm_norm(*[f[k] for k, _ in lib.lrm_norm._fields_])


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), 1), (dict(D=0), 1), (dict(dtype=3), 1), (dict(grad_dtype=-1), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(q_cols=-1), 1), (dict(x_stride=63), 1),
    (dict(D=60, x_stride=64, res_stride=64), 2), (dict(q_cols=48), 2), (dict(x_stride=68), 2),
    (dict(D=16392, x_stride=16392, res_stride=16392), 2)])
def test_norm_refuses_shapes(lib, bad, want):
    n = _norm(lib, **bad)
    assert lib.lrm_norm_workspace_bytes(n) == 0
    assert lib._lib.lrm_add_rmsnorm(ctypes.byref(n), *[256] * 8, None) == want
    assert lib._lib.lrm_add_rmsnorm_bwd(ctypes.byref(n), *[256] * 8, 1 << 30, None) == want


def test_norm_refuses_pointers(lib):
    n = _norm(lib)
    b = ctypes.byref(n)
    need = lib.lrm_norm_workspace_bytes(n)
    fwd, bwd = lib._lib.lrm_add_rmsnorm, lib._lib.lrm_add_rmsnorm_bwd
    # x, res, w, h, y, q, q_scale, rstd
    assert fwd(b, 256, 256, 256, 256, None, None, None, 256, None) == lib.LRM_ERR_INVALID_ARG
    assert fwd(b, 256, 256, 256, 256, 256, 256, None, 256, None) == lib.LRM_ERR_INVALID_ARG
    assert fwd(b, None, 256, 256, 256, 256, None, None, 256, None) == lib.LRM_ERR_INVALID_ARG
    assert fwd(b, 256, 264, 256, 256, 256, None, None, 256, None) == lib.LRM_ERR_UNSUPPORTED
    # in place over rows that are not contiguous
    wide = ctypes.byref(_norm(lib, x_stride=128))
    assert fwd(wide, 512, None, 256, None, 512, None, None, 256, None) == lib.LRM_ERR_INVALID_ARG
    # dy, dh, h, w, rstd, dx, dw, ws, bytes
    assert bwd(b, *[256] * 7, None, need, None) == lib.LRM_ERR_WORKSPACE
    assert bwd(b, *[256] * 7, 256, need - 1, None) == lib.LRM_ERR_WORKSPACE
    assert bwd(b, *[256] * 6, None, 256, need, None) == lib.LRM_ERR_INVALID_ARG
    assert bwd(b, 256, 256, 260, *[256] * 4, 256, need, None) == lib.LRM_ERR_UNSUPPORTED


def test_adamw_refuses(lib):
    def call(count=1, hyper=None, **kw):
        h = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, grad_scale=None)
        h.update(hyper or {})
        t = dict(param=256, grad=256, master=None, m=256, v=256, m_scale=256, v_scale=256, n=10,
                 param_dtype=lib.LRM_F32, grad_dtype=lib.LRM_F32, state=lib.LRM_STATE_F32,
                 reserved=0, weight_decay=0.0)
        t.update(kw)
        arr = (lib.lrm_adamw_tensor * 1)(lib.lrm_adamw_tensor(*t.values()))
        return lib._lib.lrm_adamw_step(ctypes.byref(lib.lrm_adamw(*h.values())), arr, count, None)

    bad, no = lib.LRM_ERR_INVALID_ARG, lib.LRM_ERR_UNSUPPORTED
    assert call(count=-1) == bad
    assert call(hyper=dict(beta1=1.0)) == bad and call(hyper=dict(beta2=-0.1)) == bad
    assert call(hyper=dict(step=0)) == bad and call(hyper=dict(eps=float("nan"))) == bad
    assert call(n=-1) == bad and call(grad=None) == bad and call(state=5) == bad
    assert call(param_dtype=9) == bad and call(master=256) == bad  # a master of a float32 param
    assert call(state=lib.LRM_STATE_F8, m_scale=None) == bad
    assert call(param=264) == no and call(m=264) == no
    assert call(state=lib.LRM_STATE_F8, v_scale=258) == no
    assert call(hyper=dict(grad_scale=257)) == no
    assert lib._lib.lrm_adamw_step(None, None, 0, None) == bad


def test_gate_grad_refuses(lib):
    s = lib.make_shape(4, 64, 64, 8, 2, lib.LRM_BF16)
    n = lib.lrm_workspace_bytes(s)
    f, b = lib._lib.lrm_gate_grad, ctypes.byref(s)
    assert f(b, 256, 256, 256, None, 256, n, None) == lib.LRM_ERR_INVALID_ARG
    assert f(b, 256, 264, 256, 256, 256, n, None) == lib.LRM_ERR_UNSUPPORTED
    assert f(b, 256, 256, 256, 256, None, n, None) == lib.LRM_ERR_WORKSPACE


def test_python_classes_refuse_on_the_host():
    from demand_side_expert_gb300 import AddRMSNorm, AdamW, Router

    with pytest.raises(ValueError):
        Router(4, 2048, 2)
    with pytest.raises(ValueError):
        Router(4, 8, 2, device="cpu")
    with pytest.raises(ValueError):
        AddRMSNorm(4, 30)
    with pytest.raises(ValueError):
        AddRMSNorm(4, 64, store_y=False, device="cpu")
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError):
        AdamW([], [])
