"""Host side of the operators for training under tight memory: what the classes check,
keep and refuse, with the calls of liblrm replaced by a recorder and CPU tensors in place
of device ones (no GPU)."""

import os
import types

import pytest
import torch

F8 = torch.float8_e4m3fn


@pytest.fixture
def host(monkeypatch):
    """The package's modules, on CPU tensors; ``calls`` gets (entry point, arguments)."""
    from demand_side_expert_gb300 import build as b

    if not os.path.exists(b.LIB):
        b.build()
    from demand_side_expert_gb300 import layer, lrm, pipeline

    calls = []

    def recorder(name):
        return lambda *args: calls.append((name, args))

    for module in (layer, pipeline):
        monkeypatch.setattr(module, "_device", lambda device: torch.device("cpu"))
        monkeypatch.setattr(module, "_stream", lambda device, stream: stream or 0)
    for name in ("_group_route", "_group_route_bwd", "_bias_step", "_block", "_block_bwd"):
        monkeypatch.setattr(layer, name, recorder(name))
    monkeypatch.setattr(pipeline, "_pack", recorder("_pack"))
    for name in ("lrm_clear_device_error", "lrm_dispatch_permute", "lrm_expert_fwd_grouped",
                 "lrm_score", "lrm_score_variant", "lrm_score_packed", "lrm_select_rate",
                 "lrm_compact", "lrm_compact_packed", "lrm_expert_bwd_grouped",
                 "lrm_expert_bwd_gathered", "lrm_expert_bwd_compacted"):
        monkeypatch.setattr(lrm, name, recorder(name))
    return types.SimpleNamespace(layer=layer, lrm=lrm, pipeline=pipeline, calls=calls)


def names(host):
    return [name for name, _ in host.calls]


# -- router -------------------------------------------------------------------
def test_router_checks_its_inputs(host):
    r = host.layer.GroupRouter(4, 16, 2, "bf16", groups=4, top_groups=2)
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    for bad in (x.float(), x[:3], x[:, :8], torch.zeros(16, 4, dtype=x.dtype).t()):
        with pytest.raises(ValueError, match="logits"):
            r.route(bad)
    for bad in (torch.zeros(8), torch.zeros(16, dtype=torch.bfloat16), torch.zeros(32)[::2]):
        with pytest.raises(ValueError, match="bias"):
            r.route(x, bias=bad)
    with pytest.raises(ValueError, match="mask"):
        r.route(x, mask=torch.zeros(4))
    assert not host.calls[1:]
    r.route(torch.zeros(4, 24, dtype=x.dtype)[:, :16], mask=torch.ones(4, dtype=torch.bool))
    assert r.desc.stride == 24 and names(host)[-1] == "_group_route"
    for bad in (dict(dalpha=torch.zeros(4, 3)), dict(dloss=torch.zeros(2)),
                dict(dalpha=torch.zeros(4, 2).double())):
        with pytest.raises(ValueError):
            r.backward(x, **bad)
    with pytest.raises(AttributeError):
        r.topk_idx = torch.zeros(4, 2)


def test_router_gradient_and_bias_need_choices_and_counts(host):
    x, bias = torch.zeros(4, 8), torch.zeros(8)
    r = host.layer.GroupRouter(4, 8, 2, balance_coef=0.1)
    with pytest.raises(ValueError, match="route"):
        r.backward(x)
    with pytest.raises(ValueError, match="counts"):
        r.next_bias(bias, 0.1)
    r.route(x, stats=False)
    with pytest.raises(ValueError, match="statistics"):
        r.backward(x)
    with pytest.raises(ValueError, match="counts"):
        r.next_bias(bias, 0.1)
    r.route(x)
    r.backward(x)
    assert r.next_bias(bias, 0.1) is r.next_bias(bias, 0.1) is not bias
    assert r.next_bias(bias, 0.1, out=bias) is bias
    with pytest.raises(ValueError, match="out"):
        r.next_bias(bias, 0.1, out=torch.zeros(9))
    r.route(x, stats=False)  # its counts are of other choices
    with pytest.raises(ValueError, match="statistics"):
        r.backward(x)
    r.counts.fill_(1)
    r.backward(x)
    r.next_bias(bias, 0.1)
    free = host.layer.GroupRouter(4, 8, 2)  # the loss weighs nothing
    free.route(x, stats=False)
    free.backward(x)
    own = host.layer.GroupRouter(4, 8, 2)
    own.topk_idx.fill_(0)
    own.backward(x)
    none = host.layer.GroupRouter(0, 8, 2, balance_coef=0.1)
    none.backward(x[:0])
    assert names(host).count("_group_route_bwd") == 5


# -- packed state ---------------------------------------------------------------
def layer_inputs(T=6, D=64, H=64, E=8, K=2, dt=torch.bfloat16):
    def z(*shape):
        return torch.zeros(*shape, dtype=dt)

    return dict(topk_idx=torch.zeros(T, K, dtype=torch.int32), alpha=torch.zeros(T, K),
                x=z(T, D), g=z(T, D), phi=None, w_gate=z(E, D, H), w_up=z(E, D, H),
                w_down=z(E, H, D))


# places of lrm_compact_packed's arguments
X_SCALE, X_COLS, X_C = 8, 9, 12


def test_forward_packs_and_step_takes_it(host):
    T, D, H, E, K = 6, 64, 64, 8, 2
    pipe = host.pipeline.RecalibratedExpertBackward(T, D, H, E, K, "bf16", "cpu")
    state = host.pipeline.PackedState(T, K, H, "bf16", cols=64)
    v = layer_inputs()
    with pytest.raises(ValueError, match="nothing has been packed"):
        pipe.step(**v, ab=state)
    pipe.forward(v["topk_idx"], v["alpha"], v["x"], v["w_gate"], v["w_up"], v["w_down"],
                 packed=state)
    assert names(host)[-2:] == ["lrm_expert_fwd_grouped", "_pack"]
    assert host.calls[-1][1][1] == pipe.ab.data_ptr() and state.filled
    del host.calls[:]
    pipe.step(**v, ab=state, rate=(1, 2))
    assert names(host) == ["lrm_dispatch_permute", "lrm_score_packed", "lrm_select_rate",
                           "lrm_compact_packed", "lrm_expert_bwd_grouped"]
    assert host.calls[-2][1][X_C] is pipe.x_c and host.calls[-2][1][X_SCALE] is None
    del host.calls[:]
    pipe.step(**v, ab=state, rate=(1, 2), gathered=True)
    assert names(host)[-2:] == ["lrm_compact_packed", "lrm_expert_bwd_compacted"]
    assert host.calls[-2][1][X_C] is None  # no copy of x
    del host.calls[:]
    x8 = (torch.zeros(T, D).to(F8), torch.zeros(T, 2))
    pipe.step(**{**v, "x": x8}, ab=state)
    assert host.calls[-2][1][X_COLS] == 32 and host.calls[-2][1][X_SCALE] is x8[1]
    pipe.step(**{**v, "x": (x8[0], torch.zeros(T, 1))}, ab=state)
    assert host.calls[-2][1][X_COLS] == 0
    # the other criteria read no phi
    pipe.step(**v, ab=state, metric=host.lrm.LRM_METRIC_GRAD_SQ)
    assert "lrm_score_variant" in names(host)


def test_step_refuses_before_it_begins(host):
    T, K, H = 6, 2, 64
    pipe = host.pipeline.RecalibratedExpertBackward(T, 64, H, 8, K, "bf16", "cpu")
    v = layer_inputs()
    state = host.pipeline.PackedState(T, K, H, "bf16", cols=64)
    state.q.copy_(torch.zeros(T * K, 2 * H).to(F8))  # the caller's own codes
    assert state.filled
    for other in (host.pipeline.PackedState(T + 1, K, H, "bf16"),
                  host.pipeline.PackedState(T, K, 128, "bf16"),
                  host.pipeline.PackedState(T, K, H, "f32")):
        with pytest.raises(ValueError, match="packed"):
            pipe.step(**v, ab=other)
        with pytest.raises(ValueError, match="packed"):
            pipe.forward(v["topk_idx"], v["alpha"], v["x"], v["w_gate"], v["w_up"], v["w_down"],
                         packed=other)
    x8 = (torch.zeros(T, 64).to(F8), torch.zeros(T, 1))
    with pytest.raises(ValueError, match="8-bit x"):
        pipe.step(**{**v, "x": x8}, ab=state, gathered=True)
    with pytest.raises(ValueError, match="8-bit x"):
        pipe.step(**{**v, "x": x8}, ab=torch.zeros(T * K, 2 * H, dtype=torch.bfloat16))
    for bad in ((x8[0], torch.zeros(T, 5)), (x8[0][:3], x8[1]), (x8[0], x8[1].double()),
                (v["x"], x8[1]), v["x"].float(), v["x"][:2]):
        with pytest.raises(ValueError, match="^x"):
            pipe.step(**{**v, "x": bad}, ab=state)
    for name, bad in (("g", v["g"].float()), ("g", v["g"][:, :32]),
                      ("alpha", v["alpha"].double())):
        with pytest.raises(ValueError, match=f"^{name}"):
            pipe.step(**{**v, name: bad}, ab=state)
    assert names(host) == ["lrm_clear_device_error"]


def test_pack_checks_its_rows(host):
    state = host.pipeline.PackedState(3, 2, 64, "bf16")
    good = torch.zeros(6, 128, dtype=torch.bfloat16)
    for bad in (good.float(), good[:5], good[:, :64],
                torch.zeros(6, 256, dtype=good.dtype)[:, :128]):
        with pytest.raises(ValueError, match="^ab"):
            state.pack(bad)
    assert not state.filled and not host.calls
    state.pack(good)
    assert state.filled and host.calls[-1][1][1] == good.data_ptr()
    with pytest.raises(AttributeError):
        state.q = good
    assert host.pipeline.PackedState(0, 2, 64).filled


# -- norms around a block ---------------------------------------------------------
def test_block_norm_checks_its_inputs(host):
    T, D = 4, 16
    n = host.layer.BlockNorm(T, D, "bf16", gate="column")
    b, r = torch.zeros(T, D), torch.zeros(T, D, dtype=torch.bfloat16)
    w = torch.ones(D, dtype=torch.bfloat16)
    ok = dict(block=b, residual=r, w=w, w_post=w, gate=w)
    for name, bad in (("block", r), ("block", b[:3]), ("residual", b), ("residual", r[:, :8]),
                      ("w", w.float()), ("w", w[:8]), ("w_post", None), ("w_post", w[:8]),
                      ("gate", None), ("gate", torch.ones(T, dtype=w.dtype)),
                      ("gate", torch.ones(2 * D, dtype=w.dtype)[::2])):
        with pytest.raises(ValueError, match=f"^{name}"):
            n.forward(**{**ok, name: bad})
    with pytest.raises(ValueError, match="forward"):
        n.backward(b, b, w, w, w)
    n.forward(**ok)
    dy = torch.zeros(T, D)
    for change in (dict(dy=r), dict(block=r), dict(h=b), dict(dh=r), dict(w_post=None),
                   dict(gate=None), dict(block=torch.zeros(T, 2 * D)[:, :D])):
        with pytest.raises(ValueError):
            n.backward(**{**dict(dy=dy, block=b, w=w, w_post=w, gate=w), **change})
    assert names(host) == ["_block"]
    n.backward(dy, b, w, w, w)
    assert host.calls[-1][1][3] == n.h.data_ptr()
    assert n.dres.shape == (T, D) and n.dgate.shape == (D,) and n.dblock.dtype is torch.bfloat16
    token = host.layer.BlockNorm(T, D, "f32", gate="token", post=False, residual_scale=0.5)
    assert token.block_rstd is None and token.dw_post is None and token.dgate.shape == (T,)
    with pytest.raises(ValueError, match="^w_post"):
        token.forward(b, b, w.float(), w_post=w.float(), gate=torch.ones(T))
    token.forward(b, b, w.float(), gate=torch.ones(T))
    plain = host.layer.BlockNorm(T, D, "f32")
    with pytest.raises(ValueError, match="^gate"):
        plain.forward(b, b, w.float(), w_post=w.float(), gate=w.float())
    assert plain.dgate is None


def test_block_norm_gradient_of_the_callers_rows(host):
    """Both 1/rms written by the caller serve, with the h that they are of."""
    T, D = 4, 16
    x, w = torch.zeros(T, D), torch.ones(D)
    n = host.layer.BlockNorm(T, D, "f32")
    n.rstd.fill_(1)
    with pytest.raises(ValueError, match="forward"):  # of the block there is none yet
        n.backward(x, x, w, w, h=x)
    n.block_rstd.fill_(1)
    with pytest.raises(ValueError, match="^h"):
        n.backward(x, x, w, w)
    n.backward(x, x, w, w, h=x)
    empty = host.layer.BlockNorm(0, D, "f32")
    empty.backward(x[:0], x[:0], w, w)
    with torch.inference_mode():
        m = host.layer.BlockNorm(T, D, "f32")
        m.forward(x, x, w, w)
        m.backward(x, x, w, w)
    assert names(host).count("_block_bwd") == 3


def test_refused_block_norm_calls_change_nothing(host, monkeypatch):
    T, D = 4, 8
    x, w = torch.zeros(T, D), torch.ones(D)
    n = host.layer.BlockNorm(T, D, "f32")

    def refuse(*args):
        raise host.lrm.LrmError("lrm_block_norm", host.lrm.LRM_ERR_UNSUPPORTED)

    monkeypatch.setattr(host.layer, "_block", refuse)
    with pytest.raises(host.lrm.LrmError):  # rows 12 elements apart
        n.forward(torch.zeros(T, 12)[:, :D], x, w, w)
    assert n.desc.block_stride == n.desc.res_stride == D and not n._normed


def test_calls_run_on_the_device_of_their_buffers(host, monkeypatch):
    r = host.layer.GroupRouter(4, 8, 2)
    n = host.layer.BlockNorm(4, 8, "f32")
    s = host.pipeline.PackedState(4, 2, 8, "f32", cols=32)
    x, w = torch.zeros(4, 8), torch.zeros(8)
    r.route(x)
    n.forward(x, x, w, w)
    calls = len(host.calls)

    def refuse(device, stream):
        assert device == torch.device("cpu")
        raise ValueError("current device")

    monkeypatch.setattr(host.layer, "_stream", refuse)
    monkeypatch.setattr(host.pipeline, "_stream", refuse)
    for call in (lambda: r.route(x), lambda: r.backward(x), lambda: r.next_bias(w, 0.1),
                 lambda: n.forward(x, x, w, w), lambda: n.backward(x, x, w, w),
                 lambda: s.pack(torch.zeros(8, 16))):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert len(host.calls) == calls and not s.filled
