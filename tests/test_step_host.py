"""Host side of the training-step operators: what they check, keep and refuse, with the
calls of liblrm replaced by a recorder and CPU tensors in place of device ones (no GPU)."""

import os
import types

import pytest
import torch


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

    monkeypatch.setattr(layer, "_device", lambda device: torch.device("cpu"))
    for name in ("_route", "_route_bwd", "_norm", "_norm_bwd"):
        monkeypatch.setattr(layer, name, recorder(name))
    for name in ("lrm_clear_device_error", "lrm_adamw_step", "lrm_gate_grad",
                 "lrm_dispatch_permute", "lrm_gather_tokens", "lrm_expert_fwd_grouped",
                 "lrm_expert_fc1_fwd", "lrm_expert_fc2_fwd"):
        monkeypatch.setattr(lrm, name, recorder(name))
    for module in (layer, pipeline):
        monkeypatch.setattr(module, "_stream", lambda device, stream: stream or 0)
    return types.SimpleNamespace(layer=layer, lrm=lrm, pipeline=pipeline, calls=calls)


def test_adamw_refused_gradients_leave_the_table(host):
    """A set_grads that raises for one tensor keeps every gradient of before: the object
    does not hold the others', so their memory may go to someone else."""
    params = [torch.zeros(n) for n in (8, 16, 24)]
    grads = [torch.zeros(n) for n in (8, 16, 24)]
    opt = host.layer.AdamW(params, grads)
    for bad in ([torch.ones(8, dtype=torch.bfloat16), torch.ones(16), torch.ones(25)],
                [torch.ones(8), torch.ones(16).half(), torch.ones(24)], [torch.ones(8)]):
        with pytest.raises(ValueError):
            opt.set_grads(bad)
        assert opt.grads == grads
        assert [s.grad for s in opt._table] == [g.data_ptr() for g in grads]
        assert all(s.grad_dtype == host.lrm.LRM_F32 for s in opt._table)
    new = [torch.ones(n, dtype=torch.bfloat16) for n in (8, 16, 24)]
    opt.set_grads(new)
    assert [s.grad for s in opt._table] == [g.data_ptr() for g in new]
    assert all(s.grad_dtype == host.lrm.LRM_BF16 for s in opt._table)


def test_adamw_refuses_tensors_that_got_other_storage(host):
    """A parameter or a gradient whose storage was replaced is not stepped at its old
    place, which is not its own any more."""
    params, grads = [torch.zeros(8), torch.zeros(300)], [torch.zeros(8), torch.zeros(300)]
    opt = host.layer.AdamW(params, grads)
    opt.step()
    assert opt.t == 1
    old = params[1].data
    params[1].data = torch.ones(300)
    with pytest.raises(ValueError, match=r"params\[1\]"):
        opt.step()
    params[1].data = old
    opt.step()
    grads[0].data = torch.ones(8)
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        opt.step()
    opt.set_grads(grads)
    opt.step()
    opt.grads.append(torch.zeros(8))
    with pytest.raises(ValueError):
        opt.step()
    assert opt.t == 3 and [name for name, _ in host.calls] == ["lrm_adamw_step"] * 3


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_adamw_state_buffers_cannot_be_replaced(host, state):
    """Their addresses are in the table, as the ones of Router's and AddRMSNorm's buffers."""
    opt = host.layer.AdamW([torch.zeros(8, dtype=torch.bfloat16)], [torch.zeros(8)], state=state,
                           master=True)
    for name in ("m", "v", "m_scale", "v_scale", "master"):
        with pytest.raises(AttributeError):
            setattr(opt, name, torch.zeros(256))
    assert opt.m.numel() == 256 and (opt.m_scale is None) == (state == "f32")


def test_adamw_refuses_parameters_that_overlap(host):
    """Two parameters on the same memory would be read and written by two CTAs of a
    launch at once. Neighbours are fine, and one gradient for several parameters."""
    flat, g = torch.zeros(4096), torch.zeros(64)
    p = flat[:64]
    for params in ([p, p], [p, torch.zeros(64), flat[32:96]], [flat[32:96], p],
                   [p, p.view(8, 8)]):
        with pytest.raises(ValueError, match="overlap"):
            host.layer.AdamW(params, [torch.zeros(q.shape) for q in params])
    host.layer.AdamW([flat[64:128], p, flat[:0], flat[:0]], [g, g, g[:0], g[:0]])
    with pytest.raises(ValueError, match="overlap"):  # a gradient on a parameter's memory
        host.layer.AdamW([p, flat[64:128]], [g, flat[32:96]])
    opt = host.layer.AdamW([p], [p])  # in place: the gradient of p^2 / 2 is p
    with pytest.raises(ValueError, match="overlap"):
        opt.set_grads([flat[16:80]])
    assert opt.grads == [p]


def _pipe(host, T=6, D=64, K=2, dtype="bf16"):
    return host.pipeline.RecalibratedExpertBackward(T, D, 64, 8, K, dtype, "cpu")


def test_gate_grad_refuses_other_cotangents(host):
    """g is read as [T, D] of the layer's type, whatever it is: another type or shape
    would be read past its end or as other numbers, a strided one as its neighbours."""
    pipe = _pipe(host)
    pipe.forward(None, None, None, None, None, None)
    good = torch.zeros(6, 64, dtype=torch.bfloat16)
    for bad in (good.float(), good[:5], good[:, :32], torch.zeros(64, 6, dtype=good.dtype).t(),
                torch.zeros(6, 128, dtype=good.dtype)[:, :64], good.view(-1)):
        with pytest.raises(ValueError, match="^g: "):
            pipe.gate_grad(bad)
    wide = _pipe(host, dtype="f32")
    wide.forward(None, None, None, None, None, None)
    with pytest.raises(ValueError, match="^g: "):
        wide.gate_grad(good)
    assert "lrm_gate_grad" not in [name for name, _ in host.calls]
    assert pipe.gate_grad(good).shape == (6, 2) and host.calls[-1][0] == "lrm_gate_grad"


def test_gate_grad_needs_expert_outputs(host):
    """y holds something once a forward product (or the caller, who asked for the buffer)
    wrote it; gathering the tokens alone does not."""
    g = torch.zeros(6, 64, dtype=torch.bfloat16)
    pipe = _pipe(host)
    with pytest.raises(RuntimeError):
        pipe.gate_grad(g)
    pipe.gather_tokens(None)
    with pytest.raises(RuntimeError):
        pipe.gate_grad(g)
    pipe.fc1_fwd(None, None)
    pipe.fc2_fwd(None)
    pipe.gate_grad(g)
    other = _pipe(host)
    other.gather_tokens(None)
    assert other.y.shape == (12, 64)
    other.y.fill_(1)
    other.gate_grad(g)
    third = _pipe(host)
    third.y = other.y
    third.gate_grad(g)
    assert host.calls[-1][1][2] is other.y


def test_other_devices_are_refused(monkeypatch):
    """The kernels launch on the current device: an object on another one's memory is
    refused where it is made, and its calls are while another device is current."""
    from demand_side_expert_gb300 import layer, lrm, pipeline

    monkeypatch.setattr(lrm, "current_device", lambda: 0)
    assert layer._device("cuda") == torch.device("cuda", 0) == layer._device("cuda:0")
    for other in ("cuda:1", torch.device("cuda", 7)):
        with pytest.raises(ValueError, match="current device"):
            layer._device(other)
    monkeypatch.setattr(pipeline, "_device_now", lambda: 0)
    monkeypatch.setattr(pipeline, "_stream_now", lambda index: 5 + index)
    here = torch.device("cuda", 0)
    assert layer._stream(here, None) == 5 and layer._stream(here, 9) == 9
    for stream in (None, 9):
        with pytest.raises(ValueError, match="current device"):
            layer._stream(torch.device("cuda", 1), stream)


def test_calls_run_on_the_device_of_their_buffers(host, monkeypatch):
    r = host.layer.Router(4, 8, 2)
    n = host.layer.AddRMSNorm(4, 8, "f32")
    o = host.layer.AdamW([torch.zeros(8)], [torch.zeros(8)])
    x, w = torch.zeros(4, 8), torch.zeros(8)

    def refuse(device, stream):
        assert device == torch.device("cpu")
        raise ValueError("current device")

    r.route(x)
    n.forward(x, w)
    monkeypatch.setattr(host.layer, "_stream", refuse)
    calls = len(host.calls)
    for call in (lambda: r.route(x), lambda: r.backward(x), lambda: n.forward(x, w),
                 lambda: n.backward(x, w, h=x), o.step):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert len(host.calls) == calls and o.t == 0


def test_router_gradient_needs_choices_and_counts(host):
    """The gradient reads the ids and, with a loss that weighs something, the counts: of a
    route with statistics, or written by the caller. Those of nothing are refused."""
    Router = host.layer.Router
    x = torch.zeros(4, 8)
    r = Router(4, 8, 2)
    with pytest.raises(ValueError, match="route"):
        r.backward(x)
    r.route(x, stats=False)
    with pytest.raises(ValueError, match="statistics"):
        r.backward(x)
    r.route(x)
    r.backward(x)
    r.route(x, stats=False)  # its counts are of other choices
    with pytest.raises(ValueError, match="statistics"):
        r.backward(x)
    r.counts.fill_(1)
    r.backward(x)
    with pytest.raises(ValueError):  # a refused call is no route
        r.route(x[:, :4], stats=False)
    r.backward(x)
    # the losses weigh nothing: the counts do not matter
    free = Router(4, 8, 2, balance_coef=0.0, z_coef=0.0)
    free.route(x, stats=False)
    free.backward(x)
    # the caller's own choices and counts
    own = Router(4, 8, 2, z_coef=0.1)
    own.topk_idx.fill_(0)
    with pytest.raises(ValueError, match="statistics"):
        own.backward(x)
    own.counts.fill_(1)
    own.backward(x)
    with torch.inference_mode():
        served = Router(4, 8, 2)
        with pytest.raises(ValueError, match="route"):
            served.backward(x)
        served.route(x)
        served.backward(x)
    names = [name for name, _ in host.calls if name.startswith("_route")]
    assert names.count("_route_bwd") == 6


def test_refused_norm_calls_change_nothing(host, monkeypatch):
    """backward takes the sum and the 1/rms of the last forward that ran."""
    x, w = torch.zeros(4, 8), torch.ones(8)
    n = host.layer.AddRMSNorm(4, 8, "f32")
    n.forward(x, w)
    for bad in (dict(x=x[:3], w=w, residual=x), dict(x=x, w=w[:4], residual=x),
                dict(x=x, w=w, residual=x[:2])):
        with pytest.raises(ValueError):
            n.forward(**bad)
        with pytest.raises(ValueError, match="no residual"):
            n.backward(x, w)
    n.forward(x, w, residual=x)
    with pytest.raises(ValueError):
        n.forward(x, w[:4])
    n.backward(x, w)
    assert host.calls[-1][0] == "_norm_bwd" and host.calls[-1][1][3] == n.h.data_ptr()

    def refuse(*args):
        raise host.lrm.LrmError("lrm_add_rmsnorm", host.lrm.LRM_ERR_UNSUPPORTED)

    monkeypatch.setattr(host.layer, "_norm", refuse)
    with pytest.raises(host.lrm.LrmError):  # rows 12 elements apart
        n.forward(torch.zeros(4, 12)[:, :8], w, residual=torch.zeros(4, 12)[:, :8])
    assert n.desc.x_stride == n.desc.res_stride == 8
    assert n._summed


def test_norm_gradient_needs_a_forward(host):
    """rstd is of a forward, or written by the caller: not uninitialised memory."""
    x, w = torch.zeros(4, 8), torch.ones(8)
    n = host.layer.AddRMSNorm(4, 8, "f32")
    with pytest.raises(ValueError, match="forward"):
        n.backward(x, w, h=x)
    with pytest.raises(ValueError):
        n.forward(x, w[:4])
    with pytest.raises(ValueError, match="forward"):
        n.backward(x, w, h=x)
    n.rstd.fill_(1)
    n.backward(x, w, h=x)
    m = host.layer.AddRMSNorm(4, 8, "f32")
    m.forward(x, w)
    m.backward(x, w, h=x)
    empty = host.layer.AddRMSNorm(0, 8, "f32")
    empty.backward(x[:0], w, h=x[:0])
    with torch.inference_mode():
        host.layer.AddRMSNorm(4, 8, "f32").forward(x, w)
    assert [name for name, _ in host.calls].count("_norm_bwd") == 3


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_adamw_refused_state_changes_nothing(host, state):
    def make():
        opt = host.layer.AdamW([torch.ones(300, dtype=torch.bfloat16)], [torch.ones(300)],
                               state=state, master=True)
        return opt

    opt = make()
    kept = {k: v.clone() if torch.is_tensor(v) else v for k, v in opt.state_dict().items()}
    good = {k: torch.ones_like(v.float()).to(v.dtype) if torch.is_tensor(v) else v
            for k, v in kept.items()}
    good["step"] = 7
    last = "v" if state == "f32" else "v_scale"
    for change in ({last: good[last][:-1]}, {last: None}, {last: good[last].double()},
                   {"step": None}, {"step": "x"}, {"step": -1}):
        with pytest.raises((ValueError, TypeError)):
            opt.load_state_dict({**good, **change})
        assert opt.t == 0
        for k, v in opt.state_dict().items():
            if torch.is_tensor(v):
                assert torch.equal(v.view(torch.uint8), kept[k].view(torch.uint8)), (change, k)
    with pytest.raises(KeyError):
        opt.load_state_dict({k: v for k, v in good.items() if k != "step"})
    assert torch.equal(opt.m.view(torch.uint8), kept["m"].view(torch.uint8))
    opt.load_state_dict(good)
    assert opt.t == 7
    assert torch.equal(opt.v.view(torch.uint8), good["v"].view(torch.uint8))


def test_adamw_state_is_no_part_of_a_graph(host):
    """Parameters that autograd tracks: their master copies are plain numbers, and a state
    that is loaded from tracked tensors stays so."""
    import copy

    p = torch.nn.Parameter(torch.ones(300, dtype=torch.bfloat16))
    opt = host.layer.AdamW([p], [torch.ones(300)], master=True)
    assert (opt.master[:300] == 1).all()
    other = host.layer.AdamW([p], [torch.ones(300)], master=True)
    state = {**other.state_dict(), "m": other.m.clone().requires_grad_(True)}
    opt.load_state_dict(state)
    for k, v in opt.state_dict().items():
        if torch.is_tensor(v):
            assert not v.requires_grad and v.grad_fn is None, k
    copy.deepcopy(opt.state_dict())
    opt.step()


def test_router_without_tokens_needs_no_counts(host):
    x = torch.zeros(0, 8)
    r = host.layer.Router(0, 8, 2)
    r.backward(x)
    r.route(x, stats=False)
    r.backward(x)
    assert [name for name, _ in host.calls].count("_route_bwd") == 2
