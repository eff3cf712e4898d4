"""One RecalibratedExpertBackward that serves several layers, host side: rows of a layer's own
in the place of its outputs, with the library's calls replaced by a recorder (no GPU)."""

import pytest
import torch

from test_memory_host import host, layer_inputs, names  # noqa: F401

T, D, H, E, K = 6, 64, 64, 8, 2
Y, OUT = 12, 13  # places of lrm_expert_fwd_grouped's arguments


def forward(pipe, **kw):
    v = layer_inputs()
    pipe.forward(v["topk_idx"], v["alpha"], v["x"], v["w_gate"], v["w_up"], v["w_down"], **kw)


def test_outputs_go_where_the_caller_wants_them(host):  # noqa: F811
    """Rows given before the first forward are written by it, as those given later are."""
    pipe = host.pipeline.RecalibratedExpertBackward(T, D, H, E, K, "bf16", "cpu")
    state = host.pipeline.PackedState(T, K, H, "bf16")
    for _ in range(2):
        y = torch.zeros(T * K, D, dtype=torch.bfloat16)
        out = torch.zeros(T, D)
        pipe.y, pipe.out = y, out
        forward(pipe, packed=state)
        name, args = host.calls[-2]
        assert name == "lrm_expert_fwd_grouped" and args[Y] is y and args[OUT] is out
        assert pipe.y is y and pipe.out is out


def test_outputs_are_checked(host):  # noqa: F811
    pipe = host.pipeline.RecalibratedExpertBackward(T, D, H, E, K, "bf16", "cpu")
    forward(pipe)
    y, out = pipe.y, pipe.out
    for bad in (y.float(), y[:-1], y[:, :32], torch.zeros(T * K, 2 * D, dtype=y.dtype)[:, :D]):
        with pytest.raises(ValueError, match="^y"):
            pipe.y = bad
    for bad in (out.bfloat16(), out[1:], torch.zeros(D, T).t()):
        with pytest.raises(ValueError, match="^out"):
            pipe.out = bad
    assert pipe.y is y and pipe.out is out


def test_weight_gradients_are_the_layers_own(host):  # noqa: F811
    pipe = host.pipeline.RecalibratedExpertBackward(T, D, H, E, K, "bf16", "cpu")
    state = host.pipeline.PackedState(T, K, H, "bf16")
    forward(pipe, packed=state)
    for name, shape in (("dw_gate", (E, D, H)), ("dw_up", (E, D, H)), ("dw_down", (E, H, D))):
        first = getattr(pipe, name)
        for bad in (torch.zeros(shape).double(), torch.zeros(E - 1, *shape[1:]),
                    torch.zeros(shape[1], E, shape[2]).transpose(0, 1), None):
            with pytest.raises(ValueError, match=f"^{name}"):
                setattr(pipe, name, bad)
        assert getattr(pipe, name) is first
        setattr(pipe, name, torch.zeros(shape))
        assert getattr(pipe, name) is not first
    pipe.step(**layer_inputs(), ab=state, gathered=True)
    args = host.calls[-1][1]
    assert all(any(a is getattr(pipe, n) for a in args) for n in ("dw_gate", "dw_up", "dw_down"))
