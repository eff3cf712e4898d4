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
    monkeypatch.setattr(lrm, "stream_address", lambda stream=None: stream or 0)
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
