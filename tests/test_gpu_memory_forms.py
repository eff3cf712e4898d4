"""GPU tests of the operators for training under tight memory in the forms that only large
blocks take, against the float64 oracle. Sizes are counted from the device's SMs, as the
choice of a form is; tolerances are those of test_gpu_memory_ops.
"""

import math

import numpy as np
import pytest
import torch

from oracle import memory_oracle as mo
from test_gpu_memory_ops import (TINY, U, close, dev, make_bias, make_logits,  # noqa: F401
                                 router, score_tol, to64)

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
