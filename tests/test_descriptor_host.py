"""Sizes that a descriptor's 32 bits do not hold are refused, not cut down to the low ones."""

import pytest

from test_memory_host import host  # noqa: F401

BIG = 1 << 32


@pytest.mark.parametrize("T,E,K", [(BIG + 1, 8, 2), (4, BIG + 8, 2), (4, 8, BIG + 2)])
def test_routers(host, T, E, K):  # noqa: F811
    with pytest.raises(ValueError):
        host.layer.GroupRouter(T, E, K)
    with pytest.raises(ValueError):
        host.layer.Router(T, E, K)


def test_groups(host):  # noqa: F811
    for kw in (dict(groups=BIG + 2), dict(groups=2, top_groups=BIG + 1), dict(group_top=BIG + 1)):
        with pytest.raises(ValueError):
            host.layer.GroupRouter(4, 8, 2, **kw)


@pytest.mark.parametrize("T,D", [(BIG + 4, 8), (4, BIG + 8)])
def test_norms(host, T, D):  # noqa: F811
    with pytest.raises(ValueError):
        host.layer.BlockNorm(T, D)
    with pytest.raises(ValueError):
        host.layer.AddRMSNorm(T, D)


def test_state_and_layer(host):  # noqa: F811
    with pytest.raises(ValueError):
        host.pipeline.PackedState(1, 1, BIG + 8)
    with pytest.raises(ValueError):
        host.lrm.make_shape(BIG + 4, 64, 64, 8, 2, host.lrm.LRM_BF16)
    assert host.lrm.make_shape(4, 64, 64, 8, 2, host.lrm.LRM_BF16).T == 4
