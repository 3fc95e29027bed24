"""Pins of the group norm's oracle: its gradients against central differences of its forward, its forward
against the definition of the moments."""
import numpy as np
import pytest

from oracle import layer
from test_layer_oracle_cpu import TOL, differences


@pytest.mark.parametrize("groups,silu,affine,cu", [(2, True, True, None), (1, False, True, [0, 2, 2, 5]),
                                                   (6, True, False, None), (3, True, True, [0, 1, 5])])
def test_gradients_match_differences(groups, silu, affine, cu):
    r = np.random.default_rng(8)
    B, T, D = (1, 5, 6) if cu else (2, 3, 6)
    v = dict(x=r.normal(size=(B, T, D)))
    if affine:
        v.update(weight=r.normal(size=D), bias=r.normal(size=D))
    dy = r.normal(size=(B, T, D))
    kw = dict(groups=groups, eps=1e-2, silu=silu, cu=cu)
    got = layer.group_norm(**v, **kw, dy=dy)
    for k in v:
        ref = differences(lambda: layer.group_norm(**v, **kw)[:1], v[k], (dy,))
        assert np.abs(got["d" + k] - ref).max() < TOL * 100, k


def test_rows_of_every_group_have_mean_0_and_variance_1():
    x = np.random.default_rng(9).normal(size=(2, 9, 12)) * 3 + 5
    y, stats = layer.group_norm(x, 4, eps=0.0)
    u = y.reshape(2, 9, 4, 3)
    assert np.allclose(u.mean((1, 3)), 0) and np.allclose((u ** 2).mean((1, 3)), 1)
    assert np.allclose(stats[..., 0], x.reshape(2, 9, 4, 3).mean((1, 3)))
    y1, s1 = layer.group_norm(x.reshape(18, 1, 12), 4)
    assert s1.shape == (18, 4, 2) and np.allclose(y1.reshape(18, 4, 3).mean(-1), 0)
