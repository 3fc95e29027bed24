"""Pins of the linear attention's oracle: its gradients against central differences of its forward, its
forward against closed forms."""
import numpy as np
import pytest

from oracle import layer
from test_layer_oracle_cpu import differences

# central differences in fp64 with step 1e-6: truncation ~ 1e-12 f''', cancellation ~ 1e-10
TOL = 1e-7


def make(seed, B, T, H, Hk, K, V, N, head=False):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(B, T, Hk, K)), k=r.normal(size=(B, T, Hk, K)), v=r.normal(size=(B, T, H, V)),
                log_decay=-r.uniform(0.01, 1.0, size=(H,) if head else (B, T, H)), init=r.normal(size=(N, H, V, K)))


@pytest.mark.parametrize("H,Hk,head,cu", [(2, 2, False, None), (4, 2, True, None), (3, 1, False, [0, 3, 3, 6]),
                                          (2, 2, True, [0, 1, 6])])
def test_gradients_match_differences(H, Hk, head, cu):
    B, T = (1, 6) if cu else (2, 4)
    N = len(cu) - 1 if cu else B
    v = make(3, B, T, H, Hk, 3, 2, N, head)
    r = np.random.default_rng(4)
    do, df = r.normal(size=v["v"].shape), r.normal(size=v["init"].shape)
    got = layer.linear_attention(**v, scale=0.7, cu=cu, do=do, dfin=df)
    for k, out in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_decay", "dlog_decay"), ("init", "dinitial_state")):
        ref = differences(lambda: layer.linear_attention(**v, scale=0.7, cu=cu), v[k], (do, df))
        assert np.abs(got[out] - ref).max() < TOL * 100, out


def test_matches_the_matrix_form():
    v = make(5, 2, 7, 3, 3, 4, 5, 2)
    o, fin = layer.linear_attention(**v, scale=0.5)
    G = np.cumsum(v["log_decay"], 1)
    D = np.where(np.tril(np.ones((7, 7), bool))[None, :, :, None], np.exp(G[:, :, None] - G[:, None]), 0.0)
    P = np.einsum("bthk,bshk->btsh", v["q"], v["k"]) * D
    ref = 0.5 * (np.einsum("btsh,bshv->bthv", P, v["v"]) +
                 np.exp(G)[..., None] * np.einsum("bhvk,bthk->bthv", v["init"], v["q"]))
    assert np.allclose(o, ref, rtol=1e-12, atol=1e-12)
    w = np.exp(G[:, -1:] - G)
    assert np.allclose(fin, np.exp(G[:, -1])[..., None, None] * v["init"] +
                       np.einsum("bsh,bshv,bshk->bhvk", w, v["v"], v["k"]), rtol=1e-12, atol=1e-12)


def test_a_reset_forgets_and_no_decay_sums():
    v = make(6, 1, 5, 1, 1, 3, 2, 1)
    v["log_decay"][:] = 0.0
    _, fin = layer.linear_attention(**v)
    assert np.allclose(fin[0, 0], v["init"][0, 0] + np.einsum("sv,sk->vk", v["v"][0, :, 0], v["k"][0, :, 0]))
    v["log_decay"][0, 3] = -np.inf
    o, fin = layer.linear_attention(**v)
    assert np.allclose(fin[0, 0], np.einsum("sv,sk->vk", v["v"][0, 3:, 0], v["k"][0, 3:, 0])) and np.isfinite(o).all()
