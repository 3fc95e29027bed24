"""Pins of the layer operators' oracle: its gradients against central differences of its forward,
its forward against closed forms."""
import numpy as np
import pytest

from oracle import layer

RNG = np.random.default_rng


def differences(f, x, dout, h=1e-6):
    """d <dout, f(x)> / dx by central differences; f returns a list of arrays."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = sum((d * o).sum() for d, o in zip(dout, f()))
        x[i] = keep - h
        lo = sum((d * o).sum() for d, o in zip(dout, f()))
        x[i] = keep
        g[i] = (up - lo) / (2 * h)
    return g


# central differences in fp64 with step 1e-6: truncation ~ 1e-12 f''', cancellation ~ 1e-10
TOL = 1e-7


@pytest.mark.parametrize("W,silu,cu", [(2, True, None), (3, False, None), (4, True, [0, 1, 1, 5, 7]), (4, True, None)])
def test_conv_gradients_match_differences(W, silu, cu):
    r = RNG(1)
    B, T, D = (1, 7, 3) if cu else (2, 5, 3)
    N = len(cu) - 1 if cu else B
    v = dict(x=r.normal(size=(B, T, D)), weight=r.normal(size=(D, W)), bias=r.normal(size=D),
             init=r.normal(size=(N, W - 1, D)))
    dy, df = r.normal(size=(B, T, D)), r.normal(size=(N, W - 1, D))
    got = layer.short_conv(**v, cu=cu, silu=silu, dy=dy, dfin=df)
    for k, out in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("init", "dinitial_state")):
        ref = differences(lambda: layer.short_conv(**v, cu=cu, silu=silu), v[k], (dy, df))
        assert np.abs(got[out] - ref).max() < TOL * 100, out


def test_conv_of_an_impulse_is_the_reversed_taps():
    w = RNG(2).normal(size=(5, 4))
    x = np.zeros((1, 9, 5))
    x[0, 2] = 1.0
    y, fin = layer.short_conv(x, w, silu=False)
    assert np.allclose(y[0, 2:6], w.T[::-1]) and np.all(y[0, :2] == 0) and np.all(y[0, 6:] == 0)
    assert np.array_equal(fin[0], x[0, -3:])


@pytest.mark.parametrize("G,z,softplus,cu", [(1, True, True, None), (2, False, True, [0, 3, 3, 6]), (1, True, False, None)])
def test_scan_gradients_match_differences(G, z, softplus, cu):
    r = RNG(3)
    B, T, D, S = (1, 6, 4, 3) if cu else (2, 4, 4, 3)
    N = len(cu) - 1 if cu else B
    v = dict(x=r.normal(size=(B, T, D)), dt=r.normal(size=(B, T, D)) * 0.3, A=-np.exp(r.normal(size=(D, S))),
             Bm=r.normal(size=(B, T, G, S)), Cm=r.normal(size=(B, T, G, S)), skip=r.normal(size=D),
             z=r.normal(size=(B, T, D)) if z else None, dt_bias=r.normal(size=D) * 0.1, init=r.normal(size=(N, D, S)))
    dy, df = r.normal(size=(B, T, D)), r.normal(size=(N, D, S))
    got = layer.selective_scan(**v, cu=cu, softplus_dt=softplus, dy=dy, dfin=df)
    for k, out in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("skip", "dskip"), ("z", "dz"),
                   ("dt_bias", "ddt_bias"), ("init", "dinitial_state")):
        if v[k] is None:
            assert got[out] is None
            continue
        ref = differences(lambda: layer.selective_scan(**v, cu=cu, softplus_dt=softplus), v[k], (dy, df))
        assert np.abs(got[out] - ref).max() < TOL * 100, out


def test_scan_with_constant_step_is_a_geometric_sum():
    d, a, T = 0.25, -1.5, 12
    y, fin = layer.selective_scan(np.ones((1, T, 1)), np.full((1, T, 1), d), np.array([[a]]), np.ones((1, T, 1, 1)),
                                  np.ones((1, T, 1, 1)), softplus_dt=False)
    q = np.exp(d * a)
    assert np.allclose(y[0, :, 0], d * (1 - q ** np.arange(1, T + 1)) / (1 - q), rtol=1e-14)
    assert np.allclose(fin, y[0, -1, 0])


@pytest.mark.parametrize("parts", [("post_weight",), ("gate",), ("gate", "post_weight"), ("residual", "pre_weight"),
                                   ("gate", "residual", "scale", "post_weight", "pre_weight"), ("scale",)])
@pytest.mark.parametrize("which", ["dr", "dn", "both"])
def test_norm_gradients_match_differences(parts, which):
    r = RNG(4)
    R, D = 3, 5
    v = dict(y=r.normal(size=(R, D)))
    for p in parts:
        v[p] = r.normal(size=(R, D)) if p in ("gate", "residual") else r.normal(size=D)
    if which != "dr" and "pre_weight" not in parts:
        pytest.skip("no norm behind the block")
    dr = r.normal(size=(R, D)) if which != "dn" else None
    dn = r.normal(size=(R, D)) if which != "dr" else None
    got = layer.block_norm(**v, eps=1e-2, dr=dr, dn=dn)

    def f():
        a, b = layer.block_norm(**v, eps=1e-2)
        return [a if dr is not None else np.zeros_like(a), b if dn is not None else np.zeros_like(a)]
    dout = (0.0 if dr is None else dr, 0.0 if dn is None else dn)
    for k in v:
        assert np.abs(got["d" + k] - differences(f, v[k], dout)).max() < TOL * 100, k
