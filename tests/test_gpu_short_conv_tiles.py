"""The short convolution at the token tiles that layers of real sizes get (16 and 64 tokens forward, 8 to
64 backward), against the definition in float64 on the device: batches whose tokens are no multiple of a
tile, tile counts that are no multiple of four, packed batches with several, empty and long sequences in and
across tiles. The definition is pinned to the numpy oracle on the CPU."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, conv_bwd_gamma, conv_gamma, cu_of, layer, rnd


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if request.node.get_closest_marker("gpu"):
        if not torch.cuda.is_available():
            pytest.skip("no GPU")
        yield
        torch.cuda.empty_cache()
    else:
        yield


def conv64(x, weight, bias, init, cu, silu, dy=None, dfin=None, magnitude=False):
    """oracle.layer.short_conv on torch float64 tensors of any device, for tokens that all belong to a sequence."""
    mag = torch.abs if magnitude else (lambda v: v)
    B, T, D = x.shape
    W = weight.shape[1]
    spans = [(n, n, 0, T) for n in range(B)] if cu is None else [(n, 0, int(s), int(e)) for n, (s, e) in
                                                                 enumerate(zip(cu, cu[1:]))]
    y, dx, fin, dinit = torch.empty_like(x), torch.empty_like(x), torch.empty_like(init), torch.empty_like(init)
    dw, db = torch.zeros_like(weight), torch.zeros_like(bias)
    for n, row, t0, t1 in spans:
        L = t1 - t0
        full = torch.cat([init[n], x[row, t0:t1]])
        fin[n] = full[L:]
        p, size = bias.expand(L, D).clone(), bias.abs().expand(L, D).clone()
        for k in range(W):
            p += full[k:k + L] * weight[:, k]
            size += (full[k:k + L] * weight[:, k]).abs()
        s = torch.sigmoid(p)
        if dy is None:
            y[row, t0:t1] = size if magnitude else p * s if silu else p
            continue
        dp = mag(dy[row, t0:t1])
        if silu:
            dp = dp * ((1 + size) if magnitude else s * (1 + p * (1 - s)))
        dfull = torch.zeros_like(full)
        for k in range(W):
            dfull[k:k + L] += dp * mag(weight[:, k])
            dw[:, k] += (dp * mag(full[k:k + L])).sum(0)
        db += dp.sum(0)
        dfull[L:] += mag(dfin[n])
        dx[row, t0:t1], dinit[n] = dfull[W - 1:], dfull[:W - 1]
    return (y, fin) if dy is None else dict(dx=dx, dweight=dw, dbias=db, dinitial_state=dinit)


def make(B, T, D, W, dtype, lens, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.empty(s, device=device).normal_(generator=g)  # noqa: E731
    N = B if lens is None else len(lens)
    v = dict(x=n(B, T, D), weight=n(D, W), bias=n(D), init=n(N, W - 1, D), dy=n(B, T, D), dfin=n(N, W - 1, D))
    v = {k: t if k in ("weight", "bias") else t.to(dtype) for k, t in v.items()}
    return v, {k: t.double() for k, t in v.items()}


def inputs(ref):
    return [ref[k] for k in ("x", "weight", "bias", "init")]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("magnitude", [True, False])
@pytest.mark.parametrize("lens", [None, [0, 5, 1, 2, 0, 9]])
def test_the_definition_is_the_oracles(lens, magnitude, silu):
    B, T = (2, 9) if lens is None else (1, sum(lens))
    _, ref = make(B, T, 5, 4, F32, lens, "cpu")
    cu = cu_of(lens)
    num = [t.numpy() for t in inputs(ref)]
    kw = dict(cu=cu, silu=silu, magnitude=magnitude)
    got, want = conv64(*inputs(ref), **kw), layer.short_conv(*num, **kw)
    # a few dozen float64 operations
    assert all(np.allclose(a.numpy(), b, rtol=1e-13, atol=1e-13) for a, b in zip(got, want))
    got = conv64(*inputs(ref), **kw, dy=ref["dy"], dfin=ref["dfin"])
    want = layer.short_conv(*num, **kw, dy=ref["dy"].numpy(), dfin=ref["dfin"].numpy())
    assert set(got) == set(want) and all(np.allclose(got[k].numpy(), want[k], rtol=1e-13, atol=1e-13) for k in want)


def check(name, got, ref, mag, gamma):
    """_layer_util.check on the device."""
    half = torch.finfo(got.dtype).eps / 2
    assert torch.isfinite(got).all(), name
    worst = float(((got.double() - ref).abs() / (half * ref.abs() + gamma * (1 + half) * mag + 1e-37)).max())
    print(f"{name}: worst {worst:.3f} of the bound (gamma {gamma:.1e})", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} of the bound"


def ragged(T, seed):
    """Lengths that add up to T: empty sequences, some shorter than the taps, some inside a tile, some across many."""
    r, lens = rnd(seed), []
    while sum(lens) < T:
        lens.append(int(r.choice([0, 0, r.integers(1, 4), r.integers(4, 30), r.integers(30, 300), r.integers(300, 3000)])))
    lens[-1] -= sum(lens) - T
    return lens + [0]


def tile(tokens, groups, shift):
    """Tokens per tile: the longest that leaves 131072 threads, from 64 in steps of 1 / 2^shift."""
    t = 64
    while t > 4 and tokens // t * groups < 131072:
        t >>= shift
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,W,dtype,silu,packed,want", [
    (3, 2777, 2048, 4, BF16, True, False, 16), (5, 6571, 2048, 4, BF16, True, False, 64),
    (1, 15001, 1001, 3, F32, False, True, 16), (1, 33777, 1999, 4, BF16, True, True, 64),
    (1, 33700, 1000, 2, F32, True, True, 64)])
def test_forward(B, T, D, W, dtype, silu, packed, want):
    assert tile(B * T, -(-D // (8 if dtype == BF16 else 4)), 2) == want and T % want
    lens = ragged(T, T) if packed else None
    cu = cu_of(lens)
    on, ref = make(B, T, D, W, dtype, lens, "cuda")
    y, f = comba.short_conv(on["x"], on["weight"], on["bias"], on["init"], None if cu is None else torch.from_numpy(cu).cuda(),
                            silu=silu)
    ry, rf = conv64(*inputs(ref), cu, silu)
    size, _ = conv64(*inputs(ref), cu, silu, magnitude=True)
    check("y", y, ry, size, conv_gamma(W, float(size.max())))
    assert torch.equal(f.double(), rf)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,W,dtype,silu,packed,want", [
    (3, 713, 2048, 4, BF16, True, False, 8), (2, 2113, 2048, 3, F32, False, False, 16),
    (1, 8397, 2045, 4, BF16, True, True, 32), (3, 5500, 2048, 4, BF16, True, False, 64),
    (1, 33555, 1001, 2, F32, True, True, 64), (1, 16550, 2048, 4, BF16, True, True, 64)])
@pytest.mark.parametrize("wide_dy", [False, True])
def test_backward(B, T, D, W, dtype, silu, packed, want, wide_dy):
    if wide_dy and dtype == F32:
        pytest.skip("one type only")
    lens = ragged(T, T + 1) if packed else None
    cu = cu_of(lens)
    tiles = B * -(-T // want)
    sets = -(-tiles // 4)   # one partial sum of the parameter gradients each
    size = comba.lib().comba_short_conv_bwd_workspace_size(B, T, D, W, len(lens) if packed else 0)
    assert tile(B * T, -(-D // 4), 1) == want and size == -(-sets * (W + 1) * D * 4 // 256) * 256
    assert T % want and tiles % 4
    on, ref = make(B, T, D, W, dtype, lens, "cuda", seed=1)
    args = (on["x"], on["weight"], on["bias"], on["dy"].float() if wide_dy else on["dy"], on["init"],
            None if cu is None else torch.from_numpy(cu).cuda())
    g = comba.short_conv_bwd(*args, d_final_state=on["dfin"], silu=silu)
    kw = dict(dy=ref["dy"], dfin=ref["dfin"])
    r, m = conv64(*inputs(ref), cu, silu, **kw), conv64(*inputs(ref), cu, silu, **kw, magnitude=True)
    pmax = float(conv64(*inputs(ref), cu, silu, magnitude=True)[0].max())
    # additions on a term's way: along its tile, over four tiles, along one of 16 rows of the sets, over the 16
    adds = want + 3 + -(-sets // 16) + 16
    for k in r:
        check(k, g[k], r[k], m[k], conv_bwd_gamma(W, pmax, adds if k in ("dweight", "dbias") else 0))
    again = comba.short_conv_bwd(*args, d_final_state=on["dfin"], silu=silu)
    assert all(torch.equal(g[k], again[k]) for k in g)
