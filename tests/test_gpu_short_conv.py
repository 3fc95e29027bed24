"""The short causal convolution (prompt, single token, backward) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, both, check, conv_bwd_gamma, conv_gamma, cu_dev, cu_of, dev, layer, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, T, D, W, dtype, bias, init, lens=None, seed=0):
    r = rnd(seed)
    N = B if lens is None else len(lens)
    v = dict(x=r.normal(size=(B, T, D)), weight=r.normal(size=(D, W)), bias=r.normal(size=D) if bias else None,
             init=r.normal(size=(N, W - 1, D)) if init else None, dy=r.normal(size=(B, T, D)),
             dfin=r.normal(size=(N, W - 1, D)))
    return both(v, dtype, params=("weight", "bias"))


CASES = [  # B, T, D, W, dtype, silu, bias, init, lens
    (2, 1, 8, 2, BF16, True, True, False, None),
    (2, 2, 64, 4, BF16, True, True, True, None),          # fewer tokens than taps
    (3, 37, 1, 3, BF16, False, False, True, None),
    (2, 130, 72, 4, F32, True, True, True, None),
    (1, 65, 7, 4, BF16, True, True, False, None),
    (1, 64, 9, 3, F32, True, False, True, None),
    (2, 300, 520, 4, BF16, True, True, True, None),
    (1, 101, 24, 4, BF16, True, True, True, [0, 1, 2, 0, 3, 70, 25, 0]),
    (1, 101, 25, 3, F32, False, True, True, [64, 1, 36]),
    (1, 200, 256, 2, F32, True, True, False, [3, 197]),
    (1, 0, 16, 4, BF16, True, True, True, [0, 0]),        # no tokens at all
    (2, 4096, 2048, 4, BF16, True, True, True, None),     # full tiles of 64 tokens
]


@pytest.mark.parametrize("B,T,D,W,dtype,silu,bias,init,lens", CASES)
def test_forward(B, T, D, W, dtype, silu, bias, init, lens):
    on, ref = make(B, T, D, W, dtype, bias, init, lens)
    cu = cu_of(lens)
    y, f = comba.short_conv(on["x"], on["weight"], on["bias"], on["init"], cu_dev(cu), silu=silu)
    fwd = (ref["x"], ref["weight"], ref["bias"], ref["init"])
    ry, rf = layer.short_conv(*fwd, cu=cu, silu=silu)
    size, _ = layer.short_conv(*fwd, cu=cu, silu=silu, magnitude=True)
    pmax = 0 if size.size == 0 else np.nanmax(size)
    check("y", y, ry, size, conv_gamma(W, pmax))
    assert np.array_equal(f.double().cpu().numpy(), rf)   # copies of inputs


@pytest.mark.parametrize("B,T,D,W,dtype,silu,bias,init,lens", CASES[:-1])
@pytest.mark.parametrize("wide_dy", [False, True])
def test_backward(B, T, D, W, dtype, silu, bias, init, lens, wide_dy):
    if wide_dy and dtype == F32:
        pytest.skip("one type only")
    on, ref = make(B, T, D, W, dtype, bias, init, lens, seed=1)
    dy = on["dy"].float() if wide_dy else on["dy"]
    cu = cu_of(lens)
    g = comba.short_conv_bwd(on["x"], on["weight"], on["bias"], dy, on["init"], cu_dev(cu), d_final_state=on["dfin"],
                             silu=silu)
    args = dict(cu=cu, silu=silu, dy=ref["dy"], dfin=ref["dfin"])
    fwd = (ref["x"], ref["weight"], ref["bias"], ref["init"])
    r, m = layer.short_conv(*fwd, **args), layer.short_conv(*fwd, **args, magnitude=True)
    size, _ = layer.short_conv(*fwd, cu=cu, magnitude=True)
    pmax = 0 if size.size == 0 else np.nanmax(size)
    for k in r:
        adds = B * T if k in ("dweight", "dbias") else 0
        check(k, g[k], r[k], m[k], conv_bwd_gamma(W, pmax, adds))
    again = comba.short_conv_bwd(on["x"], on["weight"], on["bias"], dy, on["init"], cu_dev(cu),
                                 d_final_state=on["dfin"], silu=silu)
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)


def test_backward_without_state_or_its_gradient():
    on, ref = make(2, 9, 16, 4, F32, True, False)
    g = comba.short_conv_bwd(on["x"], on["weight"], on["bias"], on["dy"])
    r = layer.short_conv(ref["x"], ref["weight"], ref["bias"], dy=ref["dy"])
    m = layer.short_conv(ref["x"], ref["weight"], ref["bias"], dy=ref["dy"], magnitude=True)
    for k in r:
        check(k, g[k], r[k], m[k], conv_bwd_gamma(4, 20, 18))
    assert g["dinitial_state"] is None


@pytest.mark.parametrize("N,D,W,dtype,silu,init", [(1, 1, 2, BF16, True, True), (5, 64, 4, BF16, True, True),
                                                  (33, 72, 3, F32, False, True), (7, 13, 4, BF16, True, False),
                                                  (9, 13, 4, BF16, True, True), (6, 7, 2, F32, True, True)])
def test_step(N, D, W, dtype, silu, init):
    on, ref = make(N, 1, D, W, dtype, True, init, seed=2)
    x = on["x"].view(N, D)
    y, f = comba.short_conv_step(x, on["weight"], on["bias"], on["init"], silu=silu)
    fwd = (ref["x"], ref["weight"], ref["bias"], ref["init"])
    ry, rf = layer.short_conv(*fwd, silu=silu)
    size, _ = layer.short_conv(*fwd, magnitude=True)
    check("y", y.view(N, 1, D), ry, size, conv_gamma(W, size.max()))
    assert np.array_equal(f.double().cpu().numpy(), rf)
    if init:  # in place
        state = on["init"].clone()
        y2, f2 = comba.short_conv_step(x, on["weight"], on["bias"], state, silu=silu, in_place=True)
        assert f2 is state and torch.equal(f2, f) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_steps_continue_a_prompt_bit_for_bit(dtype):
    on, _ = make(3, 21, 40, 4, dtype, True, True, seed=3)
    w, b = on["weight"], on["bias"]
    whole, fin = comba.short_conv(on["x"], w, b, on["init"])
    head, state = comba.short_conv(on["x"][:, :10].contiguous(), w, b, on["init"])
    assert torch.equal(head, whole[:, :10])
    for t in range(10, 21):
        y, state = comba.short_conv_step(on["x"][:, t].contiguous(), w, b, state, in_place=True)
        assert torch.equal(y, whole[:, t])
    assert torch.equal(state, fin)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_outside_the_sequences_are_left_alone(dtype):
    on, _ = make(1, 40, 16, 4, dtype, True, False, [40], seed=4)
    out = torch.full_like(on["x"], 7.0)
    cu = torch.tensor([3, 10, 30], dtype=torch.int32, device="cuda")
    poison = on["x"].clone()
    poison[:, :3] = float("nan")
    poison[:, 30:] = float("nan")
    comba.short_conv(poison, on["weight"], on["bias"], None, cu, out=out)
    assert torch.all(out[:, :3] == 7) and torch.all(out[:, 30:] == 7) and torch.isfinite(out).all()
    g = comba.short_conv_bwd(poison, on["weight"], on["bias"], on["dy"], None, cu)
    assert torch.isfinite(g["dweight"]).all() and torch.isfinite(g["dx"][:, 3:30]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_addresses_off_the_16_byte_grid_give_the_same(dtype):
    on, _ = make(2, 33, 64, 4, dtype, True, True, seed=5)
    base = torch.empty(on["x"].numel() + 1, dtype=dtype, device="cuda")
    shifted = base[1:].view_as(on["x"])
    shifted.copy_(on["x"])
    a, fa = comba.short_conv(on["x"], on["weight"], on["bias"], on["init"])
    b, fb = comba.short_conv(shifted, on["weight"], on["bias"], on["init"])
    assert torch.equal(a, b) and torch.equal(fa, fb)
    g = comba.short_conv_bwd(on["x"], on["weight"], on["bias"], on["dy"], on["init"])
    h = comba.short_conv_bwd(shifted, on["weight"], on["bias"], on["dy"], on["init"])
    assert all(torch.equal(g[k], h[k]) for k in g)


def test_values_at_the_edge():
    """Large inputs saturate the SiLU instead of overflowing; an infinity or NaN reaches the tokens
    that see it and no others."""
    x = torch.zeros(1, 12, 8, device="cuda")
    x[0, 2] = 3e4
    x[0, 5] = -3e4
    w = torch.zeros(8, 4, device="cuda")
    w[:, 3] = 1.0
    y, _ = comba.short_conv(x, w)
    assert torch.all(y[0, 2] == 3e4) and torch.all(y[0, 5].abs() == 0)
    x[0, 2] = float("inf")
    x[0, 5] = float("nan")
    w[:, 2] = 1.0
    y, _ = comba.short_conv(x, w)
    # tokens 2 .. 5 see the infinity, 4 and 5 through taps of weight 0: 0 * inf is NaN; 5 .. 8 see the NaN
    assert torch.all(torch.isinf(y[0, 2:4])) and torch.all(torch.isnan(y[0, 4:9]))
    assert torch.all(y[0, :2] == 0) and torch.all(y[0, 9:] == 0)


@pytest.mark.parametrize("dtype,D", [(BF16, 8), (BF16, 9), (BF16, 23), (F32, 5), (F32, 7), (F32, 4)])
def test_ragged_channels_equal_those_of_a_wider_tensor(dtype, D):
    """Every channel is computed by itself: the same bits beside whatever channels."""
    wide = 24
    on, _ = make(2, 37, wide, 4, dtype, True, True, seed=31)
    cut = {k: v if v is None else v[:D].contiguous() if k in ("weight", "bias") else v[..., :D].contiguous()
           for k, v in on.items()}
    a, b = (comba.short_conv(v["x"], v["weight"], v["bias"], v["init"]) for v in (on, cut))
    assert all(torch.equal(p[..., :D], q) for p, q in zip(a, b))
    a, b = (comba.short_conv_step(v["x"][:, 0].contiguous(), v["weight"], v["bias"], v["init"]) for v in (on, cut))
    assert all(torch.equal(p[..., :D], q) for p, q in zip(a, b))
    a, b = (comba.short_conv_bwd(v["x"], v["weight"], v["bias"], v["dy"], v["init"], d_final_state=v["dfin"])
            for v in (on, cut))
    for k in a:
        p = a[k][:D] if k in ("dweight", "dbias") else a[k][..., :D]
        assert torch.equal(p, b[k]), k
