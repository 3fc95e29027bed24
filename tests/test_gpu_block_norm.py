"""The norms after and before a block, fused with gate, scale and residual, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, both, check, layer, norm_gamma, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


PARTS = ("gate", "residual", "scale", "post_weight", "pre_weight")
ALL = PARTS
HEADS = ("gate", "post_weight")


def make(R, D, dtype, parts, seed=0):
    r = rnd(seed)
    v = dict(y=r.normal(size=(R, D)), dr=r.normal(size=(R, D)), dn=r.normal(size=(R, D)))
    for p in parts:
        v[p] = r.normal(size=(R, D)) if p in ("gate", "residual") else r.normal(size=D) * 0.2 + 1
    on, ref = both(v, dtype, ("scale", "post_weight", "pre_weight"))
    for p in PARTS:
        on.setdefault(p, None)
        ref.setdefault(p, None)
    return on, ref


def given(v):
    return {p: v[p] for p in PARTS}


CASES = [  # rows, D, dtype, parts
    (1, 1, F32, ALL), (3, 3, BF16, ALL), (5, 8, F32, HEADS), (100, 63, BF16, ALL), (70, 64, BF16, HEADS),
    (33, 65, F32, ALL), (257, 128, BF16, HEADS), (40, 128, F32, ("post_weight",)), (31, 200, BF16, ALL),
    (9, 256, BF16, ("gate", "residual")), (17, 512, F32, ALL), (12, 1000, BF16, ("residual", "pre_weight")),
    (8, 1024, F32, ("scale", "residual")), (33, 2047, F32, ALL), (20, 2048, BF16, ALL),
    (5, 2048, F32, ("pre_weight",)), (6, 4096, BF16, ALL), (3, 5000, F32, ("post_weight", "residual")),
    (4, 8192, BF16, ALL), (3, 16384, F32, ALL), (2, 16383, BF16, ("pre_weight", "residual")),
    (5000, 128, BF16, ("gate", "post_weight", "scale")), (3000, 2048, BF16, ALL),
    (1500, 1030, BF16, ("post_weight",)), (1500, 1030, F32, ("pre_weight", "gate")),
]


@pytest.mark.parametrize("R,D,dtype,parts", CASES)
def test_forward(R, D, dtype, parts):
    on, ref = make(R, D, dtype, parts)
    r, n = comba.block_norm(on["y"], **given(on))
    rr, rn = layer.block_norm(ref["y"], **given(ref))
    mr, mn = layer.block_norm(ref["y"], **given(ref), magnitude=True)
    check("r", r, rr, mr, norm_gamma())
    check("n", n, rn, mn, norm_gamma())


@pytest.mark.parametrize("which", ["both", "dr", "dn"])
@pytest.mark.parametrize("R,D,dtype,parts", CASES)
def test_backward(R, D, dtype, parts, which):
    if which == "dn" and "pre_weight" not in parts:
        pytest.skip("no norm behind the block")
    on, ref = make(R, D, dtype, parts, seed=1)
    dr, dn = which != "dn", which != "dr" and "pre_weight" in parts
    g = comba.block_norm_bwd(on["y"], on["dr"] if dr else None, on["dn"] if dn else None, **given(on))
    args = dict(**given(ref), dr=ref["dr"] if dr else None, dn=ref["dn"] if dn else None)
    r, m = layer.block_norm(ref["y"], **args), layer.block_norm(ref["y"], **args, magnitude=True)
    assert set(g) == set(r)
    for k in r:
        check(k, g[k], r[k], m[k], norm_gamma(R if k in ("dscale", "dpost_weight", "dpre_weight") else 0, True))
    again = comba.block_norm_bwd(on["y"], on["dr"] if dr else None, on["dn"] if dn else None, **given(on))
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)


def test_any_leading_shape_and_no_rows():
    on, _ = make(24, 64, BF16, HEADS)
    r, n = comba.block_norm(on["y"], gate=on["gate"], post_weight=on["post_weight"])
    r4, _ = comba.block_norm(on["y"].view(2, 3, 4, 64), gate=on["gate"].view(2, 3, 4, 64), post_weight=on["post_weight"])
    assert n is None and r4.shape == (2, 3, 4, 64) and torch.equal(r4.view(24, 64), r)
    none = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    r, n = comba.block_norm(none, pre_weight=w)
    assert r.shape == n.shape == (0, 64)
    g = comba.block_norm_bwd(none, none, none, pre_weight=w, post_weight=w)
    assert g["dy"].shape == (0, 64) and torch.all(g["dpre_weight"] == 0) and torch.all(g["dpost_weight"] == 0)


@pytest.mark.parametrize("D", [64, 128, 1024, 2048])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_addresses_off_the_16_byte_grid(D, dtype):
    on, ref = make(9, D, dtype, ALL, seed=2)
    base = torch.empty(9 * D + 1, dtype=dtype, device="cuda")
    y = base[1:].view(9, D)
    y.copy_(on["y"])
    got = comba.block_norm(y, **given(on))
    want, mag = layer.block_norm(ref["y"], **given(ref)), layer.block_norm(ref["y"], **given(ref), magnitude=True)
    for k in range(2):
        check("rn"[k], got[k], want[k], mag[k], norm_gamma())
    g = comba.block_norm_bwd(y, on["dr"], on["dn"], **given(on))
    args = dict(**given(ref), dr=ref["dr"], dn=ref["dn"])
    want, mag = layer.block_norm(ref["y"], **args), layer.block_norm(ref["y"], **args, magnitude=True)
    for k in g:
        check(k, g[k], want[k], mag[k], norm_gamma(9, True))


def test_rows_of_zeros_and_large_values():
    w = torch.ones(128, device="cuda")
    y = torch.zeros(3, 128, device="cuda")
    y[1] = 1e15          # squares of 1e30 still fit
    y[2] = float("nan")
    r, n = comba.block_norm(y, post_weight=w, pre_weight=w, eps=1e-6)
    assert torch.all(r[0] == 0) and torch.all(n[0] == 0)
    assert (r[1] - 1).abs().max() < 1e-5 and (n[1] - 1).abs().max() < 1e-5
    assert torch.isnan(r[2]).all() and torch.isnan(n[2]).all()   # and no other row
    g = comba.block_norm_bwd(y[:1], y[:1] + 1, y[:1] + 1, post_weight=w, pre_weight=w)
    assert torch.isfinite(g["dy"]).all()
