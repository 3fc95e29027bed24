"""Group norm (over tokens and over sequences, backward) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, U, both, check, cu_dev, cu_of, layer, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(B, T, D, dtype, weight=True, bias=True, seed=0, mean=0.5):
    r = rnd(seed)
    v = dict(x=r.normal(size=(B, T, D)) + mean, weight=r.normal(size=D) if weight else None,
             bias=r.normal(size=D) if bias else None, dy=r.normal(size=(B, T, D)))
    return both(v, dtype, ("weight", "bias"))


def gamma(n, backward=False, adds=0, far=0.0):
    """Roundings in units of 2^-24. A sum of n values goes through registers, lanes and tiles: at most 64 additions of
    a thread (512 tokens over 4 rows: 128), 6 + 8 joins of about 6 roundings, so 220; the deviation halves the
    relative error of the variance but counts the mean's too; 24 for the root, the products and the
    sigmoid (its argument's 2 |p| is within the magnitude's 1.1 |p| for |p| <= 20). `far`: sums about a
    thread's first value are as exact as that value is near the mean, twice the deviation or so."""
    return U * (2 * 220 * (2 if backward else 1) + 48 + adds)


CASES = [  # B, T, D, G, dtype, silu, lens, weight, bias
    (1, 1, 1, 1, F32, False, None, True, True),
    (5, 1, 64, 8, BF16, True, None, True, True),
    (70, 1, 2048, 16, BF16, True, None, True, True),
    (33, 1, 66, 3, F32, True, None, True, False),
    (9, 1, 2047, 1, F32, True, None, False, True),
    (40, 1, 40, 5, BF16, False, None, False, False),
    (3, 1, 1024, 1, BF16, True, None, True, True),
    (2, 1, 8192, 1, BF16, True, None, True, True),
    (2, 1, 8200, 1, F32, True, None, True, True),        # wider than the form in registers
    (300, 1, 96, 6, F32, True, None, True, True),
    (2, 2, 8, 2, F32, True, None, True, True),
    (2, 37, 64, 8, BF16, True, None, True, True),
    (1, 300, 1001, 7, F32, True, None, True, True),
    (3, 130, 48, 48, BF16, False, None, True, True),     # a group per channel
    (2, 200, 1000, 1, BF16, True, None, True, False),    # one group over several channel blocks
    (1, 700, 1536, 2, F32, True, None, False, False),
    (1, 65, 129, 3, BF16, True, None, True, True),
    (1, 150, 64, 4, F32, True, [0, 1, 40, 0, 33, 76, 0], True, True),
    (1, 500, 520, 5, BF16, True, [3, 400, 0, 97], True, True),
    (1, 6, 33, 11, F32, True, [1, 1, 1, 1, 1, 1], True, True),
    (1, 0, 16, 2, F32, True, [0, 0], True, True),
]


@pytest.mark.parametrize("B,T,D,G,dtype,silu,lens,weight,bias", CASES)
def test_forward_and_backward(B, T, D, G, dtype, silu, lens, weight, bias):
    on, ref = make(B, T, D, dtype, weight, bias)
    cu = cu_of(lens)
    rows = T == 1 and lens is None
    x, dy = (on[k][:, 0] if rows else on[k] for k in ("x", "dy"))
    kw = dict(weight=on["weight"], bias=on["bias"], cu_seqlens=cu_dev(cu), silu=silu)
    okw = dict(groups=G, weight=ref["weight"], bias=ref["bias"], silu=silu, cu=cu)
    y, stats = comba.group_norm(x, G, **kw)
    ry, rs = layer.group_norm(ref["x"], **okw)
    my, ms = layer.group_norm(ref["x"], **okw, magnitude=True)
    n = D // G * T
    check("y", y.view(B, T, D), ry, my, gamma(n))
    check("mean", stats[..., 0], rs[..., 0], ms[..., 0], gamma(n))
    check("rstd", stats[..., 1], rs[..., 1], rs[..., 1], gamma(n))
    got = comba.group_norm_bwd(x, dy, stats, G, **kw)
    r, m = layer.group_norm(ref["x"], **okw, dy=ref["dy"]), layer.group_norm(ref["x"], **okw, dy=ref["dy"], magnitude=True)
    check("dx", got["dx"].view(B, T, D), r["dx"], m["dx"], gamma(n, True))
    check("dweight", got["dweight"], r["dweight"], m["dweight"], gamma(n, True, B * T))
    check("dbias", got["dbias"], r["dbias"], m["dbias"], gamma(n, True, B * T))


@pytest.mark.parametrize("T", [1, 300])
def test_far_mean(T):
    """A mean of 1000 deviations: the moments are taken about a value near it, so the result is as exact as x."""
    on, ref = make(4, T, 256, F32, mean=1000.0)
    x = on["x"][:, 0] if T == 1 else on["x"]
    y, stats = comba.group_norm(x, 4, on["weight"], on["bias"])
    ry, rs = layer.group_norm(ref["x"], 4, ref["weight"], ref["bias"])
    my, _ = layer.group_norm(ref["x"], 4, ref["weight"], ref["bias"], magnitude=True)
    check("y", y.view(4, T, 256), ry, my, U * 8)  # the mean's own rounding, relative to |x|, and a few of its sum
    # sums of distances from near values: of the deviation's size, so the count of the other tests holds, and the
    # mean's error of 8 2^-24 1000 deviations adds its square, 2e-7
    check("rstd", stats[..., 1], rs[..., 1], rs[..., 1], gamma(64 * T) + 4e-7)
