"""Growing states (A > 0) in a scan that is cut along time: the product of a segment's decays may
leave float32's range while the state or the gradient that it multiplies is 0 or tiny, and then the
result is finite, as it is without a cut.

Some channels grow, the others decay. Exponents are counted as in test_growing_states_are_allowed: every
rounding of the error bound once more per unit of the exponent X along which a value is carried. The
magnitudes are the oracle's with A / 2 for the decays and A itself for the growing channels."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, both, check, cu_dev, cu_of, layer, rnd, scan_gamma
from test_gpu_selective_scan import PARAMS, args_of, opts, oracle_args, umax

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ranges(B, T, lens):
    cu = cu_of(lens)
    return [(b, 0, T) for b in range(B)] if lens is None else [(0, int(s), int(e)) for s, e in zip(cu, cu[1:])]


def make(B, T, D, S, G, dtype, lens, rate, edit, softplus=True, seed=0):
    """Inputs whose first third of channels grows by exponents of about `rate` per token; edit(v, grow) sets
    their values. Returns tensors, exact values and the largest exponent of a token."""
    r = rnd(seed)
    N = B if lens is None else len(lens)
    grow = np.arange(D) < (D + 2) // 3
    v = dict(x=r.normal(size=(B, T, D)), dt=r.normal(size=(B, T, D)) * 0.5, A=-np.exp(r.normal(size=(D, S)) * 0.7),
             Bm=r.normal(size=(B, T, G, S)), Cm=r.normal(size=(B, T, G, S)), skip=r.normal(size=D),
             z=r.normal(size=(B, T, D)), dt_bias=r.uniform(-4, 0, size=D), init=r.normal(size=(N, D, S)),
             dy=r.normal(size=(B, T, D)), dfin=r.normal(size=(N, D, S)))
    # step sizes of 2 to 2.2 in the growing channels (dt alone, or softplus of it)
    v["dt"][..., grow] = r.uniform(0, 0.2, size=(B, T, int(grow.sum())))
    v["dt_bias"][grow] = 1.86 if softplus else 2.0
    if not softplus:
        v["dt"][..., ~grow] = np.abs(v["dt"][..., ~grow]) * 0.3
        v["dt_bias"][~grow] = np.abs(v["dt_bias"][~grow]) * 0.02
    v["A"][grow] = rate / 2.0 * r.uniform(0.9, 1.0, size=(int(grow.sum()), S))
    edit(v, grow)
    on, ref = both(v, dtype, PARAMS)
    u = ref["dt"] + ref["dt_bias"]
    d = layer.softplus(u) if softplus else u
    return on, ref, grow, float((d[..., grow].max() if T else 0) * ref["A"].max())


def magnitude_args(ref):
    return args_of({**ref, "A": np.where(ref["A"] < 0, ref["A"] / 2, ref["A"])})


def forward(on, ref, lens, softplus, steps, X):
    cu = cu_of(lens)
    y, f = comba.selective_scan(*args_of(on), **opts(on), softplus=softplus, cu_seqlens=cu_dev(cu))
    o = oracle_args(ref, softplus, cu)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*magnitude_args(ref), **o, magnitude=True)
    gamma = scan_gamma(steps, umax(ref)) * (1 + X)
    check("y", y, ry, my, gamma)
    check("state", f, rf, mf, gamma)


def backward(on, ref, lens, softplus, steps, X, D, G, tokens):
    cu = cu_of(lens)
    call = dict(**opts(on), softplus=softplus, cu_seqlens=cu_dev(cu), d_final_state=on["dfin"])
    g = comba.selective_scan_bwd(*args_of(on), on["dy"], **call)
    o = dict(**oracle_args(ref, softplus, cu), dy=ref["dy"], dfin=ref["dfin"])
    r = layer.selective_scan(*args_of(ref), **o)
    m = layer.selective_scan(*magnitude_args(ref), **o, magnitude=True)
    for k in r:
        adds = D // G if k in ("dB", "dC") else tokens if k in ("dA", "dskip", "ddt_bias") else 0
        check(k, g[k], r[k], m[k] * (2 if k in ("ddt", "ddt_bias") else 1),
              scan_gamma(steps, umax(ref), adds, ways=2) * (1 + X))


LIVE = 18   # tokens along which a value of a growing channel is carried: X stays below 2.3 * 18 = 42


@pytest.mark.parametrize("B,T,D,S,G,dtype,softplus,lens", [
    (1, 700, 70, 16, 1, F32, True, None), (2, 515, 64, 4, 2, BF16, True, None), (1, 600, 33, 33, 1, F32, False, None),
    (1, 700, 66, 8, 1, F32, False, [200, 0, 1, 370, 129]), (1, 700, 66, 16, 3, BF16, True, [300, 400])])
def test_forward_from_a_state_of_zero(B, T, D, S, G, dtype, softplus, lens):
    """Zero state and inputs up to the last tokens of a sequence: 64 tokens multiply to e^118 and more."""
    def edit(v, grow):
        v["init"][:, grow] = 0
        for b, s, e in ranges(B, T, lens):
            v["x"][b, s:max(s, e - LIVE), grow] = 0
    on, ref, grow, per = make(B, T, D, S, G, dtype, lens, 2.05, edit, softplus)
    N = len(lens or ())
    assert comba.selective_scan_workspace_size(B, T, D, S, G, N) > 0 and 64 * 2.05 * 0.9 > 89   # cut; overflow
    forward(on, ref, lens, softplus, T, per * LIVE)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_from_a_tiny_state(dtype):
    """States of 1e-30 over a segment of 64 tokens whose decays multiply to e^108 and more: finite behind it."""
    lens = [65, 0, 66, 129, 4]
    def edit(v, grow):
        v["x"][..., grow] = 0
        v["init"][:, grow] *= 1e-30
        v["init"][3, grow] = 0   # the sequence of three segments: nothing to carry
    on, ref, grow, per = make(1, sum(lens), 48, 16, 1, dtype, lens, 1.88, edit)
    assert comba.selective_scan_workspace_size(1, sum(lens), 48, 16, 1, len(lens)) > 0 and 64 * 1.88 * 0.9 > 89
    assert per * 66 < 69 + 88
    forward(on, ref, lens, True, 129, per * 66)


BWD_LIVE = 7


@pytest.mark.parametrize("B,T,D,S,G,dtype,softplus,lens", [
    (1, 100, 70, 16, 1, F32, True, None),                 # segments of 16 tokens
    (2, 90, 64, 4, 2, BF16, True, None),
    (1, 90, 66, 8, 3, F32, False, [40, 0, 1, 49]),
    (12, 140, 512, 16, 1, F32, True, None),               # of 32
    (60, 20, 512, 64, 1, F32, True, None)])               # of 16, four tokens at a time
def test_backward_between_zeros(B, T, D, S, G, dtype, softplus, lens):
    """In the growing channels gradients reach the first tokens of a sequence only, inputs the last ones:
    16 tokens between them multiply to e^95 and more."""
    def edit(v, grow):
        v["init"][:, grow] = 0
        v["dfin"][:, grow] = 0
        for b, s, e in ranges(B, T, lens):
            v["x"][b, s:max(s, e - BWD_LIVE), grow] = 0
            v["dy"][b, min(e, s + BWD_LIVE):e, grow] = 0
    on, ref, grow, per = make(B, T, D, S, G, dtype, lens, 6.6, edit, softplus)
    assert 16 * 6.6 * 0.9 > 89 and per * BWD_LIVE < 88
    backward(on, ref, lens, softplus, T, per * BWD_LIVE, D, G, B * T)


def test_backward_of_tiny_states_and_gradients():
    """1e-30 carried forward and backward across a segment of 16 tokens that multiplies to e^95 and more."""
    lens = [17, 18, 0, 1, 40, 17]
    def edit(v, grow):
        for k in ("x", "dy"):
            v[k][..., grow] *= 1e-30
        for k in ("init", "dfin"):
            v[k][:, grow] *= 1e-30
        for k in ("x", "dy"):
            v[k][0, 36:76, grow] = 0     # the sequence of three segments: nothing to carry
        for k in ("init", "dfin"):
            v[k][4, grow] = 0
    on, ref, grow, per = make(1, sum(lens), 48, 16, 1, F32, lens, 6.6, edit)
    assert 16 * 6.6 * 0.9 > 89 and per * 18 < 69 + 80
    backward(on, ref, lens, True, 40, per * 18, 48, 1, sum(lens))


def test_a_state_of_zero_over_the_longest_segments():
    """Decays of 2^125 per token, the largest that are finite, over segments of 900 tokens and more: 2^112500."""
    N, D = 256, 64
    lens = [880] * (N - 1) + [5000]
    T = sum(lens)
    # enough sequences: segments of their mean length
    assert comba.selective_scan_workspace_size(1, T, D, 4, 1, N) > 0
    zero, one = torch.zeros(1, T, D, device="cuda"), torch.ones(1, T, D, device="cuda")
    A = torch.full((D, 4), 125 * float(np.log(2)), device="cuda")
    A[D // 2:] = -1
    bc = torch.ones(1, T, 1, 4, device="cuda")
    x = zero.clone()
    x[..., D // 2:] = 1
    y, f = comba.selective_scan(x, one, A, bc, bc, softplus=False, cu_seqlens=cu_dev(cu_of(lens)))
    assert torch.all(y[..., :D // 2] == 0) and torch.all(f[:, :D // 2] == 0)
    assert torch.isfinite(y).all() and torch.isfinite(f).all() and torch.all(f[:, D // 2:] > 1)
