"""The selective scan cut along time with several groups of B and C and with every number of states per lane,
packed batches in groups forward and backward, and the single-token form where a workgroup takes several
sequences. Inputs and bounds as in test_gpu_selective_scan.py."""
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, check, cu_dev, cu_of, half_A, layer, scan_gamma
from test_gpu_selective_scan import PARAMS, args_of, make, opts, oracle_args, umax

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


CUT = [  # B, T, D, S, G, dtype, softplus, lens, without
    (1, 300, 70, 17, 1, F32, True, None, ()), (2, 270, 40, 32, 2, BF16, True, None, ("init",)),
    (1, 450, 33, 33, 3, F32, True, None, ()), (1, 300, 66, 64, 1, BF16, True, None, ("z",)),
    (1, 290, 64, 64, 2, F32, True, None, ("skip", "dt_bias")), (1, 515, 66, 16, 3, F32, True, None, ()),
    (2, 400, 130, 5, 2, BF16, True, None, ()),
    (1, 600, 48, 16, 3, F32, True, [3, 0, 270, 64, 1, 262], ()), (1, 500, 70, 32, 2, F32, True, [350, 0, 150], ()),
    (1, 400, 36, 64, 3, BF16, True, [0, 129, 1, 270, 0], ("init",)), (1, 420, 66, 17, 3, BF16, True, [65, 355], ()),
    (1, 333, 150, 3, 2, F32, False, [333], ()),
]


@pytest.mark.parametrize("B,T,D,S,G,dtype,softplus,lens,without", CUT)
def test_forward_cut_along_time(B, T, D, S, G, dtype, softplus, lens, without):
    assert comba.selective_scan_workspace_size(B, T, D, S, G, len(lens or ())) > 0
    on, ref = make(B, T, D, S, G, dtype, lens, without, softplus=softplus)
    cu = cu_of(lens)
    y, f = comba.selective_scan(*args_of(on), **opts(on), softplus=softplus, cu_seqlens=cu_dev(cu))
    o = oracle_args(ref, softplus, cu)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    gamma = scan_gamma(T if lens is None else max(lens), umax(ref))
    check("y", y, ry, my, gamma)
    check("state", f, rf, mf, gamma)


BACKWARD = CUT + [
    (1, 100, 48, 16, 3, F32, True, [1, 0, 17, 16, 66], ()),                  # segments of 16 tokens
    (1, 14, 48, 16, 3, BF16, True, [3, 0, 11], ()),                          # packed, whole
    (1, 900, 512, 16, 4, F32, True, [k % 31 for k in range(40)] + [399], ()),
]


@pytest.mark.parametrize("B,T,D,S,G,dtype,softplus,lens,without", BACKWARD)
def test_backward(B, T, D, S, G, dtype, softplus, lens, without):
    on, ref = make(B, T, D, S, G, dtype, lens, without, seed=1, softplus=softplus)
    cu = cu_of(lens)
    call = dict(**opts(on), softplus=softplus, cu_seqlens=cu_dev(cu), d_final_state=on["dfin"])
    g = comba.selective_scan_bwd(*args_of(on), on["dy"], **call)
    o = dict(**oracle_args(ref, softplus, cu), dy=ref["dy"], dfin=ref["dfin"])
    r = layer.selective_scan(*args_of(ref), **o)
    m = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    for k in r:
        adds = D // G if k in ("dB", "dC") else B * T if k in ("dA", "dskip", "ddt_bias") else 0
        # ddt: half of A in its own factor
        check(k, g[k], r[k], None if m[k] is None else m[k] * (2 if k in ("ddt", "ddt_bias") else 1),
              scan_gamma(T if lens is None else max(lens), umax(ref), adds, ways=2))
    again = comba.selective_scan_bwd(*args_of(on), on["dy"], **call)
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)


@pytest.mark.parametrize("N,D,S,G,dtype,without,per", [
    (411, 640, 16, 1, BF16, (), 2), (617, 640, 13, 1, F32, ("z",), 3), (1707, 210, 4, 3, BF16, ("skip",), 5),
    (613, 640, 33, 1, F32, ("dt_bias",), 2), (1027, 2048, 8, 1, BF16, (), 16), (3281, 640, 7, 1, F32, ("init",), 16)])
def test_step_with_several_sequences_per_workgroup(N, D, S, G, dtype, without, per):
    blocks = G * -(-D // G // 64)
    assert min(16, N * blocks // 2048) == per and N % per   # the last workgroup takes fewer
    on, ref = make(N, 1, D, S, G, dtype, None, without, seed=2)
    flat = {k: (None if v is None else v if k in PARAMS else v[:, 0].contiguous()) for k, v in on.items()}
    y, f = comba.selective_step(*args_of(flat), **opts(flat))
    o = oracle_args(ref, True, None)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    check("y", y[:, None], ry, my, scan_gamma(1, umax(ref)))
    check("state", f, rf, mf, scan_gamma(1, umax(ref)))
    if flat["init"] is not None:
        kw = opts(flat)
        kw["initial_state"] = state = flat["init"].clone()
        y2, f2 = comba.selective_step(*args_of(flat), **kw, in_place=True)
        assert f2 is state and torch.equal(f2, f) and torch.equal(y2, y)
