"""The block norms where a workgroup takes several steps of rows: one grid pass and a ragged rest, for every
layout of a row over lanes, all parts together and single norms (whose steps end in another barrier), with
the parameter gradients that a workgroup carries along its rows."""
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, check, layer, norm_gamma
from test_gpu_block_norm import ALL, given, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# rows, D, dtype, parts; rows per step and workgroup: 32 up to 64 columns, 16, 8, 4 (512), 2 (1024), then one
CASES = [
    (40001, 64, BF16, ALL), (20003, 128, F32, ALL), (33001, 100, BF16, ("gate", "post_weight")),
    (9001, 256, BF16, ALL), (9001, 250, F32, ("residual", "pre_weight")), (5003, 512, F32, ALL),
    (5001, 1000, BF16, ALL), (5001, 1000, F32, ("post_weight",)), (2600, 1024, BF16, ("pre_weight",)),
    (600, 4096, BF16, ALL), (600, 4096, F32, ("pre_weight", "scale")), (600, 4095, F32, ("post_weight", "gate")),
    (600, 8192, BF16, ALL), (600, 5001, F32, ("post_weight", "residual")), (600, 8192, F32, ("pre_weight",)),
    (300, 16384, F32, ALL), (300, 16384, BF16, ("post_weight",)), (300, 9001, BF16, ("residual", "pre_weight")),
]


def steps(R, D, threads):
    """Steps of rows that a workgroup takes at the most, with `threads` in the whole grid at the most."""
    lanes = next(n for n, cols in ((8, 64), (16, 128), (32, 256), (64, 512), (128, 1024), (256, 2048), (512, 8192),
                                   (1024, 16384)) if D <= cols)
    block = max(lanes, 256)
    return -(-R // (block // lanes * (threads // block)))


@pytest.mark.parametrize("R,D,dtype,parts", CASES)
def test_forward(R, D, dtype, parts):
    assert steps(R, D, 1 << 18) >= 2
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
    if which == "both" and "pre_weight" not in parts:
        pytest.skip("the same as dr")
    many = steps(R, D, 1 << 17)
    blocks = comba.lib().comba_block_norm_bwd_workspace_size(R, D) // (3 * D * 4)
    assert many >= 2 and blocks * many * 32 >= R
    on, ref = make(R, D, dtype, parts, seed=1)
    dr, dn = which != "dn", which != "dr" and "pre_weight" in parts
    call = (on["y"], on["dr"] if dr else None, on["dn"] if dn else None)
    g = comba.block_norm_bwd(*call, **given(on))
    args = dict(**given(ref), dr=ref["dr"] if dr else None, dn=ref["dn"] if dn else None)
    r, m = layer.block_norm(ref["y"], **args), layer.block_norm(ref["y"], **args, magnitude=True)
    # additions on a term's way to a parameter's gradient: along the workgroup's steps, over its at most 32 rows
    # of a step, along one of 16 rows of the workgroups' sums, over the 16
    adds = many + 32 + -(-blocks // 16) + 16
    for k in r:
        check(k, g[k], r[k], m[k], norm_gamma(adds if k in ("dscale", "dpost_weight", "dpre_weight") else 0, True))
    again = comba.block_norm_bwd(*call, **given(on))
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)
