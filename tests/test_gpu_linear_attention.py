"""Decayed linear attention (prompt, single token, backward) against the fp64 oracle."""
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


PARAMS = ("log_decay", "init", "dfin")


def make(B, T, H, Hk, K, V, dtype, lens=None, head=False, init=True, seed=0, decay=(0.005, 0.4)):
    r = rnd(seed)
    N = B if lens is None else len(lens)
    shape = (H,) if head else (B, T, H)
    v = dict(q=r.normal(size=(B, T, Hk, K)), k=r.normal(size=(B, T, Hk, K)) / np.sqrt(K), v=r.normal(size=(B, T, H, V)),
             log_decay=-np.exp(r.uniform(*np.log(decay), size=shape)), init=r.normal(size=(N, H, V, K)),
             do=r.normal(size=(B, T, H, V)), dfin=r.normal(size=(N, H, V, K)))
    if not init:
        v["init"] = None
    return both(v, dtype, PARAMS)


def gamma(K, V, T, dtype, exact=False, ways=1):
    """Roundings on the longest way, in units of 2^-24, against sums with half the decays: a decay counts 0.74
    (3 + 1) for its argument and exponential, and once more for every chunk's and segment's carry (T / 32
    chunks, four roundings each); a sum one for every term at most (K or V, and T tokens). A bf16 product's
    operand in two terms is off by 2^-18 = 64 units, of which a way holds one per product; in three terms
    ('exact') by less than one."""
    split = 0 if exact or dtype == F32 else 2 * 64
    return U * (ways * (max(K, V) + T + 4 * (T // 32 + 1) + 10) + split)


CASES = [  # B, T, H, Hk, K, V, dtype, lens, head, init
    (1, 1, 1, 1, 8, 8, F32, None, False, True),
    (2, 1, 2, 2, 64, 64, BF16, None, False, True),
    (1, 2, 3, 1, 9, 11, BF16, None, True, True),
    (2, 31, 2, 2, 16, 64, F32, None, False, False),
    (1, 32, 2, 1, 64, 65, F32, None, True, True),
    (2, 33, 4, 2, 65, 17, F32, None, False, True),
    (1, 63, 1, 1, 128, 128, BF16, None, False, False),
    (2, 64, 2, 2, 128, 64, BF16, None, True, True),
    (1, 65, 2, 2, 64, 128, BF16, None, False, True),
    (1, 130, 2, 2, 129, 9, BF16, None, False, True),
    (1, 100, 1, 1, 256, 256, BF16, None, False, True),
    (1, 70, 1, 1, 256, 200, F32, None, False, True),
    (2, 200, 3, 3, 72, 99, BF16, None, False, True),
    (1, 700, 2, 1, 40, 48, F32, None, False, True),                # cut along time
    (1, 900, 1, 1, 128, 32, BF16, None, True, True),
    (2, 600, 1, 1, 20, 130, BF16, None, False, False),
    (1, 150, 2, 2, 32, 16, F32, [0, 1, 40, 0, 33, 76, 0], False, True),
    (1, 1500, 2, 1, 24, 40, F32, [3, 1100, 0, 397], False, True),  # packed, some sequences cut
    (1, 1100, 1, 1, 64, 64, BF16, [550, 550], True, False),
    (1, 321, 3, 3, 64, 70, BF16, [0, 64, 0, 65, 63, 128, 1], False, True),
    (1, 0, 2, 2, 16, 16, F32, [0, 0], False, True),                # no tokens at all
    (1, 0, 2, 2, 16, 16, BF16, [0], True, False),
]


@pytest.mark.parametrize("B,T,H,Hk,K,V,dtype,lens,head,init", CASES)
def test_forward(B, T, H, Hk, K, V, dtype, lens, head, init):
    on, ref = make(B, T, H, Hk, K, V, dtype, lens, head, init)
    cu, scale = cu_of(lens), K ** -0.5
    o, f = comba.linear_attention(on["q"], on["k"], on["v"], on["log_decay"], on["init"], cu_dev(cu), scale=scale)
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    kw = dict(scale=scale, init=ref["init"], cu=cu)
    ro, rf = layer.linear_attention(*args, **kw)
    mo, mf = layer.linear_attention(*args, **kw, magnitude=True)
    check("o", o, ro, mo, gamma(K, V, T, dtype))
    check("state", f, rf, mf, gamma(K, V, T, dtype, exact=True))


@pytest.mark.parametrize("B,T,H,Hk,K,V,dtype,lens,head,init", CASES)
def test_backward(B, T, H, Hk, K, V, dtype, lens, head, init):
    on, ref = make(B, T, H, Hk, K, V, dtype, lens, head, init, seed=1)
    cu, scale = cu_of(lens), K ** -0.5
    got = comba.linear_attention_bwd(on["q"], on["k"], on["v"], on["log_decay"], on["do"], on["init"], cu_dev(cu),
                                     on["dfin"], scale=scale)
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    kw = dict(scale=scale, init=ref["init"], cu=cu, do=ref["do"], dfin=ref["dfin"])
    r, m = layer.linear_attention(*args, **kw), layer.linear_attention(*args, **kw, magnitude=True)
    for n in ("dq", "dk", "dv"):
        check(n, got[n], r[n], m[n], gamma(K, V, T, dtype) + H // Hk * U)
    check("dinitial_state", got["dinitial_state"], r["dinitial_state"], m["dinitial_state"],
          gamma(K, V, T, dtype, exact=True))
    check("dlog_decay", got["dlog_decay"], r["dlog_decay"], m["dlog_decay"], gamma(K, V, T, dtype, exact=True, ways=3))


@pytest.mark.parametrize("N,H,Hk,K,V,dtype,head", [(1, 1, 1, 8, 8, F32, False), (3, 2, 2, 64, 64, BF16, False),
                                                  (2, 4, 2, 128, 128, BF16, True), (5, 3, 1, 72, 99, F32, False),
                                                  (2, 2, 2, 255, 17, BF16, False), (1, 2, 1, 256, 256, F32, True),
                                                  (70, 16, 16, 128, 40, BF16, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(N, H, Hk, K, V, dtype, head, in_place):
    on, ref = make(N, 1, H, Hk, K, V, dtype, head=head, seed=2)
    cut = {n: on[n][:, 0].contiguous() for n in ("q", "k", "v")}
    g = on["log_decay"] if head else on["log_decay"][:, 0].contiguous()
    before = on["init"].clone()
    o, f = comba.linear_attention_step(cut["q"], cut["k"], cut["v"], g, on["init"], scale=0.3, in_place=in_place)
    assert (f is on["init"]) == in_place and (in_place or torch.equal(on["init"], before))
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    ro, rf = layer.linear_attention(*args, scale=0.3, init=ref["init"])
    mo, mf = layer.linear_attention(*args, scale=0.3, init=ref["init"], magnitude=True)
    check("o", o, ro[:, 0], mo[:, 0], U * (K / 16 + 16))
    check("state", f, rf, mf, U * 8)
    z, fz = comba.linear_attention_step(cut["q"], cut["k"], cut["v"], g, None, scale=0.3, output_final_state=False)
    assert fz is None
    ro, _ = layer.linear_attention(*args, scale=0.3)
    mo, _ = layer.linear_attention(*args, scale=0.3, magnitude=True)
    check("o from zero", z, ro[:, 0], mo[:, 0], U * (K / 16 + 16))
