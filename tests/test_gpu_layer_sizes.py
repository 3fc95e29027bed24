"""The layer operators on tensors of more than 2^31 elements (offsets past 32 bits) and on batches of
thousands of short sequences. The ends of the large tensors are compared with calls on copies of the
ends; the many sequences with the fp64 oracle."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, both, check, conv_bwd_gamma, conv_gamma, cu_of, cu_dev, half_A, layer, rnd, scan_gamma

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def big(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(generator=g)


def params(D, S=16):
    r = rnd(1)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    return dict(w=t(r.normal(size=(D, 4))), b=t(r.normal(size=D)), A=t(-np.exp(r.normal(size=(D, S)))),
                skip=t(r.normal(size=D)), bias=t(np.full(D, -2.0)))


def test_short_conv_past_2_31_elements():
    D, T = 4096, (1 << 19) + 100
    x, p = big(1, T, D), params(D)
    assert x.numel() > 1 << 31
    y, f = comba.short_conv(x, p["w"], p["b"])
    tail = x[:, -200:].contiguous()
    ty, tf = comba.short_conv(tail, p["w"], p["b"])
    assert torch.equal(y[:, -197:], ty[:, 3:]) and torch.equal(f, tf)
    del y
    dy = big(1, T, D, seed=1)
    g = comba.short_conv_bwd(x, p["w"], p["b"], dy)
    h = comba.short_conv_bwd(tail, p["w"], p["b"], dy[:, -200:].contiguous())
    assert torch.equal(g["dx"][:, -197:], h["dx"][:, 3:])


def test_block_norm_past_2_31_elements():
    D, R = 4096, (1 << 19) + 33
    x, g = big(R, D), big(R, D, seed=1)
    w = torch.ones(D, device="cuda") * 1.5
    r, n = comba.block_norm(x, gate=g, post_weight=w, pre_weight=w)
    tr, tn = comba.block_norm(x[-40:].contiguous(), gate=g[-40:].contiguous(), post_weight=w, pre_weight=w)
    assert torch.equal(r[-40:], tr) and torch.equal(n[-40:], tn)
    del r, n
    a = comba.block_norm_bwd(x, g, gate=g, post_weight=w)
    b = comba.block_norm_bwd(x[-40:].contiguous(), g[-40:].contiguous(), gate=g[-40:].contiguous(), post_weight=w)
    assert torch.equal(a["dy"][-40:], b["dy"]) and torch.equal(a["dgate"][-40:], b["dgate"])


def test_selective_scan_past_2_31_elements():
    """A batch whose last sequence lies past 2^31 elements, uncut and cut, against that sequence alone."""
    B, T, D = 9, 65536, 4096
    p = params(D)
    x, dt = big(B, T, D), big(B, T, D, seed=1)
    Bm, Cm = big(B, T, 1, 16, seed=2), big(B, T, 1, 16, seed=3)
    assert x.numel() > 1 << 31
    y, f = comba.selective_scan(x, dt, p["A"], Bm, Cm, p["skip"], None, p["bias"])
    last = [t[-1:].contiguous() for t in (x, dt, Bm, Cm)]
    ty, tf = comba.selective_scan(last[0], last[1], p["A"], last[2], last[3], p["skip"], None, p["bias"])
    # the one sequence alone is cut along time: the same formulas, carried in another order
    assert (f[-1:] - tf).norm() / tf.norm() < 1e-5
    assert (y[-1:].float() - ty.float()).norm() / ty.float().norm() < 2.0 ** -8
    del y, ty
    cu = torch.tensor([0, B * T - 300, B * T], dtype=torch.int32, device="cuda")   # packed: cut
    flat = [t.view(1, B * T, *t.shape[2:]) for t in (x, dt, Bm, Cm)]
    y, f = comba.selective_scan(flat[0], flat[1], p["A"], flat[2], flat[3], p["skip"], None, p["bias"], cu_seqlens=cu)
    tail = [t[:, -300:].contiguous() for t in flat]
    ty, tf = comba.selective_scan(tail[0], tail[1], p["A"], tail[2], tail[3], p["skip"], None, p["bias"])
    assert (f[1:] - tf).norm() / tf.norm() < 1e-5
    assert (y[:, -300:].float() - ty.float()).norm() / ty.float().norm() < 2.0 ** -8


def test_selective_scan_backward_past_2_31_elements():
    B, T, D = 9, 65536, 4096
    p = params(D, 4)
    x, dt, dy = big(B, T, D), big(B, T, D, seed=1), big(B, T, D, seed=4)
    Bm, Cm = big(B, T, 1, 4, seed=2), big(B, T, 1, 4, seed=3)
    g = comba.selective_scan_bwd(x, dt, p["A"], Bm, Cm, dy, p["skip"], None, p["bias"])
    h = comba.selective_scan_bwd(*[t[-1:].contiguous() if t.dim() > 2 else t for t in (x, dt, p["A"], Bm, Cm, dy)],
                                 p["skip"], None, p["bias"])
    for k in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(g[k][-1:], h[k]), k


def test_steps_past_2_31_states():
    N, D = 1 << 16, 2056
    p = params(D)
    x, dt, Bm, Cm = big(N, D), big(N, D, seed=1), big(N, 1, 16, seed=2), big(N, 1, 16, seed=3)
    st = torch.empty(N, D, 16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    assert st.numel() > 1 << 31
    tail = [t[-3:].contiguous() for t in (x, dt, Bm, Cm, st)]
    ty, ts = comba.selective_step(tail[0], tail[1], p["A"], tail[2], tail[3], p["skip"], None, p["bias"], initial_state=tail[4])
    y, f = comba.selective_step(x, dt, p["A"], Bm, Cm, p["skip"], None, p["bias"], initial_state=st, in_place=True)
    assert torch.equal(y[-3:], ty) and torch.equal(f[-3:], ts)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_thousands_of_short_sequences(dtype):
    r = rnd(6)
    lens = r.integers(0, 5, size=3000)
    T, D, S, N = int(lens.sum()), 24, 8, len(lens)
    cu = cu_of(lens)
    v = dict(x=r.normal(size=(1, T, D)), w=r.normal(size=(D, 4)), b=r.normal(size=D), init=r.normal(size=(N, 3, D)),
             dy=r.normal(size=(1, T, D)), dfin=r.normal(size=(N, 3, D)))
    on, ref = both(v, dtype, ("w", "b"))
    fwd = (ref["x"], ref["w"], ref["b"], ref["init"])
    y, f = comba.short_conv(on["x"], on["w"], on["b"], on["init"], cu_dev(cu))
    size = layer.short_conv(*fwd, cu=cu, magnitude=True)[0]
    ry, rf = layer.short_conv(*fwd, cu=cu)
    check("conv y", y, ry, size, conv_gamma(4, size.max()))
    assert np.array_equal(f.double().cpu().numpy(), rf)
    g = comba.short_conv_bwd(on["x"], on["w"], on["b"], on["dy"], on["init"], cu_dev(cu), d_final_state=on["dfin"])
    kw = dict(cu=cu, dy=ref["dy"], dfin=ref["dfin"])
    want, mag = layer.short_conv(*fwd, **kw), layer.short_conv(*fwd, **kw, magnitude=True)
    for k in want:
        check(k, g[k], want[k], mag[k], conv_bwd_gamma(4, size.max(), T if k in ("dweight", "dbias") else 0))

    v = dict(x=v["x"], dt=r.normal(size=(1, T, D)), A=-np.exp(r.normal(size=(D, S))), Bm=r.normal(size=(1, T, 1, S)),
             Cm=r.normal(size=(1, T, 1, S)), init=r.normal(size=(N, D, S)), dy=v["dy"], dfin=r.normal(size=(N, D, S)))
    on, ref = both(v, dtype, ("A", "init", "dfin"))
    args = [on[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    rargs = lambda q: [q[k] for k in ("x", "dt", "A", "Bm", "Cm")]  # noqa: E731
    y, f = comba.selective_scan(*args, initial_state=on["init"], cu_seqlens=cu_dev(cu))
    kw = dict(init=ref["init"], cu=cu)
    ry, rf = layer.selective_scan(*rargs(ref), **kw)
    my, mf = layer.selective_scan(*rargs(half_A(ref)), **kw, magnitude=True)
    um = float(np.abs(ref["dt"]).max())
    check("scan y", y, ry, my, scan_gamma(4, um))
    check("scan state", f, rf, mf, scan_gamma(4, um))
    g = comba.selective_scan_bwd(*args, on["dy"], initial_state=on["init"], cu_seqlens=cu_dev(cu), d_final_state=on["dfin"])
    kw.update(dy=ref["dy"], dfin=ref["dfin"])
    want, mag = layer.selective_scan(*rargs(ref), **kw), layer.selective_scan(*rargs(half_A(ref)), **kw, magnitude=True)
    for k in want:
        if want[k] is not None:   # ddt: half of A in its own factor too
            check(k, g[k], want[k], mag[k] * (2 if k == "ddt" else 1), scan_gamma(4, um, T if k == "dA" else D, ways=2))
