"""The selective state space scan (prompt, single token, backward) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from _layer_util import BF16, F32, both, check, cu_dev, cu_of, half_A, layer, rnd, scan_gamma

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


PARAMS = ("A", "skip", "dt_bias", "init", "dfin")
GIVEN = ("skip", "z", "dt_bias", "init")


def make(B, T, D, S, G, dtype, lens=None, without=(), seed=0, softplus=True):
    r = rnd(seed)
    N = B if lens is None else len(lens)
    v = dict(x=r.normal(size=(B, T, D)), dt=r.normal(size=(B, T, D)) * 0.5, A=-np.exp(r.normal(size=(D, S)) * 0.7),
             Bm=r.normal(size=(B, T, G, S)), Cm=r.normal(size=(B, T, G, S)), skip=r.normal(size=D),
             z=r.normal(size=(B, T, D)), dt_bias=r.uniform(-4, 0, size=D), init=r.normal(size=(N, D, S)),
             dy=r.normal(size=(B, T, D)), dfin=r.normal(size=(N, D, S)))
    if not softplus:
        v["dt"], v["dt_bias"] = np.abs(v["dt"]) * 0.3, np.abs(v["dt_bias"]) * 0.02
    for k in without:
        v[k] = None
    return both(v, dtype, PARAMS)


def args_of(v):
    return [v[k] for k in ("x", "dt", "A", "Bm", "Cm")]


def opts(on):
    return dict(skip=on["skip"], z=on["z"], dt_bias=on["dt_bias"], initial_state=on["init"])


def oracle_args(ref, softplus, cu):
    return dict(skip=ref["skip"], z=ref["z"], dt_bias=ref["dt_bias"], init=ref["init"], softplus_dt=softplus, cu=cu)


def umax(ref):
    u = ref["dt"] + (0 if ref["dt_bias"] is None else ref["dt_bias"])
    return float(np.abs(u).max()) if u.size else 0.0


CASES = [  # B, T, D, S, G, dtype, softplus, lens, without
    (1, 1, 1, 1, 1, F32, True, None, ()),
    (2, 2, 3, 4, 1, BF16, True, None, ("z",)),
    (2, 31, 64, 5, 1, F32, True, None, ("skip",)),
    (1, 32, 65, 8, 1, BF16, True, None, ("init",)),
    (3, 33, 66, 13, 3, F32, True, None, ("dt_bias",)),
    (2, 100, 130, 16, 2, BF16, True, None, ()),
    (2, 70, 40, 16, 1, F32, False, None, ()),
    (1, 64, 34, 17, 2, F32, True, None, ("z", "skip", "init", "dt_bias")),
    (2, 45, 20, 32, 1, BF16, True, None, ()),
    (1, 40, 10, 33, 1, F32, True, None, ()),
    (1, 50, 70, 64, 1, BF16, True, None, ()),
    (1, 700, 70, 16, 1, F32, True, None, ()),                                # cut along time
    (2, 515, 64, 4, 1, BF16, True, None, ("init",)),
    (1, 150, 30, 16, 1, F32, True, [0, 1, 40, 0, 33, 76, 0], ()),
    (1, 1500, 66, 8, 1, F32, True, [3, 1100, 0, 397], ()),                   # packed, one sequence cut
    (1, 1400, 64, 16, 1, BF16, True, [700, 700], ("init", "z")),
    (1, 0, 16, 16, 1, F32, True, [0, 0], ()),                                # no tokens at all
]


@pytest.mark.parametrize("B,T,D,S,G,dtype,softplus,lens,without", CASES)
def test_forward(B, T, D, S, G, dtype, softplus, lens, without):
    on, ref = make(B, T, D, S, G, dtype, lens, without, softplus=softplus)
    cu = cu_of(lens)
    y, f = comba.selective_scan(*args_of(on), **opts(on), softplus=softplus, cu_seqlens=cu_dev(cu))
    o = oracle_args(ref, softplus, cu)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    gamma = scan_gamma(T if lens is None else max(lens), umax(ref))
    check("y", y, ry, my, gamma)
    check("state", f, rf, mf, gamma)


def test_cases_cover_both_plans():
    sizes = [comba.selective_scan_workspace_size(c[0], c[1], c[2], c[3], c[4], len(c[7] or ())) for c in CASES]
    assert sum(s > 0 for s in sizes) >= 4 and sum(s == 0 for s in sizes) >= 8


BACKWARD = CASES + [  # enough sequences for segments of several pieces (16, 8 or 4 tokens each)
    (70, 40, 512, 16, 1, F32, True, None, ()),                               # whole sequences of three pieces
    (50, 140, 512, 16, 1, BF16, True, None, ()),                             # segments of 128 tokens
    (24, 140, 512, 8, 2, F32, True, None, ("init",)),                        # of 64
    (12, 140, 512, 16, 1, F32, True, None, ("z",)),                          # of 32
    (1, 100, 512, 16, 1, F32, True, [5 * (k % 4 == 0) for k in range(80)], ()),          # packed, whole
    (1, 1082, 512, 16, 1, F32, True, [k % 21 for k in range(70)] + [300, 131], ()),      # packed, two cut
    (40, 70, 512, 32, 1, F32, True, None, ()), (70, 60, 512, 32, 1, F32, True, None, ("skip",)),
    (60, 20, 512, 64, 1, F32, True, None, ()), (70, 14, 512, 64, 1, F32, False, None, ()),
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
    m = {k: None if m[k] is None else m[k] * (2 if k == "ddt" else 1) for k in m}  # half of A in its own factor
    steps = T if lens is None else max(lens)
    for k in r:
        adds = D // G if k in ("dB", "dC") else B * T if k in ("dA", "dskip", "ddt_bias") else 0
        check(k, g[k], r[k], m[k] * (2 if k == "ddt_bias" else 1) if m[k] is not None else None,
              scan_gamma(steps, umax(ref), adds, ways=2))
    again = comba.selective_scan_bwd(*args_of(on), on["dy"], **call)
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None)


@pytest.mark.parametrize("N,D,S,G,dtype,softplus,without", [
    (1, 1, 1, 1, F32, True, ()), (3, 64, 16, 1, BF16, True, ()), (5, 66, 16, 3, F32, True, ("z",)),
    (2, 70, 13, 1, BF16, False, ("skip",)), (40, 64, 32, 1, F32, True, ("dt_bias",)), (9, 12, 64, 1, BF16, True, ()),
    (7, 20, 6, 2, F32, True, ("init",)), (300, 640, 16, 1, BF16, True, ())])
def test_step(N, D, S, G, dtype, softplus, without):
    on, ref = make(N, 1, D, S, G, dtype, None, without, seed=2, softplus=softplus)
    flat = {k: (None if v is None else v if k in PARAMS else v[:, 0].contiguous()) for k, v in on.items()}
    y, f = comba.selective_step(*args_of(flat), **opts(flat), softplus=softplus)
    o = oracle_args(ref, softplus, None)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    check("y", y[:, None], ry, my, scan_gamma(1, umax(ref)))
    check("state", f, rf, mf, scan_gamma(1, umax(ref)))
    if flat["init"] is not None:
        kw = opts(flat)
        kw["initial_state"] = state = flat["init"].clone()
        y2, f2 = comba.selective_step(*args_of(flat), **kw, softplus=softplus, in_place=True)
        assert f2 is state and torch.equal(f2, f) and torch.equal(y2, y)


@pytest.mark.parametrize("T,D", [(60, 40), (700, 64)])
def test_steps_and_pieces_continue_a_prompt(T, D):
    """A prompt in two pieces, and the tail token by token, against the whole (the same formulas in
    another order: equal to twice the bound's rounding count)."""
    on, ref = make(2, T, D, 16, 1, F32, seed=3)
    tok = lambda a, b: {k: (v if v is None or k in PARAMS else v[:, a:b].contiguous()) for k, v in on.items()}  # noqa: E731
    whole, fin = comba.selective_scan(*args_of(on), **opts(on))
    cut = T - 5
    head = tok(0, cut)
    y, state = comba.selective_scan(*args_of(head), **opts(head))
    mag, mfin = layer.selective_scan(*args_of(half_A(ref)), **oracle_args(ref, True, None), magnitude=True)
    gamma = 2 * scan_gamma(T, umax(ref))
    check("head", y, whole[:, :cut].double().cpu().numpy(), mag[:, :cut], gamma)
    for t in range(cut, T):
        s = {k: (v if v is None or k in PARAMS else v[:, t].contiguous()) for k, v in on.items()}
        s["init"] = state
        y, state = comba.selective_step(*args_of(s), **opts(s), in_place=True)
        check(f"token {t}", y, whole[:, t].double().cpu().numpy(), mag[:, t], gamma)
    check("state", state, fin.double().cpu().numpy(), mfin, gamma)


@pytest.mark.parametrize("T", [50, 700])
def test_state_may_be_updated_in_place(T):
    on, _ = make(2, T, 64, 16, 1, F32, seed=4)
    y, f = comba.selective_scan(*args_of(on), **opts(on))
    kw = opts(on)
    kw["initial_state"] = state = on["init"].clone()
    y2, f2 = comba.selective_scan(*args_of(on), **kw, final_state=state)
    assert f2 is state and torch.equal(f, f2) and torch.equal(y, y2)


@pytest.mark.parametrize("T,cu", [(60, [3, 10, 50]), (1500, [1, 1300, 1400])])
def test_rows_outside_the_sequences_are_left_alone(T, cu):
    on, _ = make(1, T, 64, 16, 1, F32, [T], ("init",), seed=5)
    a, z = cu[0], cu[-1]
    for k in ("x", "dt", "z", "Bm", "Cm", "dy"):
        on[k][:, :a] = float("nan")
        on[k][:, z:] = float("nan")
    out = torch.full_like(on["x"], 7.0)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    _, f = comba.selective_scan(*args_of(on), skip=on["skip"], z=on["z"], dt_bias=on["dt_bias"], cu_seqlens=cud, out=out)
    assert torch.all(out[:, :a] == 7) and torch.all(out[:, z:] == 7) and torch.isfinite(out).all()
    assert torch.isfinite(f).all()
    g = comba.selective_scan_bwd(*args_of(on), on["dy"], skip=on["skip"], z=on["z"], dt_bias=on["dt_bias"], cu_seqlens=cud)
    assert all(torch.isfinite(g[k]).all() for k in ("dA", "dskip", "ddt_bias"))
    assert all(torch.isfinite(g[k][:, a:z]).all() for k in ("dx", "ddt", "dz", "dB", "dC"))


def test_step_sizes_at_both_ends():
    """softplus at large negative arguments keeps its relative accuracy, at large positive ones it is
    the argument; a decay that underflows leaves the input alone."""
    dt = torch.tensor([-80.0, -30.0, -7.0, 0.0, 7.0, 30.0, 500.0], device="cuda").view(1, 1, 7)
    one = torch.ones(1, 1, 1, 1, device="cuda")
    y, _ = comba.selective_scan(torch.ones_like(dt), dt, torch.full((7, 1), -3.0, device="cuda"), one, one)
    ref = np.logaddexp(0.0, dt.double().cpu().numpy())
    assert np.abs(y.double().cpu().numpy() / ref - 1).max() < 200 * 2.0 ** -24   # 20 + 2 |u| roundings


def test_growing_states_are_allowed():
    on, ref = make(1, 20, 8, 4, 1, F32, None, ("init",), seed=6, softplus=False)
    on["A"], ref["A"] = -on["A"], -ref["A"]
    y, f = comba.selective_scan(*args_of(on), **opts(on), softplus=False)
    o = oracle_args(ref, False, None)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*args_of(ref), **o, magnitude=True)
    x = float((np.abs(ref["dt"] + ref["dt_bias"]).max(-1).sum()) * ref["A"].max())  # exponents along the whole path
    gamma = scan_gamma(20, umax(ref)) * (1 + x)
    check("y", y, ry, my, gamma)
    check("state", f, rf, mf, gamma)


@pytest.mark.parametrize("B,T,D,S,lens", [(2, 45, 20, 16, None), (1, 300, 66, 5, None), (1, 700, 40, 16, [3, 590, 0, 107])])
def test_states_that_forget_at_every_token(B, T, D, S, lens):
    """A = -infinity: the state is d x B alone, up to the last token of a sequence whose length is no
    multiple of a tile, and an empty sequence's state passes through. The oracle has -1e30, whose
    exponential is 0 for every step size that occurs (at least log(1 + e^-9))."""
    on, ref = make(B, T, D, S, 1, F32, lens, seed=21)
    gone = rnd(22).random(size=(D, S)) < 0.4
    ref["A"][gone] = -1e30
    on["A"] = torch.where(torch.from_numpy(gone).cuda(), -torch.inf, on["A"])
    cu = cu_of(lens)
    call = dict(**opts(on), cu_seqlens=cu_dev(cu))
    y, f = comba.selective_scan(*args_of(on), **call)
    o = oracle_args(ref, True, cu)
    ry, rf = layer.selective_scan(*args_of(ref), **o)
    my, mf = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    gamma = scan_gamma(T if lens is None else max(lens), umax(ref))
    check("y", y, ry, my, gamma)
    check("state", f, rf, mf, gamma)
    g = comba.selective_scan_bwd(*args_of(on), on["dy"], **call, d_final_state=on["dfin"])
    o = dict(**o, dy=ref["dy"], dfin=ref["dfin"])
    r = layer.selective_scan(*args_of(ref), **o)
    m = layer.selective_scan(*args_of(half_A(ref)), **o, magnitude=True)
    for k in r:
        adds = D if k in ("dB", "dC") else B * T if k in ("dA", "dskip", "ddt_bias") else 0
        check(k, g[k], r[k], m[k] * (2 if k in ("ddt", "ddt_bias") else 1),
              scan_gamma(T if lens is None else max(lens), umax(ref), adds, ways=2))
