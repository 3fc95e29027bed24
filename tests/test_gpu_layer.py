"""The layer operators in a run, as a recurrent layer uses them: norm, short convolution, recurrence,
gated norm and residual, forward and backward, prompt and single tokens; captured into graphs, on
other streams, two calls at once. Every stage is checked against the fp64 oracle on the values that
really went into it."""
import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
import oracle
from _layer_util import (BF16, F32, check, conv_bwd_gamma, conv_gamma, cu_of, half_A, layer, norm_gamma, rnd,
                         scan_gamma)
from _util import BF16 as CHUNK_GATES, STATE_BF16, assert_close, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


H, K, V = 2, 64, 64
D = H * V


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def t32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def make_layer(seed):
    r = rnd(seed)
    p = dict(pre=1 + 0.1 * r.normal(size=D), post=1 + 0.1 * r.normal(size=V), scale=r.uniform(0.3, 1, size=D),
             a=r.normal(size=D) * 0.1 + 1, d=np.full(H, 0.5))
    for n in "qkv":
        p["w" + n], p["b" + n] = r.normal(size=(D, 4)) * 0.5, r.normal(size=D) * 0.1
    p.update(A=-np.exp(r.normal(size=(D, 16)) * 0.5), skip=np.ones(D), dt_bias=np.full(D, -2.0))
    return {k: t32(v) for k, v in p.items()}


def activations(B, T, seed):
    r = rnd(seed)
    mk = lambda *s: torch.from_numpy(r.normal(size=s).astype(np.float32)).cuda().to(BF16)  # noqa: E731
    f = lambda *s: torch.from_numpy(r.uniform(0.6, 0.99, size=s).astype(np.float32)).cuda()  # noqa: E731
    return dict(x=mk(B, T, D), res=mk(B, T, D), gate=mk(B, T, H, V), alpha=f(B, T, H), beta=f(B, T, H),
                dt=mk(B, T, D), Bm=mk(B, T, 1, 16), Cm=mk(B, T, 1, 16), z=mk(B, T, D))


def comba_layer(p, a, cu=None):
    """norm -> short convolutions -> chunk forward -> gated norm per head -> scale, residual, next norm."""
    B, T, _ = a["x"].shape
    _, n = comba.block_norm(a["x"], pre_weight=p["pre"])
    s = dict(n=n)
    for m in "qkv":
        s[m], s["s" + m] = comba.short_conv(n, p["w" + m], p["b" + m], cu_seqlens=cu)
    heads = lambda t: t.view(B, T, H, -1)  # noqa: E731
    # contiguous inputs of the recurrence, q and k normalised inside it
    s["o"], s["state"] = comba.chunk_fwd(heads(s["q"]), heads(s["k"]), heads(s["v"]), a["alpha"], a["beta"], p["d"],
                                         cu_seqlens=cu, qk_l2norm=True)
    s["y"], _ = comba.block_norm(s["o"], gate=a["gate"], post_weight=p["post"])
    s["r"], s["next"] = comba.block_norm(s["y"].view(B, T, D), residual=a["res"], scale=p["scale"], pre_weight=p["a"])
    return s


@pytest.mark.parametrize("lens", [None, [0, 70, 1, 130, 64]])
def test_layer_around_the_chunk_forward(lens):
    B, T = (2, 150) if lens is None else (1, sum(lens))
    cu = cu_of(lens)
    p, a = make_layer(1), activations(B, T, 2)
    s = comba_layer(p, a, None if cu is None else torch.from_numpy(cu).cuda())
    ref = layer.block_norm(np64(a["x"]), pre_weight=np64(p["pre"]))[1]
    mag = layer.block_norm(np64(a["x"]), pre_weight=np64(p["pre"]), magnitude=True)[1]
    check("n", s["n"], ref, mag, norm_gamma())
    for m in "qkv":
        args = (np64(s["n"]), np64(p["w" + m]), np64(p["b" + m]))
        size = layer.short_conv(*args, cu=cu, magnitude=True)[0]
        check(m, s[m], layer.short_conv(*args, cu=cu)[0], size, conv_gamma(4, size.max()))
    heads = lambda t: np64(t).reshape(B, T, H, -1)  # noqa: E731
    q, k, al, be = oracle.fused_inputs(heads(s["q"]), heads(s["k"]), np64(a["alpha"]), np64(a["beta"]), qk_l2norm=True)
    ro, rs = oracle.comba_forward(q, k, heads(s["v"]), al, be, np64(p["d"]), None, cu)
    assert_close(to_np(s["o"]), ro, CHUNK_GATES, "o")
    assert_close(to_np(s["state"]), rs, STATE_BF16, "state")
    kw = dict(gate=np64(a["gate"]), post_weight=np64(p["post"]))
    check("y", s["y"], layer.block_norm(np64(s["o"]), **kw)[0], layer.block_norm(np64(s["o"]), **kw, magnitude=True)[0],
          norm_gamma())
    kw = dict(residual=np64(a["res"]), scale=np64(p["scale"]), pre_weight=np64(p["a"]))
    y = np64(s["y"]).reshape(B, T, D)
    for k2, got, ref, mag in zip("rn", (s["r"], s["next"]), layer.block_norm(y, **kw),
                                 layer.block_norm(y, **kw, magnitude=True)):
        check(k2, got, ref, mag, norm_gamma())


def test_backward_through_the_layer():
    """The gradients handed from operator to operator: the norm's float gradients into chunk_bwd, whose
    float32 gradients go into the convolution's backward as they are."""
    B, T = 2, 100
    p, a = make_layer(3), activations(B, T, 4)
    n = a["x"]
    q, k, v = (comba.short_conv(n, p["w" + m], p["b" + m])[0].view(B, T, H, -1) for m in "qkv")
    q, k = ((t.float() / t.float().norm(dim=-1, keepdim=True)).to(BF16) for t in (q, k))
    o, _ = comba.chunk_fwd(q, k, v, a["alpha"], a["beta"], p["d"])
    gn = comba.block_norm_bwd(o, a["z"].view(B, T, H, V), gate=a["gate"], post_weight=p["post"])
    kw = dict(gate=np64(a["gate"]), post_weight=np64(p["post"]), dr=np64(a["z"]).reshape(B, T, H, V))
    r, m = layer.block_norm(np64(o), **kw), layer.block_norm(np64(o), **kw, magnitude=True)
    for name in r:
        check(name, gn[name], r[name], m[name], norm_gamma(B * T * H, True))
    gc = comba.chunk_bwd(q, k, v, a["alpha"], a["beta"], p["d"], gn["dy"])
    assert gc["dv"].dtype == F32
    dv = gc["dv"].view(B, T, D)
    g = comba.short_conv_bwd(n, p["wv"], p["bv"], dv)
    args = (np64(n), np64(p["wv"]), np64(p["bv"]))
    r, m = layer.short_conv(*args, dy=np64(dv)), layer.short_conv(*args, dy=np64(dv), magnitude=True)
    pmax = layer.short_conv(*args, magnitude=True)[0].max()
    for name in ("dx", "dweight", "dbias"):
        check(name, g[name], r[name], m[name], conv_bwd_gamma(4, pmax, B * T if name != "dx" else 0))


def scan_layer(p, a, conv_state=None, state=None):
    u, conv_state = comba.short_conv(a["x"], p["wv"], p["bv"], conv_state)
    y, state = comba.selective_scan(u, a["dt"], p["A"], a["Bm"], a["Cm"], p["skip"], a["z"], p["dt_bias"],
                                    initial_state=state)
    r, n = comba.block_norm(y, residual=a["res"], scale=p["scale"], post_weight=p["a"], pre_weight=p["pre"])
    return u, y, r, n, conv_state, state


def test_prompt_then_single_tokens():
    """Decoding goes on where the prompt ended, state for state: the convolution bit for bit, the scan
    within twice its bound of the whole prompt's."""
    B, T, cut = 3, 60, 40
    p, a = make_layer(5), activations(B, T, 6)
    whole = scan_layer(p, a)
    part = lambda lo, hi: {k: v[:, lo:hi].contiguous() for k, v in a.items()}  # noqa: E731
    _, _, _, _, cs, st = scan_layer(p, part(0, cut))
    args = [np64(t) for t in (whole[0], a["dt"], p["A"], a["Bm"], a["Cm"])]
    args[2] = args[2] / 2
    kw = dict(skip=np64(p["skip"]), z=np64(a["z"]), dt_bias=np64(p["dt_bias"]))
    mag, mfin = layer.selective_scan(*args, **kw, magnitude=True)
    gamma = 2 * scan_gamma(T, float(np.abs(np64(a["dt"]) - 2).max()))
    for t in range(cut, T):
        b = {k: v[:, t].contiguous() for k, v in a.items()}
        u, cs = comba.short_conv_step(b["x"], p["wv"], p["bv"], cs, in_place=True)
        y, st = comba.selective_step(u, b["dt"], p["A"], b["Bm"], b["Cm"], p["skip"], b["z"], p["dt_bias"],
                                     initial_state=st, in_place=True)
        assert torch.equal(u, whole[0][:, t])
        # two bf16 roundings of nearby values are at most a step apart
        check(f"y {t}", y, np64(whole[1][:, t]), mag[:, t], 2 * gamma + 2.0 ** -8)
    assert torch.equal(cs, whole[4])
    check("state", st, np64(whole[5]), mfin, gamma)


def all_calls(p, a, ws):
    """Every entry point once, outputs in a list."""
    out = []
    _, n = comba.block_norm(a["x"], pre_weight=p["pre"])
    u, cs = comba.short_conv(n, p["wv"], p["bv"])
    y, st = comba.selective_scan(u, a["dt"], p["A"], a["Bm"], a["Cm"], p["skip"], a["z"], p["dt_bias"], workspace=ws)
    r, n2 = comba.block_norm(y, residual=a["res"], scale=p["scale"], post_weight=p["a"], pre_weight=p["pre"])
    g = comba.block_norm_bwd(y, n, n2, residual=a["res"], scale=p["scale"], post_weight=p["a"], pre_weight=p["pre"])
    gs = comba.selective_scan_bwd(u, a["dt"], p["A"], a["Bm"], a["Cm"], g["dy"], p["skip"], a["z"], p["dt_bias"])
    gc = comba.short_conv_bwd(n, p["wv"], p["bv"], gs["dx"])
    last = {k: v[:, -1].contiguous() for k, v in a.items()}
    us, cs2 = comba.short_conv_step(last["x"], p["wv"], p["bv"], cs)
    ys, st2 = comba.selective_step(us, last["dt"], p["A"], last["Bm"], last["Cm"], p["skip"], last["z"], p["dt_bias"],
                                   initial_state=st)
    for v in (n, u, cs, y, st, r, n2, g, gs, gc, us, cs2, ys, st2):
        out += [t for t in v.values() if t is not None] if isinstance(v, dict) else [v]
    return out


@pytest.mark.parametrize("T", [40, 600])   # the second cuts the scan along time
def test_captured_into_a_graph_and_replayed(T):
    p, a = make_layer(7), activations(1, T, 8)
    ws = torch.empty(max(1, comba.selective_scan_workspace_size(1, T, D, 16)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_calls(p, a, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_calls(p, a, ws)
    for i in range(4):
        fresh = activations(1, T, 20 + i)
        for k in a:
            a[k].copy_(fresh[k])
        want = [t.clone() for t in all_calls(p, fresh, None)]   # eager work between the replays
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want)), i


def test_two_streams_at_once():
    """Calls that overlap in time share nothing: every result is what it is alone."""
    p = make_layer(9)
    sets = [activations(1, 700, 30 + i) for i in range(4)]
    want = [[t.clone() for t in all_calls(p, a, None)] for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = all_calls(p, sets[i], None)
        torch.cuda.synchronize()
        for i in range(len(sets)):
            assert all(torch.equal(g, w) for g, w in zip(got[i], want[i])), i


def test_refusals_of_the_binding():
    p, a = make_layer(11), activations(1, 8, 12)
    x, w = a["x"], p["wv"]
    with pytest.raises(ValueError, match="contiguous"):
        comba.short_conv(x[..., ::2], w[::2])
    with pytest.raises(ValueError, match="weight must be torch.float32"):
        comba.short_conv(x, w.to(BF16))
    with pytest.raises(ValueError, match="initial_state must have shape"):
        comba.short_conv(x, w, initial_state=x[:, :4].contiguous())
    with pytest.raises(ValueError, match="initial_state must be torch.bfloat16"):
        comba.short_conv(x, w, initial_state=x[:, :3].float().contiguous())
    with pytest.raises(comba.CombaError, match="taps"):
        comba.short_conv(x, t32(np.zeros((D, 5))))
    s = x[:, :3].contiguous()
    with pytest.raises(comba.CombaError, match="overlaps"):
        comba.short_conv(x, w, initial_state=s, final_state=s)
    with pytest.raises(ValueError, match="in_place"):
        comba.short_conv_step(x[:, 0].contiguous(), w, in_place=True)
    with pytest.raises(ValueError, match="must divide"):
        comba.selective_scan(x, a["dt"], p["A"], a["Bm"].expand(1, 8, 3, 16).contiguous(), a["Cm"])
    with pytest.raises(ValueError, match="Cm must have shape"):
        comba.selective_scan(x, a["dt"], p["A"], a["Bm"], a["Cm"][..., :8].contiguous())
    with pytest.raises(ValueError, match="dt must be torch.bfloat16"):
        comba.selective_scan(x, a["dt"].float(), p["A"], a["Bm"], a["Cm"])
    with pytest.raises(comba.CombaError, match="64 states"):
        comba.selective_scan(x, a["dt"], t32(-np.ones((D, 65))), *[t32(np.zeros((1, 8, 1, 65))).to(BF16)] * 2)
    with pytest.raises(ValueError, match="float16|bfloat16 or float32"):
        comba.block_norm(x.half(), post_weight=p["a"])
    with pytest.raises(comba.CombaError, match="at least one"):
        comba.block_norm(x)
    with pytest.raises(comba.CombaError, match="dr or dn"):
        comba.block_norm_bwd(x, post_weight=p["a"])
    with pytest.raises(ValueError, match="gate must have shape"):
        comba.block_norm(x, gate=x[:, :4].contiguous())
    with pytest.raises(ValueError, match="out_norm goes with"):
        comba.block_norm(x, post_weight=p["a"], out_norm=x)


def test_calls_that_would_overwrite_their_inputs_are_refused():
    p, a = make_layer(12), activations(1, 8, 13)
    x, w = a["x"], p["wv"]
    with pytest.raises(comba.CombaError, match="an output overlaps an input"):
        comba.short_conv(x, w, out=x)
    with pytest.raises(comba.CombaError, match="an output overlaps an input"):
        comba.selective_scan(x, a["dt"], p["A"], a["Bm"], a["Cm"], out=a["dt"])
    with pytest.raises(comba.CombaError, match="an output overlaps an input"):
        comba.block_norm(x, post_weight=p["a"], out=x)
    s = torch.zeros((1, 3, D), dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="final_state must not be given"):
        comba.short_conv_step(x[:, 0].contiguous(), w, initial_state=s, in_place=True, final_state=torch.empty_like(s))
    for cu in ([], [0]):
        with pytest.raises(ValueError, match="N >= 1 sequences"):
            comba.short_conv(x, w, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))


def test_debug_checks_cover_packed_offsets(monkeypatch):
    from bilinear_rnn_amd import api
    p, a = make_layer(13), activations(1, 20, 14)
    bad = torch.tensor([0, 12, 8, 20], dtype=torch.int32, device="cuda")
    monkeypatch.setattr(api, "DEBUG_CHECKS", True)
    with pytest.raises(comba.CombaError, match="cu_seqlens decreases"):
        comba.short_conv(a["x"], p["wv"], cu_seqlens=bad)
    with pytest.raises(comba.CombaError, match="cu_seqlens decreases"):
        comba.selective_scan(a["x"], a["dt"], p["A"], a["Bm"], a["Cm"], cu_seqlens=bad)
    good = torch.tensor([0, 8, 12, 20], dtype=torch.int32, device="cuda")
    comba.short_conv(a["x"], p["wv"], cu_seqlens=good)
