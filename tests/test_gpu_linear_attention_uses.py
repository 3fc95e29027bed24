"""Linear attention and group norm as they are used: together, decoding after a prompt, in graphs, on several
streams, on batches with many workgroups, extreme decays, unaligned tensors and rows that belong to no sequence."""
import ctypes

import numpy as np
import pytest
import torch

import bilinear_rnn_amd as comba
from bilinear_rnn_amd import api
from _layer_util import BF16, F32, U, check, cu_dev, cu_of, dev, layer, rnd
from test_gpu_group_norm import gamma as norm_gamma
from test_gpu_linear_attention import gamma, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def np64(t):
    return t.double().cpu().numpy()


def forward(on, scale, cu=None, **kw):
    return comba.linear_attention(on["q"], on["k"], on["v"], on["log_decay"], on["init"], cu_dev(cu), scale=scale, **kw)


def backward(on, scale, cu=None, dfin=True, **kw):
    return comba.linear_attention_bwd(on["q"], on["k"], on["v"], on["log_decay"], on["do"], on["init"], cu_dev(cu),
                                      on["dfin"] if dfin else None, scale=scale, **kw)


def check_forward(o, f, ref, scale, dtype, cu=None):
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    kw = dict(scale=scale, init=ref["init"], cu=cu)
    ro, rf = layer.linear_attention(*args, **kw)
    mo, mf = layer.linear_attention(*args, **kw, magnitude=True)
    K, V, T = ref["q"].shape[-1], ref["v"].shape[-1], ref["v"].shape[1]
    check("o", o, ro, mo, gamma(K, V, T, dtype))
    check("state", f, rf, mf, gamma(K, V, T, dtype, exact=True))


def check_backward(got, ref, scale, dtype, cu=None, dfin=True):
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    kw = dict(scale=scale, init=ref["init"], cu=cu, do=ref["do"], dfin=ref["dfin"] if dfin else None)
    r, m = layer.linear_attention(*args, **kw), layer.linear_attention(*args, **kw, magnitude=True)
    K, V, T, H, Hk = ref["q"].shape[-1], ref["v"].shape[-1], ref["v"].shape[1], ref["v"].shape[2], ref["q"].shape[2]
    for n in ("dq", "dk", "dv"):
        check(n, got[n], r[n], m[n], gamma(K, V, T, dtype) + H // Hk * U)
    check("dinitial_state", got["dinitial_state"], r["dinitial_state"], m["dinitial_state"],
          gamma(K, V, T, dtype, exact=True))
    check("dlog_decay", got["dlog_decay"], r["dlog_decay"], m["dlog_decay"], gamma(K, V, T, dtype, exact=True, ways=3))


# Enough (sequence, head) pairs for workgroups of 128 columns.
@pytest.mark.parametrize("B,T,H,Hk,K,V,dtype,lens,head", [
    (8, 70, 32, 32, 16, 128, BF16, None, False), (8, 66, 32, 16, 72, 99, BF16, None, True),
    (8, 40, 32, 8, 128, 72, F32, None, False), (8, 34, 32, 32, 33, 130, F32, None, False),
    (1, 600, 64, 64, 24, 80, BF16, [300, 0, 1, 299], False)])
def test_forward_of_many_heads(B, T, H, Hk, K, V, dtype, lens, head):
    on, ref = make(B, T, H, Hk, K, V, dtype, lens, head, seed=3)
    cu = cu_of(lens)
    o, f = forward(on, K ** -0.5, cu)
    check_forward(o, f, ref, K ** -0.5, dtype, cu)


@pytest.mark.parametrize("B,T,H,Hk,K,V,dtype,lens,head", [
    (4, 66, 32, 32, 128, 128, BF16, None, False), (8, 66, 32, 16, 72, 99, BF16, None, True),
    (8, 40, 32, 8, 100, 72, F32, None, False), (8, 34, 32, 32, 66, 65, F32, None, False),
    (1, 600, 64, 32, 72, 80, BF16, [300, 0, 1, 299], False)])
def test_backward_of_many_heads(B, T, H, Hk, K, V, dtype, lens, head):
    on, ref = make(B, T, H, Hk, K, V, dtype, lens, head, seed=4)
    cu = cu_of(lens)
    check_backward(backward(on, K ** -0.5, cu), ref, K ** -0.5, dtype, cu)


# Two workgroups per compute unit (many short sequences, heads up to 64), several chunks each.
@pytest.mark.parametrize("B,T,H,Hk,K,V,dtype", [(16, 300, 32, 32, 16, 24, BF16), (16, 140, 32, 16, 12, 20, F32),
                                                (9, 200, 64, 64, 17, 10, BF16)])
def test_pairs_of_workgroups(B, T, H, Hk, K, V, dtype):
    on, ref = make(B, T, H, Hk, K, V, dtype, seed=14)
    o, f = forward(on, K ** -0.5)
    check_forward(o, f, ref, K ** -0.5, dtype)
    check_backward(backward(on, K ** -0.5), ref, K ** -0.5, dtype)


# Packed batches with a few long sequences among many short ones: more than a step of the search takes.
@pytest.mark.parametrize("N,dtype", [(64, BF16), (65, F32), (100, BF16), (600, BF16), (1100, F32)])
def test_few_long_sequences_among_many(N, dtype):
    lens = rnd(15).integers(0, 12, size=N).tolist()
    for n, x in ((3, 700), (N // 2, 1), (N - 30, 513), (N - 1, 1100)):
        lens[n] = x
    cu = cu_of(lens)
    on, ref = make(1, sum(lens), 4, 2, 16, 24, dtype, lens, seed=16)
    o, f = forward(on, 0.25, cu)
    check_forward(o, f, ref, 0.25, dtype, cu)
    check_backward(backward(on, 0.25, cu), ref, 0.25, dtype, cu)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growing_states(dtype):
    """Decays above 1: the state grows to about e^20 times a term. Relative to the whole tensor, an output is off by its
    rounding, the rest by T + K + V roundings of 2^-24 and, for decays, four for each of the T exponents."""
    T, K, V = 300, 24, 40
    on, ref = make(2, T, 2, 2, K, V, dtype, seed=17)
    on["log_decay"], ref["log_decay"] = dev(rnd(18).uniform(-0.05, 0.2, size=(2, T, 2)))
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    o, f = forward(on, 0.2)
    ro, rf = layer.linear_attention(*args, scale=0.2, init=ref["init"])
    off = lambda a, b: np.linalg.norm(np64(a) - b) / np.linalg.norm(b)  # noqa: E731
    u = U * (5 * T + K + V)
    step = torch.finfo(dtype).eps / 2
    assert off(o, ro) < step + u + 2.0 ** -16 and off(f, rf) < u
    got = backward(on, 0.2)
    r = layer.linear_attention(*args, scale=0.2, init=ref["init"], do=ref["do"], dfin=ref["dfin"])
    for n in ("dq", "dk", "dv"):
        assert off(got[n], r[n]) < step + u + 2.0 ** -16, n
    assert off(got["dinitial_state"], r["dinitial_state"]) < u


def extreme(on, ref, seed):
    """Decays from none at all to resets of the state."""
    some = np.array([0.0, -1e-7, -1e-3, -0.3, -5.0, -60.0, -150.0, -300.0, -1e30, -np.inf])
    on["log_decay"], ref["log_decay"] = dev(rnd(seed).choice(some, size=ref["log_decay"].shape))


@pytest.mark.parametrize("T,K,V,dtype,head", [(150, 40, 24, F32, False), (700, 64, 64, BF16, False),
                                              (130, 64, 128, BF16, True), (1, 16, 16, F32, False)])
def test_extreme_decays(T, K, V, dtype, head):
    on, ref = make(1, T, 10 if head else 2, 2, K, V, dtype, head=head, seed=5)
    extreme(on, ref, 6)
    o, f = forward(on, 1.0)
    check_forward(o, f, ref, 1.0, dtype)
    got = backward(on, 1.0)
    check_backward(got, ref, 1.0, dtype)
    assert (got["dlog_decay"][on["log_decay"] < -104] == 0).all()
    step = comba.linear_attention_step(on["q"][:, 0], on["k"][:, 0], on["v"][:, 0],
                                       on["log_decay"] if head else on["log_decay"][:, 0], on["init"])
    first = {n: t if n == "init" or (head and n == "log_decay") else t[:, :1] for n, t in ref.items() if n not in ("do", "dfin")}
    args = [first[n] for n in ("q", "k", "v", "log_decay")]
    r, m = layer.linear_attention(*args, init=first["init"]), layer.linear_attention(*args, init=first["init"], magnitude=True)
    check("step's o", step[0], r[0][:, 0], m[0][:, 0], U * (K / 16 + 16))
    check("step's state", step[1], r[1], m[1], U * 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_without_a_final_gradient(dtype):
    on, ref = make(2, 90, 4, 2, 40, 24, dtype, seed=7)
    check_backward(backward(on, 1.0, dfin=False), ref, 1.0, dtype, dfin=False)
    on["init"] = ref["init"] = None
    got = backward(on, 1.0, dfin=False)
    check_backward(got, ref, 1.0, dtype, dfin=False)
    assert (got["dlog_decay"][:, 0] == 0).all()   # decays nothing


def off_by_one(t):
    """The same values one element behind a 16-byte boundary."""
    if t is None:
        return None
    big = t.new_empty(t.numel() + 1)
    big[1:] = t.reshape(-1)
    return big[1:].view(t.shape)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unaligned_tensors(dtype):
    on, ref = make(2, 100, 2, 1, 64, 128, dtype, seed=8)
    on = {n: off_by_one(t) for n, t in on.items()}
    out, fin = off_by_one(on["v"]), off_by_one(on["init"])
    forward(on, 0.5, out=out, final_state=fin)
    check_forward(out, fin, ref, 0.5, dtype)
    check_backward(backward(on, 0.5), ref, 0.5, dtype)
    for T in (1, 100):
        x, dy = (off_by_one(on[n][:, :T, :].reshape(2, T, 256).contiguous()) for n in ("v", "do"))
        w = off_by_one(torch.linspace(0.5, 1.5, 256, device="cuda"))
        if T == 1:
            x, dy = x.view(2, 256), dy.view(2, 256)
        y, st = comba.group_norm(x, 4, w, w, silu=True, out=off_by_one(x))
        g = comba.group_norm_bwd(x, dy, st, 4, w, w, silu=True)
        a = [np64(x).reshape(2, T, 256), 4, np64(w), np64(w)]
        r, m = (layer.group_norm(*a, silu=True, magnitude=b) for b in (False, True))
        check("y", y.view(2, T, 256), r[0], m[0], norm_gamma(64 * T))
        r, m = (layer.group_norm(*a, silu=True, dy=np64(dy).reshape(2, T, 256), magnitude=b) for b in (False, True))
        check("dx", g["dx"].view(2, T, 256), r["dx"], m["dx"], norm_gamma(64 * T, True))
        check("dweight", g["dweight"], r["dweight"], m["dweight"], norm_gamma(64 * T, True, 2 * T))


@pytest.mark.parametrize("T,lens", [(100, None), (900, None), (900, [30, 0, 870])])
def test_state_in_place(T, lens):
    """final_state may be initial_state: whole and cut sequences, empty ones too."""
    cu = cu_of(lens)
    on, _ = make(1, T, 2, 2, 64, 128, BF16, lens, seed=9)
    o, f = forward(on, 1.0, cu)
    assert f is not on["init"]
    again, g = forward(on, 1.0, cu, final_state=on["init"])
    assert g is on["init"] and torch.equal(again, o) and torch.equal(g, f)


def raw(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("Hk,dtype", [(4, BF16), (2, BF16), (2, F32)])
def test_rows_of_no_sequence_are_left_as_they_were(Hk, dtype):
    """Offsets that begin behind the first token and end before the last."""
    T, H, K, V, cu = 500, 4, 24, 40, np.array([5, 40, 40, 425], np.int32)
    on, ref = make(1, T, H, Hk, K, V, dtype, [1, 1, 1], seed=10)
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    inside[5:425] = True
    mark = lambda *s, t=dtype: torch.full(s, 777.0, dtype=t, device="cuda")  # noqa: E731
    o = mark(1, T, H, V)
    _, f = forward(on, 1.0, cu, out=o)
    check_forward(o, f, ref, 1.0, dtype, cu)
    assert (o[:, ~inside] == 777).all()
    got = dict(dq=mark(1, T, Hk, K), dk=mark(1, T, Hk, K), dv=mark(1, T, H, V), dlog_decay=mark(1, T, H, t=F32),
               dinitial_state=mark(3, H, V, K, t=F32))
    L, c = comba.lib(), cu_dev(cu)
    ws = torch.full((int(L.comba_linear_attn_bwd_workspace_size(1, T, H, Hk, K, V, 3)),), 255, dtype=torch.uint8,
                    device="cuda")
    fp = ctypes.POINTER(ctypes.c_float)
    f32 = lambda t: ctypes.cast(raw(t), fp)  # noqa: E731
    rc = L.comba_linear_attn_bwd(
        raw(on["q"]), raw(on["k"]), raw(on["v"]), f32(on["log_decay"]), 1, f32(on["init"]),
        ctypes.cast(raw(c), ctypes.POINTER(ctypes.c_int32)), 3, 1, T, H, Hk, K, V, 0 if dtype == BF16 else 1, 1.0,
        raw(on["do"]), f32(on["dfin"]), raw(got["dq"]), raw(got["dk"]), raw(got["dv"]), f32(got["dlog_decay"]),
        f32(got["dinitial_state"]), raw(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, api.last_error()
    check_backward(got, ref, 1.0, dtype, cu)
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert (got[n][:, ~inside] == 777).all(), n
    # group norm: the same offsets
    x, y = on["v"].view(1, T, H * V), mark(1, T, H * V)
    _, st = comba.group_norm(x, H, cu_seqlens=c, silu=True, out=y)
    r, m = (layer.group_norm(ref["v"].reshape(1, T, H * V), H, silu=True, cu=cu, magnitude=b) for b in (False, True))
    check("y", y, r[0], m[0], norm_gamma(V * T))
    assert (y[:, ~inside] == 777).all() and (st[1] == 0).all()
    w = torch.ones(H * V, device="cuda")
    g = comba.group_norm_bwd(x, on["do"].view(1, T, H * V), st, H, w, w * 0, cu_seqlens=c, silu=True)
    a = dict(weight=np.ones(H * V), bias=np.zeros(H * V), silu=True, cu=cu, dy=ref["do"].reshape(1, T, H * V))
    r, m = (layer.group_norm(ref["v"].reshape(1, T, H * V), H, **a, magnitude=b) for b in (False, True))
    for n in ("dx", "dweight", "dbias"):
        check(n, g[n], r[n], m[n], norm_gamma(V * T, True, T))


def test_results_do_not_depend_on_the_workspace_or_the_run():
    for lens in (None, [300, 0, 600]):
        on, _ = make(1, 900, 4, 2, 40, 72, BF16, lens, seed=11)
        cu, N = cu_of(lens), 0 if lens is None else 3
        size = comba.linear_attention_workspace_size(1, 900, 4, 2, 40, 72, N)
        bsize = int(comba.lib().comba_linear_attn_bwd_workspace_size(1, 900, 4, 2, 40, 72, N))
        x, w = on["v"].view(1, 900, 288), torch.ones(288, device="cuda")
        nsize = max(int(fn(1, 900, 288, 4, N)) for fn in (comba.lib().comba_group_norm_workspace_size,
                                                         comba.lib().comba_group_norm_bwd_workspace_size))
        want = None
        for fill in (0, 255, 127, 0):
            ws = [torch.full((n,), fill, dtype=torch.uint8, device="cuda") for n in (size, bsize, nsize)]
            y, st = comba.group_norm(x, 4, w, w, cu_dev(cu), silu=True, workspace=ws[2])
            got = [*forward(on, 1.0, cu, workspace=ws[0]), *backward(on, 1.0, cu, workspace=ws[1]).values(), y, st]
            ws[2].fill_(fill)
            got += comba.group_norm_bwd(x, y, st, 4, w, w, cu_dev(cu), silu=True, workspace=ws[2]).values()
            assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
            want = got


def test_what_is_not_finite_stays_in_its_sequence_and_head():
    lens, cu = [70, 0, 500, 60], cu_of([70, 0, 500, 60])
    clean, _ = make(1, 630, 3, 3, 64, 64, BF16, lens, seed=12)
    on = {n: t.clone() for n, t in clean.items()}
    bad = [("q", 100, 0, np.nan), ("k", 300, 0, np.inf), ("v", 90, 0, -np.inf), ("do", 80, 0, np.nan)]
    for n, t, h, x in bad:
        on[n][0, t, h, 3] = x
    on["init"][2, 0, 1, 1] = np.nan
    w, wf = forward(clean, 1.0, cu)
    o, f = forward(on, 1.0, cu)
    keep = torch.ones(630, 3, dtype=torch.bool, device="cuda")
    keep[70:570, 0] = False
    assert torch.equal(o[0][keep], w[0][keep]) and torch.equal(f[[0, 1, 3]], wf[[0, 1, 3]]) and torch.equal(f[2, 1:], wf[2, 1:])
    assert not torch.isfinite(o[0, 100, 0]).all() and not torch.isfinite(f[2, 0]).all()
    wg, g = backward(clean, 1.0, cu), backward(on, 1.0, cu)
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert torch.equal(g[n][0][keep], wg[n][0][keep]), n
    assert torch.equal(g["dinitial_state"][[0, 1, 3]], wg["dinitial_state"][[0, 1, 3]])
    assert not torch.isfinite(g["dq"][0, 80, 0]).all()
    # group norm: of its sequence and group
    x, c = on["v"].reshape(1, 630, 192), cu_dev(cu)
    y, st = comba.group_norm(x, 3, cu_seqlens=c)
    z, sz = comba.group_norm(clean["v"].reshape(1, 630, 192), 3, cu_seqlens=c)
    assert torch.equal(y.view(630, 3, 64)[keep], z.view(630, 3, 64)[keep])
    assert torch.isnan(y.view(630, 3, 64)[70:570, 0]).all() and torch.isnan(st[2, 0]).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_thousands_of_short_sequences(dtype):
    lens = rnd(13).integers(0, 4, size=3000).tolist()
    T, cu = sum(lens), cu_of(lens)
    on, ref = make(1, T, 2, 1, 12, 9, dtype, lens, seed=13)
    o, f = forward(on, 1.0, cu)
    check_forward(o, f, ref, 1.0, dtype, cu)
    check_backward(backward(on, 1.0, cu), ref, 1.0, dtype, cu)


# --- together ------------------------------------------------------------------------------------

D, H, HK, K, V = 128, 4, 2, 24, 32


def activations(B, T, seed, dtype=BF16):
    on, _ = make(B, T, H, HK, K, V, dtype, seed=seed)
    on["w"], on["b"] = (torch.from_numpy(rnd(50).normal(size=D).astype(np.float32) + i).cuda() for i in (1, 0))
    return on


def mixer(a, **kw):
    """The operator and the norm of its heads, as a layer has them."""
    o, f = comba.linear_attention(a["q"], a["k"], a["v"], a["log_decay"], a["init"], scale=K ** -0.5, **kw)
    rows = o.shape[0] * o.shape[1]
    y, st = comba.group_norm(o.view(rows, D), H, a["w"], a["b"], silu=True)
    return o, f, y, st


def test_backward_through_the_layer():
    B, T = 2, 100
    a = activations(B, T, 20)
    o, f, y, st = mixer(a)
    dy = a["do"].view(B * T, D)
    gn = comba.group_norm_bwd(o.view(B * T, D), dy, st, H, a["w"], a["b"], silu=True)
    args = dict(weight=np64(a["w"]), bias=np64(a["b"]), silu=True, dy=np64(dy)[:, None])
    r, m = (layer.group_norm(np64(o).reshape(B * T, 1, D), H, **args, magnitude=x) for x in (False, True))
    check("dx", gn["dx"][:, None], r["dx"], m["dx"], norm_gamma(V, True))
    for n in ("dweight", "dbias"):
        check(n, gn[n], r[n], m[n], norm_gamma(V, True, B * T))
    a["do"] = gn["dx"].view(B, T, H, V)
    ref = {n: np64(t) for n, t in a.items()}
    check_backward(backward(a, K ** -0.5), ref, K ** -0.5, BF16)


def test_prompt_then_single_tokens():
    """Decoding goes on where the prompt ended."""
    B, T, cut = 3, 60, 40
    a = activations(B, T, 21)
    part = lambda lo, hi: {n: t if n in ("init", "dfin", "w", "b") else t[:, lo:hi].contiguous() for n, t in a.items()}  # noqa: E731
    whole, fin, y, _ = mixer(a)
    _, st, _, _ = mixer(part(0, cut))
    ref = {n: np64(t) for n, t in a.items()}
    args = [ref[n] for n in ("q", "k", "v", "log_decay")]
    r, m = (layer.linear_attention(*args, scale=K ** -0.5, init=ref["init"], magnitude=x) for x in (False, True))
    for t in range(cut, T):
        s = {n: x[:, 0] for n, x in part(t, t + 1).items() if n in ("q", "k", "v", "log_decay")}
        o, st = comba.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], st, scale=K ** -0.5, in_place=True)
        check(f"o {t}", o, r[0][:, t], m[0][:, t], gamma(K, V, T, BF16) + U * 16 * T)
        n, _ = comba.group_norm(o.view(B, D), H, a["w"], a["b"], silu=True, output_stats=False)
        rn, mn = (layer.group_norm(np64(o).reshape(B, 1, D), H, np64(a["w"]), np64(a["b"]), silu=True, magnitude=x)[0]
                  for x in (False, True))
        check(f"norm {t}", n[:, None], rn, mn, norm_gamma(V))
    check("state", st, r[1], m[1], gamma(K, V, T, BF16, exact=True) + U * 16 * T)


def all_calls(a, ws, bws, c):
    """Every entry point once, outputs in a list."""
    B, T = a["q"].shape[:2]
    o, f, y, st = mixer(a, workspace=ws)
    g = comba.group_norm_bwd(o.view(B * T, D), y, st, H, a["w"], a["b"], silu=True)
    gl = comba.linear_attention_bwd(a["q"], a["k"], a["v"], a["log_decay"], g["dx"].view(o.shape), a["init"], None, a["dfin"],
                                    workspace=bws)
    head = a["log_decay"][0, 0].clone()
    gh = comba.linear_attention_bwd(a["q"], a["k"], a["v"], head, o)
    s, sst = comba.group_norm(o.view(B, T, D), 8, a["w"], a["b"], silu=True)
    gs = comba.group_norm_bwd(o.view(B, T, D), s, sst, 8, a["w"], a["b"], silu=True)
    p, pst = comba.group_norm(o.view(1, B * T, D), 8, cu_seqlens=c, out=torch.zeros_like(y).view(1, B * T, D))
    last = [a[n][:, -1].contiguous() for n in ("q", "k", "v", "log_decay")]
    os, fs = comba.linear_attention_step(*last, f)
    out = []
    for v in (o, f, y, st, g, gl, gh, s, sst, gs, p, pst, os, fs):
        out += [t for t in v.values() if t is not None] if isinstance(v, dict) else [v]
    return out


@pytest.mark.parametrize("T", [40, 600])   # the second cuts the sequences along time
def test_captured_into_a_graph_and_replayed(T):
    a, c = activations(1, T, 22), cu_dev(np.array([0, 7, 7, T - 1]))
    size = comba.linear_attention_workspace_size(1, T, H, HK, K, V)
    ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    bws = torch.empty(int(comba.lib().comba_linear_attn_bwd_workspace_size(1, T, H, HK, K, V, 0)), dtype=torch.uint8,
                      device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_calls(a, ws, bws, c)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_calls(a, ws, bws, c)
    for i in range(4):
        fresh = activations(1, T, 30 + i)
        for k in a:
            a[k].copy_(fresh[k])
        want = [t.clone() for t in all_calls(fresh, None, None, c)]   # eager work between the replays
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(got, want)), i


def test_two_streams_at_once():
    """Calls that overlap in time share nothing: every result is what it is alone."""
    T = 700
    c = cu_dev(np.array([0, 7, 7, T]))
    sets = [activations(1, T, 40 + i) for i in range(4)]
    want = [[t.clone() for t in all_calls(a, None, None, c)] for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * len(sets)
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = all_calls(sets[i], None, None, c)
        torch.cuda.synchronize()
        for i in range(len(sets)):
            assert all(torch.equal(g, w) for g, w in zip(got[i], want[i])), i


def test_refusals_of_the_binding():
    a = activations(2, 8, 23)
    q, k, v, g, s = (a[n] for n in ("q", "k", "v", "log_decay", "init"))
    la = comba.linear_attention
    with pytest.raises(ValueError, match="contiguous"):
        la(q[..., ::2], k[..., ::2], v, g)
    with pytest.raises(ValueError, match="k must have shape"):
        la(q, k[..., :8].contiguous(), v, g)
    with pytest.raises(ValueError, match="v must be torch.bfloat16"):
        la(q, k, v.float(), g)
    with pytest.raises(ValueError, match="must divide"):
        la(q, k, v[:, :, :3].contiguous(), g)
    with pytest.raises(ValueError, match="log_decay must be torch.float32"):
        la(q, k, v, g.to(BF16))
    with pytest.raises(ValueError, match="log_decay must have shape"):
        la(q, k, v, g[0, 0, :2].contiguous())
    with pytest.raises(ValueError, match="initial_state must have shape"):
        la(q, k, v, g, s.transpose(2, 3).contiguous())
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        la(q.half(), k.half(), v.half(), g)
    with pytest.raises(comba.CombaError, match="an output overlaps an input"):
        la(q, k, v, g, out=v)
    with pytest.raises(comba.CombaError, match="scale"):
        la(q, k, v, g, scale=float("nan"))
    with pytest.raises(comba.CombaError, match="K or V"):
        la(q[..., :4].contiguous(), k[..., :4].contiguous(), v, g)
    with pytest.raises(ValueError, match="N >= 1 sequences"):
        la(q[:1], k[:1], v[:1], g[:1], cu_seqlens=torch.tensor([0], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="in_place"):
        comba.linear_attention_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), g[:, 0].contiguous(),
                                    in_place=True)
    with pytest.raises(ValueError, match="do must have shape"):
        comba.linear_attention_bwd(q, k, v, g, q)
    with pytest.raises(ValueError, match="d_final_state must have shape"):
        comba.linear_attention_bwd(q, k, v, g, v, d_final_state=s[:1])
    x = v.reshape(2, 8, D)
    with pytest.raises(ValueError, match="must divide"):
        comba.group_norm(x, 3)
    with pytest.raises(ValueError, match="weight must have shape"):
        comba.group_norm(x, 4, a["w"][:4])
    with pytest.raises(ValueError, match="bias must be torch.float32"):
        comba.group_norm(x, 4, a["w"], a["b"].to(BF16))
    with pytest.raises(comba.CombaError, match="eps"):
        comba.group_norm(x, 4, eps=-1.0)
    with pytest.raises(comba.CombaError, match="an output overlaps an input"):
        comba.group_norm(x, 4, out=x)
    with pytest.raises(ValueError, match="stats must have shape"):
        comba.group_norm_bwd(x, x, torch.zeros(2, 2, 2, device="cuda"), 4)


def test_debug_checks_cover_packed_offsets(monkeypatch):
    a = activations(1, 20, 24)
    bad = torch.tensor([0, 12, 8, 20], dtype=torch.int32, device="cuda")
    monkeypatch.setattr(api, "DEBUG_CHECKS", True)
    for call in (lambda: comba.linear_attention(a["q"], a["k"], a["v"], a["log_decay"], cu_seqlens=bad),
                 lambda: comba.linear_attention_bwd(a["q"], a["k"], a["v"], a["log_decay"], a["v"], cu_seqlens=bad),
                 lambda: comba.group_norm(a["v"].reshape(1, 20, D), 4, cu_seqlens=bad)):
        with pytest.raises(comba.CombaError, match="cu_seqlens decreases"):
            call()


# --- sequences of few channels, and large tensors --------------------------------------------------

@pytest.mark.parametrize("B,T,C,G,dtype", [(2, 9, 5, 5, F32), (1, 300, 3, 1, BF16), (1, 1030, 7, 7, BF16), (3, 40, 1, 1, F32),
                                           (2, 70, 9, 3, BF16), (1, 5, 15, 1, F32), (1, 700, 513, 27, BF16)])
def test_norm_of_few_and_odd_channels(B, T, C, G, dtype):
    r = rnd(60)
    x, rx = dev(r.normal(size=(B, T, C)) + 0.5, dtype)
    dy, rdy = dev(r.normal(size=(B, T, C)), dtype)
    w, rw = dev(r.normal(size=C))
    a = dict(weight=rw, bias=rw, silu=True)
    y, st = comba.group_norm(x, G, w, w, silu=True)
    ry, my = (layer.group_norm(rx, G, **a, magnitude=b)[0] for b in (False, True))
    check("y", y, ry, my, norm_gamma(C // G * T))
    g = comba.group_norm_bwd(x, dy, st, G, w, w, silu=True)
    rg, mg = (layer.group_norm(rx, G, **a, dy=rdy, magnitude=b) for b in (False, True))
    for n in ("dx", "dweight", "dbias"):
        check(n, g[n], rg[n], mg[n], norm_gamma(C // G * T, True, B * T))


def big(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(generator=g)


def close(a, b, tol):
    return ((a.float() - b.float()).norm() / b.float().norm()).item() < tol


def test_past_2_31_elements():
    """A batch whose last sequence lies past 2^31 elements, against that sequence alone (cut along time, so the
    same formulas carried in another order)."""
    B, T, heads, width = 9, 65536, 32, 128
    q, k, v = (big(B, T, heads, width, seed=i) for i in range(3))
    assert q.numel() > 1 << 31
    g = -torch.rand((B, T, heads), device="cuda")
    o, f = comba.linear_attention(q, k, v, g, scale=width ** -0.5)
    last = [t[-1:].contiguous() for t in (q, k, v, g)]
    to, tf = comba.linear_attention(*last, scale=width ** -0.5)
    assert close(f[-1:], tf, 1e-5) and close(o[-1:], to, 2.0 ** -8)
    del o, f, to, tf
    d = comba.linear_attention_bwd(q, k, v, g, v, scale=width ** -0.5)
    t = comba.linear_attention_bwd(*last, last[2], scale=width ** -0.5)
    for n in ("dq", "dk", "dv"):
        assert close(d[n][-1:], t[n], 2.0 ** -8), n
    assert close(d["dlog_decay"][-1:], t["dlog_decay"], 1e-5)
    del d, t, k, v
    torch.cuda.empty_cache()
    # group norm: sequences, and every token alone
    x, w = q.view(B, T, heads * width), torch.ones(heads * width, device="cuda")
    dy = big(B, T, heads * width, seed=5)
    y, st = comba.group_norm(x, heads, w, w, silu=True)
    ty, ts = comba.group_norm(x[-1:].contiguous(), heads, w, w, silu=True)
    assert close(y[-1:], ty, 2.0 ** -8) and close(st[-1:], ts, 1e-6)
    dx = comba.group_norm_bwd(x, dy, st, heads, w, w, silu=True)["dx"]
    assert close(dx[-1:], comba.group_norm_bwd(x[-1:].contiguous(), dy[-1:].contiguous(), ts, heads, w, w, silu=True)["dx"],
                 2.0 ** -8)
    del y, dx
    x, dy = x.view(B * T, heads * width), dy.view(B * T, heads * width)
    y, st = comba.group_norm(x, heads, w, w, silu=True)
    ty, ts = comba.group_norm(x[-33:].contiguous(), heads, w, w, silu=True)
    assert torch.equal(y[-33:], ty) and torch.equal(st[-33:], ts)
    dx = comba.group_norm_bwd(x, dy, st, heads, w, w, silu=True)["dx"]
    assert torch.equal(dx[-33:], comba.group_norm_bwd(x[-33:].contiguous(), dy[-33:].contiguous(), ts, heads, w, w,
                                                      silu=True)["dx"])
    del x, y, dx, dy, q
    torch.cuda.empty_cache()


def test_norm_of_a_sequence_of_millions():
    T, C = 4_300_007, 8
    x = big(1, T, C) + 3
    w = torch.linspace(0.5, 1.5, C, device="cuda")
    y, st = comba.group_norm(x, 2, w, None)
    d = x.double().view(T, 2, 4)
    mean = d.mean((0, 2))
    rstd = 1 / (d.sub(mean.view(1, 2, 1)).square().mean((0, 2)) + 1e-5).sqrt()
    assert (st[0, :, 0] / mean - 1).abs().max() < 1e-5 and (st[0, :, 1] / rstd - 1).abs().max() < 1e-5
    want = (d - mean.view(1, 2, 1)) * rstd.view(1, 2, 1) * w.view(1, 2, 4)
    # half a step of bf16, and 1e-5 of the deviations, of which no value is more than 7 away
    assert ((y.double().view(T, 2, 4) - want).abs() <= want.abs() * 2.0 ** -8 + 1.5e-4).all()


def test_steps_past_2_31_state_elements():
    N, heads, width = 4200, 32, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    s = torch.empty((N, heads, width, width), device="cuda").normal_(generator=g)
    assert s.numel() > 1 << 31
    q, k, v = (big(N, heads, width, seed=i) for i in range(3))
    d = -torch.rand((N, heads), device="cuda")
    o, f = comba.linear_attention_step(q, k, v, d, s)
    to, tf = comba.linear_attention_step(q[-3:], k[-3:], v[-3:], d[-3:], s[-3:])
    assert torch.equal(o[-3:], to) and torch.equal(f[-3:], tf)
