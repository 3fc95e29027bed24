"""Refusals of linear attention and group norm that need no GPU: the C ABI returns the documented status before
anything is enqueued, the binding raises, and the workspace sizes follow from the sizes."""
import ctypes

import pytest
import torch

import bilinear_rnn_amd as comba
from bilinear_rnn_amd import api

INVALID, UNSUPPORTED, SHORT = api.COMBA_ERR_INVALID_ARG, api.COMBA_ERR_UNSUPPORTED, api.COMBA_ERR_WORKSPACE
P = 4096            # never dereferenced: every call below fails validation first
BIG = 1 << 60


def ptr(v):
    return ctypes.c_void_p(v) if isinstance(v, int) and v else None


def attn(**kw):
    a = dict(q=P, k=P, v=P, g=P, per=1, s0=None, cu=None, n=0, B=2, T=8, H=4, Hk=2, K=16, V=16, dt=0, scale=1.0, o=P,
             sf=None, ws=P, wsb=BIG)
    a.update(kw)
    return comba.lib().comba_linear_attn_fwd(
        ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["g"]), a["per"], ptr(a["s0"]), ptr(a["cu"]), a["n"], a["B"], a["T"],
        a["H"], a["Hk"], a["K"], a["V"], a["dt"], a["scale"], ptr(a["o"]), ptr(a["sf"]), ptr(a["ws"]), a["wsb"], None)


def attn_step(**kw):
    a = dict(q=P, k=P, v=P, g=P, per=1, s0=None, N=2, H=4, Hk=2, K=16, V=16, dt=0, scale=1.0, o=P, sf=None)
    a.update(kw)
    return comba.lib().comba_linear_attn_step(
        ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["g"]), a["per"], ptr(a["s0"]), a["N"], a["H"], a["Hk"], a["K"], a["V"],
        a["dt"], a["scale"], ptr(a["o"]), ptr(a["sf"]), None)


def attn_bwd(**kw):
    a = dict(q=P, k=P, v=P, g=P, per=1, s0=None, cu=None, n=0, B=2, T=8, H=4, Hk=2, K=16, V=16, dt=0, scale=1.0, do=P,
             dsf=None, dq=P, dk=P, dv=P, dg=P, ds0=None, ws=P, wsb=BIG)
    a.update(kw)
    return comba.lib().comba_linear_attn_bwd(
        ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["g"]), a["per"], ptr(a["s0"]), ptr(a["cu"]), a["n"], a["B"], a["T"],
        a["H"], a["Hk"], a["K"], a["V"], a["dt"], a["scale"], ptr(a["do"]), ptr(a["dsf"]), ptr(a["dq"]), ptr(a["dk"]),
        ptr(a["dv"]), ptr(a["dg"]), ptr(a["ds0"]), ptr(a["ws"]), a["wsb"], None)


def norm(**kw):
    a = dict(x=P, w=P, b=P, cu=None, n=0, B=2, T=8, D=16, G=2, eps=1e-5, dt=0, y=P, st=P, ws=P, wsb=BIG)
    a.update(kw)
    return comba.lib().comba_group_norm_fwd(
        ptr(a["x"]), ptr(a["w"]), ptr(a["b"]), ptr(a["cu"]), a["n"], a["B"], a["T"], a["D"], a["G"], a["eps"], a["dt"], 1,
        ptr(a["y"]), ptr(a["st"]), ptr(a["ws"]), a["wsb"], None)


def norm_bwd(**kw):
    a = dict(x=P, dy=P, st=P, w=P, b=P, cu=None, n=0, B=2, T=8, D=16, G=2, dt=0, dx=P, dw=P, db=P, ws=P, wsb=BIG)
    a.update(kw)
    return comba.lib().comba_group_norm_bwd(
        ptr(a["x"]), ptr(a["dy"]), ptr(a["st"]), ptr(a["w"]), ptr(a["b"]), ptr(a["cu"]), a["n"], a["B"], a["T"], a["D"],
        a["G"], a["dt"], 1, ptr(a["dx"]), ptr(a["dw"]), ptr(a["db"]), ptr(a["ws"]), a["wsb"], None)


BATCH = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(cu=P, n=2), INVALID), (dict(cu=P, n=0, B=1), INVALID),
         (dict(cu=P, n=1, B=1, T=-1), INVALID), (dict(B=1 << 16, T=1 << 15), UNSUPPORTED),
         (dict(B=1, T=(1 << 31) - 40), UNSUPPORTED)]
ATTN = [(dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
        (dict(dt=2), INVALID), (dict(dt=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(Hk=3), INVALID),
        (dict(Hk=8), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(K=7), UNSUPPORTED),
        (dict(V=7), UNSUPPORTED), (dict(K=257), UNSUPPORTED), (dict(V=257), UNSUPPORTED),
        (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
        (dict(H=1 << 15, Hk=1, K=129), UNSUPPORTED)]
NORM = [(dict(x=None), INVALID), (dict(dt=2), INVALID), (dict(D=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
        (dict(G=32), INVALID), (dict(D=(1 << 22) + 1, G=1), UNSUPPORTED)]

ALL = ([(attn, k, c) for k, c in BATCH + ATTN + [
           (dict(o=None), INVALID), (dict(s0=P, sf=P + 4), INVALID),
           # cut along time: the states of the segments
           (dict(B=1, T=4096, ws=None), SHORT), (dict(B=1, T=4096, wsb=64), SHORT), (dict(B=1, T=4096, ws=P + 16), INVALID),
           # more than 2^32 - 1 threads
           (dict(B=1 << 20, T=1, H=16, Hk=16), UNSUPPORTED), (dict(cu=P, n=1 << 24, B=1, T=1 << 24, H=1, Hk=1), UNSUPPORTED)]]
       + [(attn_step, k, c) for k, c in ATTN + [
           (dict(o=None), INVALID), (dict(N=0), INVALID), (dict(s0=P, sf=P + 4), INVALID),
           (dict(N=1 << 24, V=32), UNSUPPORTED)]]
       + [(attn_bwd, k, c) for k, c in BATCH + ATTN + [
           (dict(do=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
           (dict(dg=None), INVALID), (dict(ws=None), SHORT), (dict(wsb=64), SHORT), (dict(ws=P + 16), INVALID),
           (dict(B=1 << 20, T=1, H=16, Hk=16), UNSUPPORTED)]]
       + [(norm, k, c) for k, c in BATCH + NORM + [
           (dict(y=None), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
           (dict(eps=float("inf")), INVALID), (dict(ws=None), SHORT), (dict(wsb=8), SHORT), (dict(ws=P + 16), INVALID),
           (dict(cu=P, n=1 << 20, B=1, T=1 << 20, D=1 << 14), UNSUPPORTED)]]
       + [(norm_bwd, k, c) for k, c in BATCH + NORM + [
           (dict(dy=None), INVALID), (dict(st=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
           (dict(db=None), INVALID), (dict(w=None), INVALID), (dict(b=None), INVALID), (dict(ws=None), SHORT),
           (dict(wsb=8), SHORT), (dict(ws=P + 16), INVALID), (dict(T=1, ws=None), SHORT),
           (dict(cu=P, n=1 << 20, B=1, T=1 << 20, D=1 << 14), UNSUPPORTED)]])


@pytest.mark.parametrize("fn,kw,code", ALL, ids=lambda v: getattr(v, "__name__", str(v)))
def test_bad_arguments_are_refused_before_launch(fn, kw, code):
    assert fn(**kw) == code
    assert api.last_error() != ""


# Distinct addresses for the tensors of a call, far enough apart for the sizes used below.
def apart(names):
    return {k: (i + 1) << 32 for i, k in enumerate(names)}


ATTN_T, STEP_T = apart(("q", "k", "v", "g", "s0", "o", "sf", "ws")), apart(("q", "k", "v", "g", "s0", "o", "sf"))
ATTN_B = apart(("q", "k", "v", "g", "s0", "do", "dsf", "dq", "dk", "dv", "dg", "ds0", "ws"))
NORM_T = apart(("x", "w", "b", "y", "st", "ws"))
NORM_B = apart(("x", "dy", "st", "w", "b", "dx", "dw", "db", "ws"))
VO, QK, G = 2 * 8 * 4 * 16 * 2, 2 * 8 * 2 * 16 * 2, 2 * 8 * 4 * 4   # bytes of v and o, of q and k, of the decays


@pytest.mark.parametrize("fn,base,kw", [
    (attn, ATTN_T, dict(o=ATTN_T["v"])), (attn, ATTN_T, dict(o=ATTN_T["q"] + QK - 2)), (attn, ATTN_T, dict(o=ATTN_T["g"])),
    (attn, ATTN_T, dict(o=ATTN_T["k"] - VO + 2)), (attn, ATTN_T, dict(o=ATTN_T["s0"])),
    (attn, ATTN_T, dict(o=ATTN_T["sf"])), (attn, ATTN_T, dict(sf=ATTN_T["q"])), (attn, ATTN_T, dict(sf=ATTN_T["g"] + G - 4)),
    (attn, ATTN_T, dict(B=1, T=4096, ws=ATTN_T["v"])), (attn, ATTN_T, dict(B=1, T=4096, ws=ATTN_T["sf"])),
    (attn, ATTN_T, dict(B=1, T=4096, ws=ATTN_T["o"])),
    (attn_step, STEP_T, dict(o=STEP_T["v"])), (attn_step, STEP_T, dict(o=STEP_T["sf"])),
    (attn_step, STEP_T, dict(o=STEP_T["s0"])), (attn_step, STEP_T, dict(sf=STEP_T["k"])),
    (attn_bwd, ATTN_B, dict(dq=ATTN_B["q"])), (attn_bwd, ATTN_B, dict(dk=ATTN_B["dq"])),
    (attn_bwd, ATTN_B, dict(dv=ATTN_B["do"])), (attn_bwd, ATTN_B, dict(dg=ATTN_B["g"])),
    (attn_bwd, ATTN_B, dict(ds0=ATTN_B["s0"])), (attn_bwd, ATTN_B, dict(ds0=ATTN_B["dsf"])),
    (attn_bwd, ATTN_B, dict(ws=ATTN_B["dsf"])), (attn_bwd, ATTN_B, dict(ws=ATTN_B["dq"])),
    (norm, NORM_T, dict(y=NORM_T["x"])), (norm, NORM_T, dict(st=NORM_T["x"])), (norm, NORM_T, dict(st=NORM_T["y"] + 8)),
    (norm, NORM_T, dict(ws=NORM_T["x"])), (norm, NORM_T, dict(y=NORM_T["w"])),
    (norm_bwd, NORM_B, dict(dx=NORM_B["dy"])), (norm_bwd, NORM_B, dict(dx=NORM_B["st"])),
    (norm_bwd, NORM_B, dict(dw=NORM_B["db"])), (norm_bwd, NORM_B, dict(dw=NORM_B["w"])),
    (norm_bwd, NORM_B, dict(ws=NORM_B["dx"])),
], ids=lambda v: getattr(v, "__name__", "-".join(v) if isinstance(v, dict) else str(v)))
def test_overlapping_tensors_are_refused(fn, base, kw):
    assert fn(**{**base, **kw}) == INVALID
    assert "overlap" in api.last_error()


def test_workspace_sizes():
    L = comba.lib()
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    size = comba.linear_attention_workspace_size
    assert size(8, 4096, 16, 16, 128, 128) == 0          # 8 x 16 heads x 2 column blocks are 256 workgroups
    # one prompt: 16 workgroups of 128 columns, segments of 65536 * 16 / 256 tokens
    assert size(1, 65536, 16, 16, 128, 128) == up(16 * 16 * 128 * 128 * 4) + up(16 * 16 * 8)
    # packed: segments of 1.5 times a compute unit's share, T / L + N + 1 slots
    assert size(1, 5000, 4, 2, 64, 64, 3) == up((5000 // 256 + 4) * 4 * 64 * 64 * 4) + up((5000 // 256 + 4) * 4 * 8)
    assert size(1, 256, 1, 1, 8, 8) == 0 and size(1, 257, 1, 1, 8, 8) > 0     # nothing to cut
    assert size(1, 4096, 4, 3, 64, 64) == 0 and size(1, 4096, 1, 1, 7, 64) == 0 and size(1, 4096, 1, 1, 64, 257) == 0
    # backward: segments of B T H / 128 tokens; two states, decays, <gradient, state>, dot products, head sums
    bwd, slots = L.comba_linear_attn_bwd_workspace_size, 8
    units = slots * 16
    want = 2 * up(units * 128 * 128 * 4) + up(units * 8) + up(units * 16 * 8) + up(4 * 2 * 4 * 2048 * 16 * 4) + up(units * 8)
    assert bwd(4, 2048, 16, 16, 128, 128, 0) == want
    assert bwd(4, 2048, 16, 8, 128, 128, 0) == want + up(2 * 4 * 2048 * 16 * 128 * 4)   # shared heads: all heads' dq, dk
    norm, nb = L.comba_group_norm_workspace_size, L.comba_group_norm_bwd_workspace_size
    assert norm(32768, 1, 2048, 16, 0) == 0                       # rows are in registers
    # backward of rows: 512 workgroups of 16 rows, of 16 groups per token; two sums per channel
    assert nb(32768, 1, 2048, 16, 0) == 512 * 2 * 2048 * 4
    # sequences: four channel blocks of 512, 4 x 2048 x 4 / 1024 tokens per tile; a pair per group and block
    assert norm(4, 2048, 2048, 32, 0) == up(4 * 64 * (32 + 4) * 2 * 4)
    assert nb(4, 2048, 2048, 32, 0) == up(4 * 64 * ((32 + 4) * 2 + 2 * 2048) * 4)
    assert norm(2, 5, 10, 3, 0) == 0 and nb(0, 5, 9, 3, 0) == 0


def test_a_long_sequence_has_few_tiles():
    # every workgroup joins all tiles of its sequence: at most 4096
    assert comba.lib().comba_group_norm_workspace_size(1, 1 << 30, 8, 1, 0) <= 4096 * (1 + 1) * 2 * 4


def test_binding_refuses():
    q, g = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2)
    x, st = torch.zeros(1, 4, 8), torch.zeros(1, 2, 2)
    for call in (lambda: comba.linear_attention(q, q, q, g), lambda: comba.linear_attention_step(q[0], q[0], q[0], g[0]),
                 lambda: comba.linear_attention_bwd(q, q, q, g, q), lambda: comba.group_norm(x, 2),
                 lambda: comba.group_norm_bwd(x, x, st, 2)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    for call in (lambda: comba.linear_attention(None, q, q, g), lambda: comba.group_norm(None, 2)):
        with pytest.raises(TypeError):
            call()
