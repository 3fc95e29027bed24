"""Refusals of the layer operators (short convolution, selective scan, block norms) that need no GPU:
the C ABI returns the documented status before anything is enqueued, the binding raises, and the
workspace sizes follow from the sizes."""
import ctypes

import pytest
import torch

import bilinear_rnn_amd as comba
from bilinear_rnn_amd import api

INVALID, UNSUPPORTED, SHORT = api.COMBA_ERR_INVALID_ARG, api.COMBA_ERR_UNSUPPORTED, api.COMBA_ERR_WORKSPACE
P = 4096            # never dereferenced: every call below fails validation first
BIG = 1 << 50


def ptr(v):
    return ctypes.c_void_p(v) if isinstance(v, int) and v else None


def conv(**kw):
    a = dict(x=P, w=P, b=P, s0=None, cu=None, n=0, B=2, T=8, D=16, W=4, dt=0, y=P, sf=None)
    a.update(kw)
    return comba.lib().comba_short_conv_fwd(ptr(a["x"]), ptr(a["w"]), ptr(a["b"]), ptr(a["s0"]), ptr(a["cu"]), a["n"],
                                            a["B"], a["T"], a["D"], a["W"], a["dt"], 1, ptr(a["y"]), ptr(a["sf"]), None)


def conv_step(**kw):
    a = dict(x=P, w=P, b=P, s0=None, N=2, D=16, W=4, dt=0, y=P, sf=None)
    a.update(kw)
    return comba.lib().comba_short_conv_step(ptr(a["x"]), ptr(a["w"]), ptr(a["b"]), ptr(a["s0"]), a["N"], a["D"],
                                             a["W"], a["dt"], 1, ptr(a["y"]), ptr(a["sf"]), None)


def conv_bwd(**kw):
    a = dict(x=P, w=P, b=P, s0=None, cu=None, n=0, B=2, T=8, D=16, W=4, dt=0, dy=P, dydt=0, dx=P, dw=P, db=None, ws=P,
             wsb=BIG)
    a.update(kw)
    return comba.lib().comba_short_conv_bwd(ptr(a["x"]), ptr(a["w"]), ptr(a["b"]), ptr(a["s0"]), ptr(a["cu"]), a["n"],
                                            a["B"], a["T"], a["D"], a["W"], a["dt"], 1, ptr(a["dy"]), a["dydt"], None,
                                            ptr(a["dx"]), ptr(a["dw"]), ptr(a["db"]), None, ptr(a["ws"]), a["wsb"], None)


def scan(**kw):
    a = dict(x=P, d=P, A=P, Bm=P, C=P, s0=None, cu=None, n=0, B=2, T=8, D=16, S=16, G=1, dt=0, y=P, sf=None, ws=None,
             wsb=0)
    a.update(kw)
    return comba.lib().comba_selective_scan_fwd(
        ptr(a["x"]), ptr(a["d"]), ptr(a["A"]), ptr(a["Bm"]), ptr(a["C"]), None, None, None, 1, ptr(a["s0"]),
        ptr(a["cu"]), a["n"], a["B"], a["T"], a["D"], a["S"], a["G"], a["dt"], ptr(a["y"]), ptr(a["sf"]), ptr(a["ws"]),
        a["wsb"], None)


def scan_step(**kw):
    a = dict(x=P, d=P, A=P, Bm=P, C=P, s0=None, N=2, D=16, S=16, G=1, dt=0, y=P, sf=None)
    a.update(kw)
    return comba.lib().comba_selective_step(ptr(a["x"]), ptr(a["d"]), ptr(a["A"]), ptr(a["Bm"]), ptr(a["C"]), None,
                                            None, None, 1, ptr(a["s0"]), a["N"], a["D"], a["S"], a["G"], a["dt"],
                                            ptr(a["y"]), ptr(a["sf"]), None)


def scan_bwd(**kw):
    a = dict(x=P, d=P, A=P, Bm=P, C=P, z=None, s0=None, cu=None, n=0, B=2, T=8, D=16, S=16, G=1, dt=0, dy=P, dx=P, dd=P,
             dA=P, dB=P, dC=P, dz=None, ws=P, wsb=BIG)
    a.update(kw)
    return comba.lib().comba_selective_scan_bwd(
        ptr(a["x"]), ptr(a["d"]), ptr(a["A"]), ptr(a["Bm"]), ptr(a["C"]), None, ptr(a["z"]), None, 1, ptr(a["s0"]),
        ptr(a["cu"]), a["n"], a["B"], a["T"], a["D"], a["S"], a["G"], a["dt"], ptr(a["dy"]), None, ptr(a["dx"]),
        ptr(a["dd"]), ptr(a["dA"]), ptr(a["dB"]), ptr(a["dC"]), None, ptr(a["dz"]), None, None, ptr(a["ws"]), a["wsb"],
        None)


def norm(**kw):
    a = dict(y=P, g=None, res=None, sc=None, post=P, pre=P, rows=4, D=64, eps=1e-6, dt=0, r=P, n=P)
    a.update(kw)
    return comba.lib().comba_block_norm_fwd(ptr(a["y"]), ptr(a["g"]), ptr(a["res"]), ptr(a["sc"]), ptr(a["post"]),
                                            ptr(a["pre"]), a["rows"], a["D"], a["eps"], a["dt"], ptr(a["r"]),
                                            ptr(a["n"]), None)


def norm_bwd(**kw):
    a = dict(y=P, g=None, res=None, sc=None, post=P, pre=P, rows=4, D=64, eps=1e-6, dt=0, dr=P, dn=P, dy=P, dg=None,
             dres=None, dsc=None, dpost=P, dpre=P, ws=P, wsb=BIG)
    a.update(kw)
    return comba.lib().comba_block_norm_bwd(
        ptr(a["y"]), ptr(a["g"]), ptr(a["res"]), ptr(a["sc"]), ptr(a["post"]), ptr(a["pre"]), a["rows"], a["D"],
        a["eps"], a["dt"], ptr(a["dr"]), ptr(a["dn"]), ptr(a["dy"]), ptr(a["dg"]), ptr(a["dres"]), ptr(a["dsc"]),
        ptr(a["dpost"]), ptr(a["dpre"]), ptr(a["ws"]), a["wsb"], None)


SEQ = [(dict(x=None), INVALID), (dict(dt=2), INVALID), (dict(dt=-1), INVALID), (dict(D=0), INVALID),
       (dict(D=(1 << 22) + 1), UNSUPPORTED)]
BATCH = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(cu=P, n=2), INVALID), (dict(cu=P, n=0, B=1), INVALID),
         (dict(cu=P, n=1, B=1, T=-1), INVALID), (dict(B=1 << 16, T=1 << 15), UNSUPPORTED)]
STEP = [(dict(N=0), INVALID)]
CONV = [(dict(w=None), INVALID), (dict(W=0), INVALID), (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED)]
SCAN = [(dict(d=None), INVALID), (dict(A=None), INVALID), (dict(Bm=None), INVALID), (dict(C=None), INVALID),
        (dict(S=0), INVALID), (dict(S=65), UNSUPPORTED), (dict(G=0), INVALID), (dict(G=3), INVALID)]
NORM = [(dict(y=None), INVALID), (dict(dt=7), INVALID), (dict(rows=-1), INVALID), (dict(D=0), INVALID),
        (dict(D=16385), UNSUPPORTED), (dict(rows=(1 << 40) + 1), UNSUPPORTED), (dict(eps=-1e-6), INVALID),
        (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID)]

ALL = ([(conv, k, c) for k, c in SEQ + BATCH + CONV + [
           (dict(y=None), INVALID), (dict(s0=P, sf=P), INVALID), (dict(s0=P, sf=P + 2), INVALID),
           (dict(B=1, T=(1 << 31) - 1, D=1 << 22), UNSUPPORTED)]]
       + [(conv_step, k, c) for k, c in SEQ + STEP + CONV + [
           (dict(y=None), INVALID), (dict(s0=P, sf=P + 2), INVALID), (dict(N=1 << 20, D=1 << 12), UNSUPPORTED)]]
       + [(conv_bwd, k, c) for k, c in SEQ + BATCH + CONV + [
           (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(dydt=2), INVALID),
           (dict(dt=1, dydt=0), INVALID), (dict(ws=None), SHORT), (dict(wsb=64), SHORT), (dict(ws=P + 16), INVALID)]]
       + [(scan, k, c) for k, c in SEQ + BATCH + SCAN + [
           (dict(y=None), INVALID), (dict(s0=P, sf=P + 4), INVALID),
           (dict(B=1, T=4096, D=64), SHORT), (dict(B=1, T=4096, D=64, ws=P, wsb=64), SHORT),
           (dict(B=1, T=4096, D=64, ws=P + 16, wsb=BIG), INVALID),
           (dict(B=1 << 20, T=1, D=1 << 22), UNSUPPORTED)]]
       + [(scan_step, k, c) for k, c in SEQ + STEP + SCAN + [
           (dict(y=None), INVALID), (dict(s0=P, sf=P + 4), INVALID), (dict(N=1 << 30, D=1 << 12), UNSUPPORTED)]]
       + [(scan_bwd, k, c) for k, c in SEQ + BATCH + SCAN + [
           (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dd=None), INVALID), (dict(dA=None), INVALID),
           (dict(dB=None), INVALID), (dict(dC=None), INVALID), (dict(z=P), INVALID), (dict(dz=P), INVALID),
           (dict(ws=None), SHORT), (dict(wsb=64), SHORT), (dict(ws=P + 16), INVALID)]]
       + [(norm, k, c) for k, c in NORM + [
           (dict(r=None), INVALID), (dict(n=None), INVALID), (dict(pre=None), INVALID),
           (dict(post=None, pre=None, n=None), INVALID)]]
       + [(norm_bwd, k, c) for k, c in NORM + [
           (dict(dy=None), INVALID), (dict(dr=None, dn=None), INVALID), (dict(pre=None, dpre=None), INVALID),
           (dict(g=P), INVALID), (dict(dg=P), INVALID), (dict(res=P), INVALID), (dict(sc=P), INVALID),
           (dict(dpost=None), INVALID), (dict(dpre=None), INVALID), (dict(ws=None), SHORT), (dict(wsb=64), SHORT),
           (dict(ws=P + 16), INVALID)]])


@pytest.mark.parametrize("fn,kw,code", ALL, ids=lambda v: getattr(v, "__name__", str(v)))
def test_bad_arguments_are_refused_before_launch(fn, kw, code):
    assert fn(**kw) == code
    assert api.last_error() != ""


def test_workspace_sizes():
    L = comba.lib()
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    # convolution: W + 1 float32 rows of D per set of four token tiles; none without tokens
    ws = L.comba_short_conv_bwd_workspace_size
    assert ws(4, 2048, 2048, 4, 0) == up(4 * 2048 // 32 // 4 * 5 * 2048 * 4)
    assert ws(1, 0, 16, 4, 2) == 0 and ws(1, 8, 16, 5, 0) == 0
    # scan: none while the sequences and channels fill the chip
    size = comba.selective_scan_workspace_size
    assert size(8, 4096, 2048, 16) == 0
    # 2048 channels are 64 workgroups: segments of 65536 * 64 / 2048, at most 1024 tokens
    assert size(1, 65536, 2048, 16) == up(64 * 2048 * 16 * 4) + up(64 * 2048 * 4)
    # packed: T / L + N + 1 slots; few workgroups, so the shortest segments, 64 tokens
    assert size(1, 5000, 64, 8, 1, 3) == up((5000 // 64 + 4) * 64 * 8 * 4) + up((5000 // 64 + 4) * 64 * 4)
    assert size(1, 255, 64, 8) == 0 and size(1, 256, 64, 8) > 0      # short batches stay whole
    assert size(1, 100, 65, 16, 2) == 0          # G does not divide D
    # backward: 128 tokens per segment up to 16 states; three state arrays, four rows of D, B and C
    bwd = L.comba_selective_scan_bwd_workspace_size
    slots = 4 * 2048 // 128
    assert bwd(4, 2048, 2048, 16, 1, 0) == (3 * up(slots * 2048 * 16 * 4) + up(slots * 2048 * 4) + up(slots * 2 * 2048 * 4)
                                            + up(32 * 4 * 2048 * 2 * 16 * 4))
    # a small batch: segments of one piece, 16 tokens
    slots = 7
    assert bwd(1, 100, 64, 16, 1, 0) == (3 * up(slots * 64 * 16 * 4) + up(slots * 64 * 4) + up(slots * 2 * 64 * 4)
                                         + up(100 * 2 * 16 * 4))
    norm_ws = L.comba_block_norm_bwd_workspace_size
    assert norm_ws(8192, 2048) == 512 * 3 * 2048 * 4 and norm_ws(0, 64) == 0 and norm_ws(5, 16385) == 0
    assert norm_ws(3, 64) == 3 * 64 * 4 and norm_ws(33, 64) == up(2 * 3 * 64 * 4)   # 32 rows per workgroup


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: comba.short_conv(x, w), lambda: comba.short_conv_step(x[0], w),
                 lambda: comba.short_conv_bwd(x, w, None, x),
                 lambda: comba.selective_scan(x, x, w, x[..., None], x[..., None]),
                 lambda: comba.selective_step(x[0], x[0], w, x[0][..., None], x[0][..., None]),
                 lambda: comba.selective_scan_bwd(x, x, w, x[..., None], x[..., None], x),
                 lambda: comba.block_norm(x, post_weight=w[0]), lambda: comba.block_norm_bwd(x, x, post_weight=w[0])):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        comba.block_norm(None)


# Distinct addresses for the tensors of a call, far enough apart for the sizes used below.
def apart(names):
    return {k: (i + 1) << 32 for i, k in enumerate(names)}


CONV_T, STEP_T = apart(("x", "w", "b", "y")), apart(("x", "w", "b", "s0", "sf", "y"))
CONV_B = apart(("x", "w", "b", "dy", "dx", "dw", "ws"))
SCAN_T, SCAN_S = apart(("x", "d", "A", "Bm", "C", "y")), apart(("x", "d", "A", "Bm", "C", "s0", "sf", "y"))
SCAN_B = apart(("x", "d", "A", "Bm", "C", "dy", "dx", "dd", "dA", "dB", "dC", "ws"))
NORM_T, NORM_B = apart(("y", "post", "pre", "r", "n")), apart(("y", "post", "pre", "dr", "dn", "dy", "dpost", "dpre", "ws"))


@pytest.mark.parametrize("fn,base,kw", [
    (conv, CONV_T, dict(y=CONV_T["x"])), (conv, CONV_T, dict(y=CONV_T["x"] + 2 * 8 * 16 * 2 - 2)),
    (conv, CONV_T, dict(y=CONV_T["b"] + 60)), (conv, CONV_T, dict(sf=CONV_T["x"])), (conv, CONV_T, dict(sf=CONV_T["y"])),
    (conv_step, STEP_T, dict(y=STEP_T["x"])), (conv_step, STEP_T, dict(y=STEP_T["s0"])),
    (conv_step, STEP_T, dict(sf=STEP_T["x"])),
    (conv_bwd, CONV_B, dict(dx=CONV_B["dy"])), (conv_bwd, CONV_B, dict(dw=CONV_B["w"])),
    (conv_bwd, CONV_B, dict(ws=CONV_B["x"])), (conv_bwd, CONV_B, dict(dw=CONV_B["dx"])),
    (scan, SCAN_T, dict(y=SCAN_T["x"])), (scan, SCAN_T, dict(y=SCAN_T["d"])), (scan, SCAN_T, dict(sf=SCAN_T["A"])),
    (scan, SCAN_T, dict(sf=SCAN_T["y"])), (scan, SCAN_T, dict(B=1, T=4096, D=64, ws=SCAN_T["C"], wsb=BIG)),
    (scan_step, SCAN_S, dict(y=SCAN_S["x"])), (scan_step, SCAN_S, dict(y=SCAN_S["sf"])),
    (scan_step, SCAN_S, dict(sf=SCAN_S["Bm"])),
    (scan_bwd, SCAN_B, dict(dx=SCAN_B["x"])), (scan_bwd, SCAN_B, dict(dd=SCAN_B["dy"])),
    (scan_bwd, SCAN_B, dict(dB=SCAN_B["dC"])), (scan_bwd, SCAN_B, dict(ws=SCAN_B["dy"])),
    (norm, NORM_T, dict(r=NORM_T["y"])), (norm, NORM_T, dict(n=NORM_T["r"] + 4 * 64 * 2 - 16)),
    (norm_bwd, NORM_B, dict(dy=NORM_B["dr"])), (norm_bwd, NORM_B, dict(dpost=NORM_B["dpre"])),
], ids=lambda v: getattr(v, "__name__", "-".join(v) if isinstance(v, dict) else str(v)))
def test_overlapping_tensors_are_refused(fn, base, kw):
    assert fn(**{**base, **kw}) == INVALID
    assert "overlap" in api.last_error()


@pytest.mark.parametrize("fn,kw", [
    # token counters of 32 bits run past the last token by less than two tiles
    (conv, dict(B=1, T=(1 << 31) - 40, D=1)), (conv_bwd, dict(B=1, T=(1 << 31) - 40, D=1)),
    (scan, dict(B=1, T=(1 << 31) - 40, D=1)), (scan_bwd, dict(B=1, T=(1 << 31) - 40, D=1, S=1)),
    # a tile of B and C: 32-bit offsets
    (scan, dict(D=1 << 20, G=1 << 20, S=16)), (scan_step, dict(D=1 << 20, G=1 << 20, S=16)),
    (scan_bwd, dict(D=1 << 20, G=1 << 20, S=16)),
    # a launch of 2^32 threads or more: workgroups, and threads per carried state
    (scan, dict(cu=P, n=1 << 20, B=1, T=1 << 20, D=1 << 12)), (scan_step, dict(N=1 << 27, D=1 << 12)),
    (scan_bwd, dict(cu=P, n=1 << 18, B=1, T=1 << 18, D=1 << 13)), (scan_bwd, dict(B=1 << 16, T=1 << 10, D=4, S=64)),
    (scan_bwd, dict(B=1, T=128, D=1 << 22, S=64)),
], ids=str)
def test_sizes_past_the_kernels_counters_are_refused(fn, kw):
    assert fn(**kw) == UNSUPPORTED
    assert api.last_error() != ""
