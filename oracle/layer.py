"""Plain fp64 oracle of the layer operators around the recurrence. TEST INFRASTRUCTURE ONLY.

numpy, token by token, from the formulas in include/comba.h: the short causal depthwise
convolution, the selective state space scan and the block norms, each with its reverse mode.
Layouts as there; with ``cu_seqlens`` rows of tokens in no sequence are NaN in what is returned.

``magnitude=True`` evaluates the same sums with every term replaced by its absolute value: the
scale against which the rounding errors of an evaluation in lower precision are counted.
"""
from __future__ import annotations

import numpy as np

from .reference import _segments


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-x)), np.exp(np.minimum(x, 0)) / (1.0 + np.exp(np.minimum(x, 0))))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def _num_seqs(B, cu):
    return B if cu is None else len(cu) - 1


def short_conv(x, weight, bias=None, init=None, cu=None, silu=True, dy=None, dfin=None, magnitude=False):
    """Returns (y, final_state), or with dy a dict of the gradients."""
    x, weight, bias, init, dy, dfin = (_f(v) for v in (x, weight, bias, init, dy, dfin))
    mag = np.abs if magnitude else (lambda v: v)
    B, T, D = x.shape
    W = weight.shape[1]
    N = _num_seqs(B, cu)
    y = np.full_like(x, np.nan)
    fin = np.zeros((N, W - 1, D))
    dx = np.full_like(x, np.nan)
    dw, db, dinit = np.zeros((D, W)), np.zeros(D), np.zeros((N, W - 1, D))
    b = np.zeros(D) if bias is None else bias
    for n, row, t0, t1 in _segments(B, T, cu):
        L = t1 - t0
        full = np.concatenate([np.zeros((W - 1, D)) if init is None else init[n], x[row, t0:t1]])
        fin[n] = full[L:]
        p = b + sum(full[k:k + L] * weight[:, k] for k in range(W))
        size = np.abs(b) + sum(np.abs(full[k:k + L] * weight[:, k]) for k in range(W))
        s = sigmoid(p)
        if dy is None:
            y[row, t0:t1] = (size if magnitude else p * s if silu else p)
            continue
        # the derivative of p sigmoid(p); its magnitude also covers how far p itself may be off
        slope = 1.0 if not silu else s * (1 + p * (1 - s)) if not magnitude else 1 + size
        dp = mag(dy[row, t0:t1]) * slope
        dfull = np.zeros_like(full)
        for k in range(W):
            dfull[k:k + L] += dp * mag(weight[:, k])
            dw[:, k] += (dp * mag(full[k:k + L])).sum(0)
        db += dp.sum(0)
        if dfin is not None:
            dfull[L:] += mag(dfin[n])
        dx[row, t0:t1] = dfull[W - 1:]
        dinit[n] = dfull[:W - 1]
    if dy is None:
        return y, fin
    return dict(dx=dx, dweight=dw, dbias=None if bias is None else db, dinitial_state=None if init is None else dinit)


def selective_scan(x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, softplus_dt=True, init=None, cu=None, dy=None,
                   dfin=None, magnitude=False):
    """Returns (y, final_state), or with dy a dict of the gradients."""
    x, dt, A, Bm, Cm, skip, z, dt_bias, init, dy, dfin = (
        _f(v) for v in (x, dt, A, Bm, Cm, skip, z, dt_bias, init, dy, dfin))
    mag = np.abs if magnitude else (lambda v: v)
    B, T, D = x.shape
    S, G = A.shape[1], Bm.shape[2]
    N = _num_seqs(B, cu)
    u = dt + (0.0 if dt_bias is None else dt_bias)
    dl = softplus(u) if softplus_dt else u
    x, Bm, Cm, Am = mag(x), mag(Bm), mag(Cm), mag(A)
    sk = np.zeros(D) if skip is None else mag(skip)
    sg = sigmoid(z) if z is not None else None
    gate = mag(z * sg) if z is not None else np.ones_like(x)
    y = np.full_like(x, np.nan)
    fin = np.zeros((N, D, S))
    g = dict(dx=np.full_like(x, np.nan), ddt=np.full_like(x, np.nan), dA=np.zeros_like(A), dB=np.full_like(Bm, np.nan),
             dC=np.full_like(Cm, np.nan), dskip=np.zeros(D), dz=np.full_like(x, np.nan), ddt_bias=np.zeros(D),
             dinitial_state=np.zeros((N, D, S)))
    rep = D // G
    for n, row, t0, t1 in _segments(B, T, cu):
        h = np.zeros((D, S)) if init is None else mag(init[n])
        hs, raw = [h], []
        for t in range(t0, t1):
            d = dl[row, t][:, None]
            h = np.exp(d * A) * h + mag(d) * x[row, t][:, None] * np.repeat(Bm[row, t], rep, 0)
            hs.append(h)
            raw.append((np.repeat(Cm[row, t], rep, 0) * h).sum(1) + sk * x[row, t])
            y[row, t] = raw[-1] * gate[row, t]
        fin[n] = h
        if dy is None:
            continue
        gh = np.zeros((D, S)) if dfin is None else mag(dfin[n])
        for t in reversed(range(t0, t1)):
            d, xt = dl[row, t][:, None], x[row, t]
            b, c = np.repeat(Bm[row, t], rep, 0), np.repeat(Cm[row, t], rep, 0)
            p = mag(dy[row, t]) * gate[row, t]
            gh = gh + p[:, None] * c
            g["dC"][row, t] = (p[:, None] * hs[t - t0 + 1]).reshape(G, rep, S).sum(1)
            g["dB"][row, t] = (gh * mag(d) * xt[:, None]).reshape(G, rep, S).sum(1)
            sb = (gh * b).sum(1)
            g["dx"][row, t] = sk * p + mag(d[:, 0]) * sb
            gh = gh * np.exp(d * A)
            k = gh * hs[t - t0]
            dd = xt * sb + (Am * k).sum(1)
            if softplus_dt:
                dd = dd * sigmoid(u[row, t])
            g["ddt"][row, t] = dd
            g["dA"] += mag(d) * k
            g["dskip"] += p * xt
            g["ddt_bias"] += dd
            if z is not None:
                zt, st = z[row, t], sg[row, t]
                g["dz"][row, t] = mag(dy[row, t]) * raw[t - t0] * (st * (1 + mag(zt) * (1 - st)))
        g["dinitial_state"][n] = gh
    if dy is None:
        return y, fin
    for key, given in (("dskip", skip), ("dz", z), ("ddt_bias", dt_bias), ("dinitial_state", init)):
        if given is None:
            g[key] = None
    return g


def block_norm(y, gate=None, residual=None, scale=None, post_weight=None, pre_weight=None, eps=1e-6, dr=None, dn=None,
               magnitude=False):
    """Returns (r, n), or with dr or dn a dict of the gradients."""
    y, gate, residual, scale, post, pre, dr, dn = (
        _f(v) for v in (y, gate, residual, scale, post_weight, pre_weight, dr, dn))
    mag = np.abs if magnitude else (lambda v: v)
    k1 = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    h = y if post is None else y * k1 * post
    u, v = h, mag(h)  # v: with the magnitudes
    if gate is not None:
        s = sigmoid(gate)
        u, v = u * gate * s, v * mag(gate * s)
    r = (u if scale is None else scale * u) + (0.0 if residual is None else residual)
    rv = (v if scale is None else mag(scale) * v) + (0.0 if residual is None else mag(residual))
    k2 = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    if dr is None and dn is None:
        return rv, None if pre is None else rv * k2 * mag(pre)
    sign = 1.0 if magnitude else -1.0
    g = dict(dgate=None, dresidual=None, dscale=None, dpost_weight=None, dpre_weight=None)
    d = np.zeros_like(y) if dr is None else mag(dr)
    if pre is not None:
        if dn is None:
            g["dpre_weight"] = np.zeros(y.shape[-1])
        else:
            e = mag(dn) * mag(pre)
            g["dpre_weight"] = (mag(dn) * rv * k2).reshape(-1, y.shape[-1]).sum(0)
            d = d + k2 * (e + sign * rv * k2 * k2 * (e * rv).mean(-1, keepdims=True))
    if residual is not None:
        g["dresidual"] = d
    if scale is not None:
        g["dscale"] = (d * v).reshape(-1, y.shape[-1]).sum(0)
        d = d * mag(scale)
    if gate is not None:
        g["dgate"] = d * mag(h) * s * (1 + mag(gate) * (1 - s))
        d = d * mag(gate * s)
    if post is not None:
        g["dpost_weight"] = (d * mag(y) * k1).reshape(-1, y.shape[-1]).sum(0)
        d = d * mag(post)
        d = k1 * (d + sign * mag(y) * k1 * k1 * (d * mag(y)).mean(-1, keepdims=True))
    g["dy"] = d
    return g
