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


def linear_attention(q, k, v, log_decay, scale=1.0, init=None, cu=None, do=None, dfin=None, magnitude=False):
    """Returns (o, final_state), or with do a dict of the gradients. log_decay is [B, T, H] or [H].

    With ``magnitude``, decays are taken at half their logarithm (X e^-X <= (2 / e) e^(-X / 2) counts a
    relative error of X per decay), and dlog_decay sums |q . dq| + |k . dk| over the rest of the sequence,
    the terms of the sum that an evaluation may take it from."""
    q, k, v, log_decay, init, do, dfin = (_f(x) for x in (q, k, v, log_decay, init, do, dfin))
    mag = np.abs if magnitude else (lambda x: x)
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    N = _num_seqs(B, cu)
    rep = H // Hk
    head = log_decay.ndim == 1
    g = np.broadcast_to(log_decay, (B, T, H))
    a = np.exp(g / 2 if magnitude else g)
    qh, kh = (mag(np.repeat(x, rep, 2)) for x in (q, k))
    v, scale = mag(v), mag(scale)
    o = np.full_like(v, np.nan)
    fin = np.zeros((N, H, V, K))
    dq, dk = np.full_like(q, np.nan), np.full_like(q, np.nan)
    dv, dg, dinit = np.full_like(v, np.nan), np.full((B, T, H), np.nan), np.zeros_like(fin)
    for n, row, t0, t1 in _segments(B, T, cu):
        S = np.zeros((H, V, K)) if init is None else mag(init[n])
        states = [S]
        for t in range(t0, t1):
            S = a[row, t][:, None, None] * S + v[row, t][:, :, None] * kh[row, t][:, None]
            o[row, t] = scale * np.einsum("hvk,hk->hv", S, qh[row, t])
            states.append(S)
        fin[n] = S
        if do is None:
            continue
        E = np.zeros((H, V, K)) if dfin is None else mag(dfin[n])
        terms = (E * S).sum((1, 2))
        for t in reversed(range(t0, t1)):
            d = scale * mag(do[row, t])
            hq = np.einsum("hvk,hv->hk", states[t - t0 + 1], d)
            E = E + d[:, :, None] * qh[row, t][:, None]
            hk = np.einsum("hvk,hv->hk", E, v[row, t])
            dv[row, t] = np.einsum("hvk,hk->hv", E, kh[row, t])
            dq[row, t], dk[row, t] = (x.reshape(Hk, rep, K).sum(1) for x in (hq, hk))
            E = a[row, t][:, None, None] * E
            terms = terms + (hq * qh[row, t]).sum(1) + (hk * kh[row, t]).sum(1)
            dg[row, t] = terms if magnitude else (E * states[t - t0]).sum((1, 2))
        dinit[n] = E
    if do is None:
        return o, fin
    return dict(dq=dq, dk=dk, dv=dv, dlog_decay=np.nansum(dg, (0, 1)) if head else dg,
                dinitial_state=None if init is None else dinit)


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, silu=False, cu=None, dy=None, magnitude=False):
    """x [B, T, D]. Returns (y, stats), or with dy a dict of the gradients. ``magnitude``: the terms of x - mean
    and of p are added up as absolute values; a relative error of 1 / deviation shows in p itself."""
    x, weight, bias, dy = (_f(v) for v in (x, weight, bias, dy))
    mag = np.abs if magnitude else (lambda v: v)
    B, T, D = x.shape
    C, N = D // groups, _num_seqs(B, cu)
    w = (np.ones(D) if weight is None else weight).reshape(groups, C)
    b = (np.zeros(D) if bias is None else bias).reshape(groups, C)
    y, dx = np.full_like(x, np.nan), np.full_like(x, np.nan)
    stats, dw, db = np.zeros((N, groups, 2)), np.zeros(D), np.zeros(D)
    for n, row, t0, t1 in _segments(B, T, cu):
        if t1 == t0:
            continue
        u = x[row, t0:t1].reshape(t1 - t0, groups, C)
        mean = u.mean((0, 2))
        rstd = 1.0 / np.sqrt(((u - mean[:, None]) ** 2).mean((0, 2)) + eps)
        stats[n] = np.stack([np.abs(u).mean((0, 2)) if magnitude else mean, rstd], -1)
        h = (u - mean[:, None]) * rstd[:, None]
        hm = (np.abs(u) + np.abs(u).mean((0, 2))[:, None]) * rstd[:, None]  # how far h may be off
        p = h * w + b
        pm = hm * np.abs(w) + np.abs(b)
        s = sigmoid(p)
        y[row, t0:t1] = (1.1 * pm if magnitude else p * s if silu else p).reshape(-1, D)
        if dy is None:
            continue
        d = dy[row, t0:t1].reshape(u.shape)
        if silu:  # the slope's own slope is at most 0.5
            d = np.abs(d) * (1.1 + 0.5 * pm) if magnitude else d * s * (1 + p * (1 - s))
        d = mag(d)
        if magnitude:
            h = hm
        g = d * mag(w)
        sign = 1.0 if magnitude else -1.0
        dx[row, t0:t1] = (rstd[:, None] * (g + sign * g.mean((0, 2))[:, None] +
                                           sign * h * (g * h).mean((0, 2))[:, None])).reshape(-1, D)
        dw += (d * h).sum(0).reshape(D)
        db += d.sum(0).reshape(D)
    if dy is None:
        return y, stats
    return dict(dx=dx, dweight=None if weight is None else dw, dbias=None if bias is None else db)
