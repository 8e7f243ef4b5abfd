"""Token-by-token definitions, in float64, of what a layer runs around a recurrence: the short causal convolution, the
selective scan and the norm, with their gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Every function also runs on magnitudes (``magnitudes=True``): the same sums over absolute values, which bound the rounding
errors of any evaluation order.

Pinned by: closed forms, ``numpy.convolve``, the decayed linear attention with one decay for a head, central differences
(``tests/test_oracle_layer.py``)."""
from __future__ import annotations

import numpy as np

from .decay import _f, _spans, pack


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def _silu(x, magnitudes):
    """x sigmoid(x); with magnitudes x may be the magnitude of a sum, whose silu is at most it."""
    return np.abs(x) if magnitudes else x * sigmoid(x)


def _dsilu(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


# ------------------------------------------------------------------------------------------------ convolution
def _conv_pre(x, w, b, e0):
    W = w.shape[1]
    e = np.concatenate([e0, x])
    return e, b + sum(w[:, j] * e[j:j + len(x)] for j in range(W))


def conv(x, w, b=None, state=None, cu=None, act="silu", magnitudes=False):
    """(y [B,T,C], state_T [N,W-1,C]). Rows outside every sequence stay zero."""
    x, w = _f(x, magnitudes), _f(w, magnitudes)
    B, T, C = x.shape
    W = w.shape[1]
    b = np.zeros(C) if b is None else _f(b, magnitudes)
    spans = _spans(B, T, cu)
    y, last = np.zeros((B, T, C)), np.zeros((len(spans), W - 1, C))
    for n, (r, t0, t1) in enumerate(spans):
        e, u = _conv_pre(x[r, t0:t1], w, b, np.zeros((W - 1, C)) if state is None else _f(state[n], magnitudes))
        y[r, t0:t1] = _silu(u, magnitudes) if act == "silu" else u
        last[n] = e[t1 - t0:]
    return y, last


def conv_grad(x, w, b, state, cu, act, dy, dstate_T=None, magnitudes=False):
    """Dict of dx, dweight, dbias, dstate."""
    x, w, dy = np.asarray(x, np.float64), np.asarray(w, np.float64), _f(dy, magnitudes)
    B, T, C = x.shape
    W = w.shape[1]
    b = np.zeros(C) if b is None else np.asarray(b, np.float64)
    spans = _spans(B, T, cu)
    dx, dw, db, ds = np.zeros(x.shape), np.zeros(w.shape), np.zeros(C), np.zeros((len(spans), W - 1, C))
    for n, (r, t0, t1) in enumerate(spans):
        L = t1 - t0
        e, u = _conv_pre(x[r, t0:t1], w, b, np.zeros((W - 1, C)) if state is None else np.asarray(state[n], np.float64))
        du = dy[r, t0:t1]
        if act == "silu":  # |silu'| <= 1.1, |silu''| <= 1/2: an error of u moves du by half of it
            mag = _conv_pre(np.abs(x[r, t0:t1]), np.abs(w), np.abs(b), np.abs(e[:W - 1]))[1] if magnitudes else 0.0
            du = du * (1.1 + 0.5 * mag if magnitudes else _dsilu(u))
        if magnitudes:
            e = np.abs(e)
        de = np.zeros((L + W - 1, C))
        for j in range(W):
            de[j:j + L] += _f(w[:, j], magnitudes) * du
            dw[:, j] += (du * e[j:j + L]).sum(0)
        if dstate_T is not None:
            de[L:] += _f(dstate_T[n], magnitudes)
        db += du.sum(0)
        ds[n], dx[r, t0:t1] = de[:W - 1], de[W - 1:]
    return dict(dx=dx, dweight=dw, dbias=db, dstate=ds)


# ------------------------------------------------------------------------------------------------ selective scan
def _wide(m, C):
    """[.., G, N] by channel: [.., C, N]."""
    return np.repeat(m, C // m.shape[-2], axis=-2)


def _steps(dt, bias, soft):
    raw = np.asarray(dt, np.float64) + (0.0 if bias is None else np.asarray(bias, np.float64))
    return raw, softplus(raw) if soft else raw


def scan(x, dt, A, B, C, D=None, z=None, bias=None, S0=None, cu=None, soft=True, magnitudes=False, states=False):
    """(y [Bt,T,Ch], S_T [N,Ch,n]), with ``states`` also the y before the gate and for each sequence the states before each
    token and after the last. Rows outside every sequence stay zero."""
    A = np.asarray(A, np.float64)
    raw, d = _steps(dt, bias, soft)
    x, Bm, Cm = _f(x, magnitudes), _wide(_f(B, magnitudes), x.shape[-1]), _wide(_f(C, magnitudes), x.shape[-1])
    Bt, T, Ch = x.shape
    spans = _spans(Bt, T, cu)
    y, S_T, kept = np.zeros(x.shape), np.zeros((len(spans),) + A.shape), []
    for n, (b, t0, t1) in enumerate(spans):
        h = np.zeros(A.shape) if S0 is None else _f(S0[n], magnitudes)
        seen = [h]
        for t in range(t0, t1):
            h = np.exp(d[b, t][:, None] * A) * h + _f(d[b, t] * x[b, t], magnitudes)[:, None] * Bm[b, t]
            y[b, t] = (h * Cm[b, t]).sum(-1) + (0.0 if D is None else _f(D, magnitudes) * x[b, t])
            seen.append(h)
        S_T[n] = h
        kept.append(seen)
    gated = y if z is None else y * (np.abs(z) if magnitudes else _silu(np.asarray(z, np.float64), False))
    return (gated, S_T, y, kept) if states else (gated, S_T)


def scan_grad(x, dt, A, B, C, D, z, bias, S0, cu, soft, dy, dS_T=None, magnitudes=False):
    """Dict of dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dS0."""
    _, _, pre, kept = scan(x, dt, A, B, C, D, z, bias, S0, cu, soft, magnitudes, states=True)
    A = np.asarray(A, np.float64)
    raw, d = _steps(dt, bias, soft)
    sg = sigmoid(raw) if soft else np.ones_like(raw)
    G, N = np.shape(B)[-2:]
    x, dy = _f(x, magnitudes), _f(dy, magnitudes)
    Bt, T, Ch = x.shape
    Bm, Cm = _wide(_f(B, magnitudes), Ch), _wide(_f(C, magnitudes), Ch)
    spans = _spans(Bt, T, cu)
    o = dict(dx=np.zeros(x.shape), ddt=np.zeros(x.shape), dA=np.zeros(A.shape), dB=np.zeros((Bt, T, G, N)), dC=np.zeros((Bt, T, G, N)),
             dD=np.zeros(Ch), dz=np.zeros(x.shape), ddt_bias=np.zeros(Ch), dS0=np.zeros((len(spans),) + A.shape))
    gy = dy
    if z is not None:
        z = np.asarray(z, np.float64)
        o["dz"] = dy * pre * (1.1 if magnitudes else _dsilu(z))
        gy = dy * (np.abs(z) if magnitudes else _silu(z, False))
    Dv, dm = (0.0 if D is None else _f(D, magnitudes)), _f(d, magnitudes)
    for n, (b, t0, t1) in enumerate(spans):
        g = np.zeros(A.shape) if dS_T is None else _f(dS_T[n], magnitudes)
        for t in range(t1 - 1, t0 - 1, -1):
            g = g + gy[b, t][:, None] * Cm[b, t]
            a = np.exp(d[b, t][:, None] * A)
            o["dC"][b, t] = (kept[n][t - t0 + 1] * gy[b, t][:, None]).reshape(G, -1, N).sum(1)
            o["dB"][b, t] = (g * (dm[b, t] * x[b, t])[:, None]).reshape(G, -1, N).sum(1)
            u = (g * Bm[b, t]).sum(-1)
            w = g * a * kept[n][t - t0]
            o["dA"] += w * dm[b, t][:, None]
            o["dx"][b, t] = u * dm[b, t] + Dv * gy[b, t]
            o["ddt"][b, t] = ((w * _f(A, magnitudes)).sum(-1) + u * x[b, t]) * sg[b, t]
            g = g * a
        o["dS0"][n] = g
        o["dD"] += (gy[b, t0:t1] * x[b, t0:t1]).sum(0)
        o["ddt_bias"] += o["ddt"][b, t0:t1].sum(0)
    return o


# ------------------------------------------------------------------------------------------------ norm
def norm(h, w, eps=1e-5, fmt=None):
    """y of rows h [R,C], or with ``fmt`` (values held, scales): p = h w as float32 numbers held as a row of the 8-bit cache is,
    times 1 / sqrt(mean h^2 + eps)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    if fmt is None:
        return h * w * r
    held, scale = pack((h * w).astype(np.float32), fmt)
    return held * r, scale * r[:, 0]


def norm_grad(h, w, dy, dh=None, eps=1e-5):
    """Dict of dx, dweight."""
    h, w, dy = (np.asarray(a, np.float64) for a in (h, w, dy))
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    wd = w * dy
    dx = r * (wd - h * r * r * (wd * h).mean(-1, keepdims=True))
    return dict(dx=dx if dh is None else dx + np.asarray(dh, np.float64), dweight=(dy * h * r).sum(0))
