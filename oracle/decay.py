"""Token-by-token definition of the decayed linear attention, its gradients and the 8-bit state cache, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t

with one scalar decay a_t for each head, and query/key heads shared by groups of value heads. Gradients for dO_t and
dS_T, by the chain rule on that rule (G_t the gradient reaching S_t):

    G_T = dS_T + q_T dO_T^T,   G_{t-1} = a_t G_t + q_{t-1} dO_{t-1}^T,   dS0 = a_1 G_1
    dq_t = S_t dO_t,   dk_t = G_t v_t,   dv_t = G_t^T k_t,   da_t = <G_t, S_{t-1}>

Every function also runs on magnitudes (``magnitudes=True``): the same sums over absolute values, which bound the
rounding errors of any evaluation order.

Pinned by: closed forms (a = 0, a = 1, a constant decay), matrix products, central differences, and the gated
delta rule with its erase gate at zero (``tests/test_oracle_decay.py``)."""
from __future__ import annotations

import numpy as np


def _f(x, magnitudes):
    x = np.asarray(x, dtype=np.float64)
    return np.abs(x) if magnitudes else x


def _group(x, H):
    """[.., Hk, d] as [.., H, d]."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def _spans(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, alpha, S0=None, cu=None, magnitudes=False, states=False):
    """(o [B,T,H,dv], S_T [N,H,dk,dv]); with ``states`` also a list with the states before each token and after the
    last, [len + 1, H, dk, dv] for each sequence. Rows outside every sequence stay zero."""
    q, k, v, a = (_f(x, magnitudes) for x in (q, k, v, alpha))
    B, T, H, dv = v.shape
    dk = q.shape[-1]
    q, k = _group(q, H), _group(k, H)
    a = np.broadcast_to(a, (B, T, H)) if a.ndim == 1 else a
    spans = _spans(B, T, cu)
    o, S_T, kept = np.zeros((B, T, H, dv)), np.zeros((len(spans), H, dk, dv)), []
    for n, (b, t0, t1) in enumerate(spans):
        S = np.zeros((H, dk, dv)) if S0 is None else _f(S0[n], magnitudes).copy()
        seen = [S]
        for t in range(t0, t1):
            S = a[b, t][:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = np.matmul(q[b, t][:, None, :], S)[:, 0]
            if states:
                seen.append(S)
        S_T[n] = S
        kept.append(seen)
    return (o, S_T, kept) if states else (o, S_T)


def backward(q, k, v, alpha, dO, dS_T=None, S0=None, cu=None, magnitudes=False):
    """Dict of dq, dk, dv, dalpha (shape of alpha) and dS0."""
    _, _, kept = forward(q, k, v, alpha, S0, cu, magnitudes, states=True)
    per_head = np.ndim(alpha) == 1
    q, k, v, a, dO = (_f(x, magnitudes) for x in (q, k, v, alpha, dO))
    B, T, H, dv = v.shape
    Hk, dk = q.shape[-2:]
    qg, kg = _group(q, H), _group(k, H)
    a = np.broadcast_to(a, (B, T, H)) if per_head else a
    dq, dk_, dv_, da = np.zeros((B, T, H, dk)), np.zeros((B, T, H, dk)), np.zeros((B, T, H, dv)), np.zeros((B, T, H))
    spans = _spans(B, T, cu)
    dS0 = np.zeros((len(spans), H, dk, dv))
    for n, (b, t0, t1) in enumerate(spans):
        G = np.zeros((H, dk, dv)) if dS_T is None else _f(dS_T[n], magnitudes).copy()
        for t in range(t1 - 1, t0 - 1, -1):
            G = G + qg[b, t][:, :, None] * dO[b, t][:, None, :]
            before, after = kept[n][t - t0], kept[n][t - t0 + 1]
            dq[b, t] = np.matmul(after, dO[b, t][:, :, None])[..., 0]
            dk_[b, t] = np.matmul(G, v[b, t][:, :, None])[..., 0]
            dv_[b, t] = np.matmul(kg[b, t][:, None, :], G)[:, 0]
            da[b, t] = (G * before).sum((-1, -2))
            G = a[b, t][:, None, None] * G
        dS0[n] = G
    share = lambda x: x.reshape(B, T, Hk, H // Hk, dk).sum(3)  # noqa: E731
    return dict(dq=share(dq), dk=share(dk_), dv=dv_, dalpha=da.sum((0, 1)) if per_head else da, dS0=dS0)


def step(S, q, k, v, alpha, magnitudes=False):
    """One token: (S_t, o_t) for S [N,H,dk,dv], q, k [N,Hk,dk], v [N,H,dv], alpha [N,H] or [H]."""
    S, q, k, v, a = (_f(x, magnitudes) for x in (S, q, k, v, alpha))
    H = v.shape[1]
    q, k = _group(q, H), _group(k, H)
    a = np.broadcast_to(a, v.shape[:2])
    S = a[..., None, None] * S + k[..., :, None] * v[..., None, :]
    return S, np.matmul(q[..., None, :], S)[..., 0, :]


def pack(S, fmt):
    """(values held, scales) of states in the 8-bit cache: values are code * scale. A row with a non-finite entry
    reads back as NaN. The scale of int8 is a float32 number; everything else is exact in float64."""
    S = np.asarray(S, dtype=np.float64)
    top = np.abs(S).max(-1)
    bad = ~np.isfinite(S).all(-1)
    top = np.where(bad, 0.0, top)
    x = np.where(bad[..., None], 0.0, S)
    if fmt == "int8":
        r = np.float64(np.float32(1) / np.float32(127))
        scale = np.maximum((top * r).astype(np.float32).astype(np.float64), 2.0 ** -126)
        held = np.rint(x / scale[..., None])
    else:
        m, e = np.frexp(top)
        scale = np.ldexp(1.0, np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126))
        scale = np.where(top == 0, 2.0 ** -126, scale)
        y = x / scale[..., None]
        step_ = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)  # spacing of e4m3 around y
        held = np.rint(y / step_) * step_
    scale = np.where(bad, np.nan, scale)
    return held * scale[..., None], scale
