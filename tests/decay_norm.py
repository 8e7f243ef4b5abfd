"""The decayed linear attention's stated precision: errors in the 2-norm, and a model of the chunked evaluation."""
from __future__ import annotations

import numpy as np
import torch

from oracle import decay as oracle

# A result passes in its chunk some twelve sums of a matrix core (terms, halves of the tokens) and the state's part as
# many for each chunk that it remembers: with decays of 1 - 2^-9 a chunk leaves 0.88 of the state, so that
# 1 / (1 - 0.88^2) = 4.5 chunks' roundings of independent sign add up, 12 + 12 * 4.5 = 66 in all. Each is at most 2^-23
# of its value (a matrix core may cut a sum), 2^-23 / sqrt(3) in the mean square.
LIMIT = (66 / 3) ** 0.5 * 2.0 ** -23  # 5.6e-7
# Gradients pass the states, the state gradients and 36 sums of their chunk: sqrt(168 / 3) 2^-23 = 8.9e-7; the
# header's statement is about 1e-6 of the output's size.
LIMIT_GRAD = 1e-6


def norm_error(got, want, size=None):
    got = got.detach().cpu().double().numpy() if torch.is_tensor(got) else np.asarray(got, np.float64)
    want = np.asarray(want, np.float64)
    assert got.shape == want.shape and np.isfinite(got).all()
    size = np.linalg.norm(want if size is None else size)
    return float(np.linalg.norm(got - want) / size) if size > 0 else float(np.linalg.norm(got))


def close_in_norm(got, want, what, limit=LIMIT, size=None):
    e = norm_error(got, want, size)
    assert e <= limit, f"{what}: {e:.3g} of its 2-norm"
    return e


def terms(x, n):
    """x as the sum of n bf16 numbers, each the remainder rounded to nearest; exact in float64."""
    x = np.asarray(x, np.float32)
    out = np.zeros(x.shape)
    for _ in range(n):
        t = torch.from_numpy(x).bfloat16().float().numpy()
        out += t
        x = x - t
    return out


def model(x, n=3, wide=True, C=64):
    """(o, S_T) of dense fp32 inputs by chunks: operands cut into n bf16 terms, every product rounded to fp32, the
    products of decays formed in float64 (wide) or one fp32 rounding after another."""
    f32 = lambda a: np.asarray(a, np.float32)  # noqa: E731
    q, k, v = x["q"], x["k"], x["v"]
    B, T, H, dv = v.shape
    a = np.broadcast_to(x["alpha"], (B, T, H))
    o, S = np.zeros((B, T, H, dv), np.float32), np.zeros((B, H, k.shape[-1], dv), np.float32)
    for b in range(B):
        for h in range(H):
            hk = h // (H // k.shape[2])
            st = np.zeros(S.shape[2:], np.float32) if x["S0"] is None else x["S0"][b, h]
            for c in range(0, T, C):
                t = slice(c, min(c + C, T))
                ac = a[b, t, h].astype(np.float64 if wide else np.float32)
                L = len(ac)
                ratio = np.zeros((L, L), ac.dtype)
                for s in range(L):
                    ratio[s:, s] = np.multiply.accumulate(np.concatenate([np.ones(1, ac.dtype), ac[s + 1:]]))
                gamma = np.multiply.accumulate(ac)
                Q, K, V = (terms(m[b, t, i], n) for m, i in ((q, hk), (k, hk), (v, h)))
                P = terms(f32(f32(Q @ K.T) * f32(ratio)), n)
                o[b, t, h] = f32(P @ V) + f32(f32(gamma)[:, None] * f32(Q @ terms(st, n)))
                kept = f32(st * (gamma[-1] if wide else f32(gamma[-1])))
                st = f32(kept + K.T @ terms(f32(V) * f32(ratio[-1])[:, None], n))
            S[b, h] = st
    return o, S


def exact(x, cu=None):
    return oracle.forward(*[x[n] for n in ("q", "k", "v", "alpha")], x["S0"], cu)
