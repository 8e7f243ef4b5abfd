"""Inputs, oracle calls and error bounds of the decayed linear attention's tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import decay as oracle

# One rounding of a float32 accumulation. A matrix core may cut a sum instead of rounding it: a whole unit
# in the last place, 2^-23, instead of half of one.
ULP = 2.0 ** -23


def bound(magnitude, T, extra=0):
    """Largest error of a result whose terms' magnitudes sum to ``magnitude``. A term of a chunked evaluation meets at
    most: 63 products of decays in its chunk and 3 across tiles; the cut of each operand into three bf16 terms
    (2^-24, dropped products of the smallest terms 3 2^-24); a sum of 128 channels, twice (scores, then
    tokens: 64), and for every chunk it crosses one product with the chunk's decay (itself 63 roundings),
    64 sums into the state and one join of segments. Each is at most one ULP of that term."""
    per_chunk = 63 + 1 + 64 + 2
    once = 63 + 3 + 4 + 128 + 128 + 64
    return (once + per_chunk * (T // 64 + 1) + extra) * ULP * magnitude + 1e-37


def make(seed, B, T, H, Hk, dk, dv, dtype="bf16", decay="token", n=None, s0=True):
    """Float32 numpy inputs (bf16 data already rounded): q, k of unit length, v normal, decays by kind:
    token exp(-0.1 softplus), signed tanh with exact zeros and ones, head one per head, small 1e-6..1."""
    r = np.random.default_rng(seed)
    unit = lambda *s: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(r.standard_normal(s))  # noqa: E731
    x = dict(q=unit(B, T, Hk, dk), k=unit(B, T, Hk, dk), v=r.standard_normal((B, T, H, dv)))
    x = {name: a.astype(np.float32) for name, a in x.items()}
    if dtype == "bf16":
        x = {name: torch.from_numpy(a).bfloat16().float().numpy() for name, a in x.items()}
    z = r.standard_normal((B, T, H))
    if decay == "head":
        a = 1 - 2.0 ** (-5 - 4 * r.random(H))
    elif decay == "signed":
        a = np.tanh(1.5 * z)
        u = r.random(z.shape)
        a = np.where(u < 0.1, np.sign(z), np.where(u > 0.95, 0.0, a))
    elif decay == "small":
        a = 10.0 ** (-6 * r.random(z.shape))
    else:
        a = np.exp(-0.1 * np.log1p(np.exp(z)))
    x["alpha"] = a.astype(np.float32)
    n = B if n is None else n
    x["S0"] = (r.standard_normal((n, H, dk, dv)) / np.sqrt(dk)).astype(np.float32) if s0 else None
    return x


def dev(x, dtype=None):
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.bfloat16() if dtype == "bf16" else t


def tensors(x, dtype):
    return {name: dev(a, dtype if name in ("q", "k", "v") else None) for name, a in x.items()}


def close(got, want, magnitude, T, what, extra=0):
    got = got.detach().cpu().double().numpy() if torch.is_tensor(got) else got
    err, lim = np.abs(got - want), bound(magnitude, T, extra)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float((err / lim).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound (largest {err.max():.3g})"
    return worst
