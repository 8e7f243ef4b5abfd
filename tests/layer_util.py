"""Inputs, oracle calls and error bounds of the convolution's, the scan's and the norm's tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import layer as oracle

ULP = 2.0 ** -23  # one unit in the last place of a float32: a rounding is half of it, the hardware's exp2, rcp and rsq one
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def held(a, dtype):
    """float32 numpy values that a tensor of the type holds."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(TYPES[dtype]).float().numpy()


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", TYPES[dtype])


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def close(got, want, mag, k, what, slack=0.0):
    """|got - want| <= k ULP of the magnitudes (and ``slack``), and half a step of a bf16 output."""
    half = 2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0.0
    g = got.detach().float().cpu().numpy().astype(np.float64)
    assert g.shape == want.shape, f"{what}: shape {g.shape}, expected {want.shape}"
    assert np.isfinite(g).all(), f"{what}: not finite"
    lim = (1 + 2.0 ** -8) * (k * ULP * mag + slack) + half + 1e-37
    err = np.abs(g - want)
    worst = float((err / lim).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound (largest {err.max():.3g})"
    if got.dtype == torch.float32 and err.size and np.linalg.norm(want) > 0:
        rel = float(np.linalg.norm(err) / np.linalg.norm(want))
        # the statement of the header, where no output is the small difference of large sums
        assert rel <= 2e-6 * max(1.0, float(np.linalg.norm(mag) / np.linalg.norm(want)) / 4), f"{what}: 2-norm error {rel:.3g}"


# ------------------------------------------------------------------------------------------------ convolution
def make_conv(seed, B, T, C, W, dtype, n=None):
    r = np.random.default_rng(seed)
    n = B if n is None else n
    f = lambda *s: held(r.standard_normal(s), dtype)  # noqa: E731
    return dict(x=f(B, T, C), w=(r.standard_normal((C, W)) / np.sqrt(W)).astype(np.float32), b=(0.2 * r.standard_normal(C)).astype(np.float32),
                state=f(n, W - 1, C), dy=f(B, T, C), dl=f(n, W - 1, C))


CONV_K = 20  # width + 1 products and sums, sigmoid's exponent (its derivative times its size: 0.3 of an ULP of the sum), exp2, rcp, two products


# ------------------------------------------------------------------------------------------------ selective scan
def make_scan(seed, B, T, C, G, N, dtype, n=None, soft=True):
    r = np.random.default_rng(seed)
    n = B if n is None else n
    f = lambda *s: held(r.standard_normal(s), dtype)  # noqa: E731
    step = np.exp(r.random(C) * np.log(100.0) + np.log(1e-3))
    x = dict(x=f(B, T, C), dt=held(0.5 * r.standard_normal((B, T, C)), dtype), A=-(np.arange(1, N + 1) * np.exp(0.1 * r.standard_normal((C, N)))).astype(np.float32),
             B=f(B, T, G, N), C=f(B, T, G, N), D=(1 + 0.1 * r.standard_normal(C)).astype(np.float32), z=f(B, T, C),
             bias=(step + np.log(-np.expm1(-step))).astype(np.float32), S0=r.standard_normal((n, C, N)).astype(np.float32),
             dy=f(B, T, C), dS=r.standard_normal((n, C, N)).astype(np.float32))
    if not soft:  # steps given as they are
        x["dt"], x["bias"] = held(0.02 + 0.1 * r.random((B, T, C)), dtype), (0.01 * r.random(C)).astype(np.float32)
    return x


SCAN_IN = ("x", "dt", "A", "B", "C", "D", "z", "bias")


def scan_tensors(x, dtype):
    return {k: dev(v, dtype if k in ("x", "dt", "B", "C", "z", "dy") else "f32") for k, v in x.items()}


def scan_k(L, N):
    """ULPs of a term of the scan (and of its gradients): per token crossed the exponential's own error and argument's rounding, a product and
    a sum (4); its step d about 8 (exp2, rcp, seven terms), the sum over N states, joins and gates."""
    return 4 * L + N + 96


def scan_slack(x, N, gate):
    """An error of d (8 ULPs at most) also moves the exponents: e^-X by X e^-X times that, X e^-X <= 0.37, of a term as it was when it
    entered: 3 ULPs of the largest term there is, for each that an output sums."""
    top = lambda a: float(np.abs(a).max()) if a is not None and a.size else 0.0  # noqa: E731
    raw, d = oracle._steps(x["dt"], x["bias"], True)
    enter = max(top(x["S0"]), top(d) * top(x["x"]) * top(x["B"]))
    return 3 * ULP * enter * (N * top(x["C"]) * (top(x["z"]) if gate else 1.0))
