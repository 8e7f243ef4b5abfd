"""The decayed linear attention's stated precision: errors against float64 in the 2-norm, small enough that a lost
bf16 term of an operand or a decay product rounded step by step would show (test_oracle_decay_precision.py)."""
import numpy as np
import pytest

import delta_rule_linear_chunked_amd as drl
from decay_norm import LIMIT_GRAD, close_in_norm, exact
from decay_util import dev, make, oracle, tensors
from gpu_util import seed_of

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "alpha")


def slow(x):
    """One decay for each head close to 1: every chunk leaves the same roundings, and a state remembers several."""
    x["alpha"][:] = 1 - 2.0 ** -9 * (1 + 0.1 * x["alpha"])
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "slow"])
@pytest.mark.parametrize("dk,dv,T,seg", [(64, 64, 300, 0), (128, 128, 1333, 0), (32, 32, 1333, 0), (32, 32, 1333, 4096), (64, 128, 1333, 256)])
def test_prefill(dk, dv, T, seg, decay, dtype, monkeypatch):
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("norm", dk, dv, T, seg, decay, dtype), 1, T, 4, 2, dk, dv, dtype, "head" if decay == "slow" else decay)
    x = slow(x) if decay == "slow" else x
    t = tensors(x, dtype)
    o, S = drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"])
    want, wS = exact(x)
    print(f"o {close_in_norm(o, want, 'o'):.2e} S_T {close_in_norm(S, wS, 'S_T'):.2e}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "signed", "head", "slow"])
@pytest.mark.parametrize("dk,dv,T", [(64, 64, 300), (128, 128, 700), (32, 64, 1333)])
def test_gradients(dk, dv, T, decay, dtype):
    x = make(seed_of("norm bwd", dk, dv, T, decay, dtype), 1, T, 4, 2, dk, dv, dtype, "head" if decay == "slow" else decay)
    x = slow(x) if decay == "slow" else x
    r = np.random.default_rng(1)
    dO = r.standard_normal(x["v"].shape).astype(np.float32)
    dS = r.standard_normal(x["S0"].shape).astype(np.float32)
    t = tensors(x, dtype)
    g = drl.decay_bwd(*[t[n] for n in NAMES], S0=t["S0"], dO=dev(dO), dS_T=dev(dS))
    want = oracle.backward(*[x[n] for n in NAMES], dO, dS, x["S0"])
    # One decay's gradient is the sum of its tokens' gradients: with |e_t| <= L |da_t| for each of them the sum is off by
    # at most sum |e_t| <= L sum |da_t|, which is what its error is held against. Against the sum itself there is
    # no bound: the tokens' gradients have both signs and cancel (here down to 1/29 of their magnitudes).
    size = {}
    if x["alpha"].ndim == 1:
        each = np.broadcast_to(x["alpha"], x["v"].shape[:3])
        size["dalpha"] = np.abs(oracle.backward(*[x[n] for n in NAMES[:3]], each, dO, dS, x["S0"])["dalpha"]).sum((0, 1))
    print(" ".join(f"{n} {close_in_norm(g[n], want[n], n, LIMIT_GRAD, size.get(n)):.2e}" for n in want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step(dtype):
    # forty tokens one by one: each rounds the state and its two terms once
    N, H, Hk, d = 5, 4, 2, 64
    x = make(seed_of("norm step", dtype), 40, N, H, Hk, d, d, dtype, "token", n=N)
    t = tensors(x, dtype)
    S, want = t["S0"].clone(), x["S0"].astype(np.float64)
    for i in range(40):
        o = drl.decay_step(*[t[n][i] for n in NAMES], S)
        want, wo = oracle.step(want, *[x[n][i] for n in NAMES])
    close_in_norm(S, want, "S")
    close_in_norm(o, wo, "o")
