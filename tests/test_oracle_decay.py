"""Pins of the decayed linear attention's oracle and of the cache's definition, and the error bound of their GPU tests."""
import numpy as np
import pytest
import torch

import oracle as rules
from decay_util import bound, make
from oracle import decay as oracle

NAMES = ("q", "k", "v", "alpha")


def test_no_decay_is_a_prefix_sum_and_full_decay_forgets():
    x = make(1, 1, 9, 2, 1, 4, 3, "f32", s0=False)
    q, k, v = (x[n].astype(np.float64) for n in "qkv")
    one, zero = np.ones((1, 9, 2)), np.zeros((1, 9, 2))
    o, S = oracle.forward(q, k, v, one)
    for h in range(2):
        for t in range(9):
            want = sum((q[0, t, 0] @ k[0, s, 0]) * v[0, s, h] for s in range(t + 1))
            assert np.allclose(o[0, t, h], want, rtol=1e-13, atol=1e-13)
        assert np.allclose(S[0, h], k[0, :, 0].T @ v[0, :, h], rtol=1e-13, atol=1e-13)
    o, S = oracle.forward(q, k, v, zero, S0=np.ones((1, 2, 4, 3)))
    assert np.allclose(o[0, :, 1], (q[0, :, 0] * k[0, :, 0]).sum(-1)[:, None] * v[0, :, 1], rtol=1e-13, atol=1e-13)


def test_constant_decay_is_a_weighted_sum():
    x = make(2, 1, 12, 2, 2, 4, 4, "f32", "head")
    o, S = oracle.forward(*[x[n] for n in NAMES], x["S0"])
    q, k, v, a = (x[n].astype(np.float64) for n in NAMES)
    for h in range(2):
        t = 11
        w = a[h] ** (t - np.arange(12))
        want = q[0, t, h] @ (a[h] ** 12 * x["S0"][0, h].astype(np.float64) + (w[:, None] * k[0, :, h]).T @ v[0, :, h])
        assert np.allclose(o[0, t, h], want, rtol=1e-12, atol=1e-13)


def test_is_the_gated_delta_rule_without_erasing():
    # RDA's rule with e = 0, w = 1 and one decay for all channels
    x = make(3, 2, 20, 2, 2, 8, 8, "f32", "signed")
    a = np.repeat(x["alpha"][..., None], 8, -1)
    zero, one = np.zeros((2, 20, 2)), np.ones((2, 20, 2))
    want, wS = rules.step_recurrence(x["q"], x["k"], x["v"], a, zero, one, "rda", S0=x["S0"])
    o, S = oracle.forward(*[x[n] for n in NAMES], x["S0"])
    assert np.allclose(o, want, rtol=1e-13, atol=1e-13) and np.allclose(S, wS, rtol=1e-13, atol=1e-13)


def test_packed_sequences_and_steps():
    x = make(4, 1, 30, 4, 2, 4, 4, "f32", n=3)
    cu = [0, 11, 11, 28]
    o, S = oracle.forward(*[x[n] for n in NAMES], x["S0"], cu)
    for n in (0, 2):
        part = [x[m][:, cu[n]:cu[n + 1]] for m in NAMES]
        o1, S1 = oracle.forward(*part, x["S0"][n:n + 1])
        assert np.array_equal(o[:, cu[n]:cu[n + 1]], o1) and np.array_equal(S[n], S1[0])
    assert np.array_equal(S[1], x["S0"][1].astype(np.float64)) and (o[:, 28:] == 0).all()
    state = x["S0"][:1]
    for t in range(11):
        state, o1 = oracle.step(state, *[x[m][:, t] for m in NAMES])
        assert np.allclose(o1[0], o[0, t], rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("decay", ["token", "signed", "head"])
@pytest.mark.parametrize("cu", [None, [0, 5, 5, 9]])
def test_gradients_are_those_of_central_differences(decay, cu):
    n = 1 if cu is None else 3
    x = make(5, 1, 10, 4, 2, 3, 2, "f32", decay, n=n)
    r = np.random.default_rng(6)
    dO, dS = r.standard_normal(x["v"].shape), r.standard_normal(x["S0"].shape)
    args = [x[m].astype(np.float64) for m in NAMES] + [x["S0"].astype(np.float64)]
    end = 10 if cu is None else cu[-1]

    def loss(a):
        o, S = oracle.forward(*a, cu)
        return (o[:, :end] * dO[:, :end]).sum() + (S * dS).sum()

    g = oracle.backward(*args[:4], dO, dS, args[4], cu)
    for i, name in enumerate(("dq", "dk", "dv", "dalpha", "dS0")):
        flat = args[i].reshape(-1)
        for j in r.choice(flat.size, min(12, flat.size), replace=False):
            # a cubic at most in one decay shared by tokens... a polynomial in the entry: a step of 1e-4 leaves a
            # truncation of 1e-8 times its third derivative, and 1e-16 / 1e-4 of rounding
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i].reshape(-1)[j] += 1e-4
            dn[i].reshape(-1)[j] -= 1e-4
            num, got = (loss(up) - loss(dn)) / 2e-4, g[name].reshape(-1)[j]
            assert abs(num - got) <= 1e-5 * (1 + abs(num)), (name, j, num, got)


def test_magnitudes_bound_the_results():
    x = make(7, 1, 20, 2, 1, 4, 4, "f32", "signed")
    a = [x[n] for n in NAMES]
    assert (np.abs(oracle.forward(*a, x["S0"])[0]) <= oracle.forward(*a, x["S0"], magnitudes=True)[0] * (1 + 1e-12)).all()


@pytest.mark.parametrize("mistake", ["late decay", "missing token", "wrong head", "bf16 scores", "dropped state"])
def test_the_bound_catches_mistakes(mistake):
    # evaluations with one planted mistake leave the bound that the GPU tests hold the kernels to
    x = make(8, 1, 150, 2, 2, 64, 64, "f32", "token")
    q, k, v, a = (x[n].astype(np.float64) for n in NAMES)
    want, _ = oracle.forward(q, k, v, a, x["S0"])
    mag, _ = oracle.forward(q, k, v, a, x["S0"], magnitudes=True)
    S0 = x["S0"]
    if mistake == "late decay":
        a = np.roll(a, 1, axis=1)
    elif mistake == "missing token":
        v = v.copy()
        v[:, 70] = 0
    elif mistake == "wrong head":
        k = k[:, :, ::-1]
    elif mistake == "dropped state":
        S0 = None
    got, _ = oracle.forward(q, k, v, a, S0)
    if mistake == "bf16 scores":
        got = np.zeros_like(want)
        for h in range(2):
            c = np.cumprod(a[0, :, h])
            P = (q[0, :, h] @ k[0, :, h].T) * np.tril(c[:, None] / c[None, :])
            P = torch.from_numpy(P).bfloat16().double().numpy()
            got[0, :, h] = P @ v[0, :, h] + c[:, None] * (q[0, :, h] @ S0[0, h])
    assert (np.abs(got - want) > bound(mag, 150)).any()


# ------------------------------------------------------------------------------------------------ cache
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_cache_values(fmt):
    r = np.random.default_rng(9)
    S = (r.standard_normal((3, 2, 16, 32)) * np.exp(3 * r.standard_normal((3, 2, 16, 1)))).astype(np.float32)
    held, scale = oracle.pack(S, fmt)
    codes = held / scale[..., None]
    top = np.abs(S).max(-1)
    if fmt == "int8":
        assert np.array_equal(codes, np.rint(codes)) and np.abs(codes).max() <= 127
        assert (np.abs(codes).max(-1) == 127).all()
        assert (np.abs(held - S) <= scale[..., None] / 2 * (1 + 1e-12)).all()
    else:
        # torch's own conversion of the exact quotients, and a scale that half of itself would not do
        exact = torch.from_numpy((S / scale[..., None]).astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(codes, exact)
        assert (np.log2(scale) == np.rint(np.log2(scale))).all()
        assert (top <= 448 * scale).all() and (top > 448 * scale / 2).all()


def test_cache_borders():
    z = np.zeros((1, 1, 1, 16), np.float32)
    assert oracle.pack(z, "int8")[1].item() == 2.0 ** -126 and (oracle.pack(z, "e4m3")[0] == 0).all()
    z[..., 3] = np.inf
    for fmt in ("int8", "e4m3"):
        held, scale = oracle.pack(z, fmt)
        assert np.isnan(held).all() and np.isnan(scale).all()
    half = np.zeros((1, 1, 1, 16), np.float32)
    half[0, 0, 0, :5] = [127, 0.5, 1.5, -0.5, -2.5]
    assert oracle.pack(half, "int8")[0][0, 0, 0, :5].tolist() == [127, 0, 2, 0, -2]  # ties to even
