"""Gradients of the decayed linear attention against the float64 chain rule, and its autograd node."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from decay_util import close, dev, make, oracle, tensors
from gpu_util import seed_of

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "alpha")
# A gradient's term passes a second level of sums on top of a forward term's (see decay_util.bound): 128 channels of
# dO . v, 128 of the other contraction, 64 tokens of the decay's path sums, 66 products of their decays, and
# over at most 4 heads and the two scans (12 steps of two roundings) of one chunk.
EXTRA = 128 + 128 + 64 + 66 + 4 + 24


def check(x, dtype, cu=None, dS=True, seed=0):
    r = np.random.default_rng(seed)
    B, T, H, dv = x["v"].shape
    dk = x["q"].shape[-1]
    n = B if cu is None else len(cu) - 1
    dO = r.standard_normal((B, T, H, dv)).astype(np.float32)
    dS_T = r.standard_normal((n, H, dk, dv)).astype(np.float32) if dS else None
    t = tensors(x, dtype)
    g = drl.decay_bwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"], dO=dev(dO), dS_T=dev(dS_T),
                      cu_seqlens=None if cu is None else dev(np.asarray(cu, np.int32)))
    args = [x[m] for m in NAMES] + [dO, dS_T, x["S0"], cu]
    want, mag = oracle.backward(*args), oracle.backward(*args, magnitudes=True)
    end = T if cu is None else cu[-1]
    # a decay per head sums its tokens' gradients: a compensated sum of each thread's, then 8 joins
    extra = {"dalpha": EXTRA + (10 if x["alpha"].ndim == 1 else 0)}
    for name in ("dq", "dk", "dv", "dalpha", "dS0"):
        a, b, m = g[name], want[name], mag[name]
        if name in ("dq", "dk", "dv") or (name == "dalpha" and x["alpha"].ndim == 3):
            a, b, m = a[:, :end], b[:, :end], m[:, :end]
        close(a, b, m, T, name, extra.get(name, EXTRA))
    return g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 128), (64, 32), (128, 16), (128, 64), (128, 128), (16, 128), (64, 64)])
@pytest.mark.parametrize("decay", ["token", "signed", "head"])
def test_backward(dk, dv, dtype, decay):
    x = make(seed_of("bwd", dk, dv, dtype, decay), 2, 150, 4, 2, dk, dv, dtype, decay)
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129])
def test_backward_lengths(T, dtype):
    x = make(seed_of("bwd len", T, dtype), 1, T, 2, 1, 64, 32, dtype, "signed")
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_without_state(dtype):
    x = make(31, 2, 100, 2, 2, 64, 64, dtype, "small", s0=False)
    check(x, dtype, dS=False)


@pytest.mark.parametrize("seg", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_segments(seg, dtype, monkeypatch):
    monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("bwd seg", seg, dtype), 2, 333, 2, 1, 64, 128, dtype, "token")
    check(x, dtype)


CU = [0, 70, 70, 71, 199, 263, 263, 300]


@pytest.mark.parametrize("seg", [0, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_backward_packed(seg, dtype, decay, monkeypatch):
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("bwd packed", seg, dtype, decay), 1, 310, 6, 2, 64, 64, dtype, decay, n=len(CU) - 1)
    for n in ("q", "k", "v"):
        x[n][:, 300:] = np.nan  # rows that no sequence holds are not read
    x = dict(x)
    ref = {n: (np.nan_to_num(a) if a is not None else None) for n, a in x.items()}
    t = tensors(x, dtype)
    r = np.random.default_rng(0)
    dO, dS_T = r.standard_normal(x["v"].shape).astype(np.float32), r.standard_normal(x["S0"].shape).astype(np.float32)
    out = [torch.full(s, 7.0, device="cuda") for s in (x["q"].shape, x["k"].shape, x["v"].shape, x["alpha"].shape)]
    drl.dr_decay_bwd(t["q"], t["k"], t["v"], t["alpha"], t["S0"], dev(np.asarray(CU, np.int32)), dev(dO), dev(dS_T), *out,
                     torch.empty_like(t["S0"]))
    for a in out[:3] + ([out[3]] if decay == "token" else []):
        assert (a[:, 300:] == 7.0).all(), "rows behind the last sequence were written"
    check(ref, dtype, cu=CU)


def test_gradients_of_zero_decays_are_those_of_differences():
    # documents reset by a = 0: the decay's gradient there, against central differences of the forward in float64
    x = make(33, 1, 70, 1, 1, 16, 16, "f32", "token")
    x["alpha"][0, [0, 20, 33, 34]] = 0.0
    g = check(x, "f32", seed=5)
    r = np.random.default_rng(5)
    dO = r.standard_normal(x["v"].shape).astype(np.float32).astype(np.float64)
    dS = r.standard_normal(x["S0"].shape).astype(np.float32).astype(np.float64)

    def loss(a):
        o, S = oracle.forward(x["q"], x["k"], x["v"], a, x["S0"])
        return (o * dO).sum() + (S * dS).sum()

    for t in (0, 1, 20, 33, 34, 69):
        # the loss is linear in one token's decay: the difference has no truncation error, only float64
        # rounding, 1e-16 times the loss's terms over the step: below 1e-9
        a = x["alpha"].astype(np.float64)
        up, dn = a.copy(), a.copy()
        up[0, t, 0] += 0.25
        dn[0, t, 0] -= 0.25
        num = (loss(up) - loss(dn)) / 0.5
        got = float(g["dalpha"][0, t, 0])
        mag = oracle.backward(*[x[m] for m in NAMES], dO, dS, x["S0"], magnitudes=True)["dalpha"][0, t, 0]
        close(np.asarray([got]), np.asarray([num]), np.asarray([mag]), 70, f"token {t}", EXTRA)


def test_same_call_same_bits():
    x = make(34, 2, 400, 4, 1, 64, 64, "bf16", "head")
    a = check(x, "bf16", seed=1)
    b = check(x, "bf16", seed=1)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_views(dtype):
    B, T, H, d = 2, 140, 4, 64
    x = make(35, B, T, H, H, d, d, dtype, "token")
    t = tensors(x, dtype)
    big = torch.full((B, T + 9, 4, H, d), float("nan"), device="cuda", dtype=t["q"].dtype)
    for i, n in enumerate("qkv"):
        big[:, 4:T + 4, i] = t[n]
    v = [big[:, 4:T + 4, i] for i in range(3)]
    dO = torch.randn(B, T, H, d, device="cuda")
    a = drl.decay_bwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"], dO=dO)
    b = drl.decay_bwd(*v, t["alpha"], S0=t["S0"], dO=dO)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("packed", [False, True])
def test_autograd(packed):
    x = make(36, 1, 200, 4, 2, 64, 32, "bf16", "token", n=2 if packed else 1)
    t = tensors(x, "bf16")
    leaves = {n: a.clone().requires_grad_() for n, a in t.items()}
    cu = dev(np.asarray([0, 90, 180], np.int32)) if packed else None
    o, S = drl.decay_attention(leaves["q"], leaves["k"], leaves["v"], leaves["alpha"], leaves["S0"], cu)
    w, u = torch.randn_like(o), torch.randn_like(S)
    ((o * w).sum() + (S * u).sum()).backward()
    if packed:
        assert (o[:, 180:] == 0).all()
    g = drl.decay_bwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"], cu_seqlens=cu, dO=w, dS_T=u)
    end = 180 if packed else 200
    for n in NAMES:
        a, b = leaves[n].grad, g["d" + n].to(t[n].dtype)
        assert a.dtype == t[n].dtype and torch.equal(a[:, :end], b[:, :end]), n
        assert (a[:, end:] == 0).all(), n
    assert torch.equal(leaves["S0"].grad, g["dS0"])


def test_autograd_outputs_that_the_loss_does_not_use():
    x = make(37, 2, 70, 2, 1, 32, 32, "f32", "head")
    t = tensors(x, "f32")
    leaves = {n: a.clone().requires_grad_() for n, a in t.items()}
    o, S = drl.decay_attention(*[leaves[n] for n in NAMES], leaves["S0"])
    S.sum().backward()
    g = drl.decay_bwd(*[t[n] for n in NAMES], S0=t["S0"], dO=torch.zeros_like(o), dS_T=torch.ones_like(S))
    assert all(torch.equal(leaves[n].grad, g["d" + n]) for n in NAMES)
    (drl.decay_attention(*[t[n] for n in NAMES[:3]], leaves["alpha"])[0]).sum().backward()  # only the decay asks


def test_empty():
    x = make(38, 2, 0, 2, 2, 32, 32, "bf16", "head")
    t = tensors(x, "bf16")
    dS = torch.randn_like(t["S0"])
    g = drl.decay_bwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"], dO=torch.empty(2, 0, 2, 32, device="cuda"), dS_T=dS)
    assert torch.equal(g["dS0"], dS) and (g["dalpha"] == 0).all()
