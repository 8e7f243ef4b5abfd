"""The selective scan on the GPU against its definition in float64."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from gpu_util import seed_of
from layer_util import SCAN_IN, close, dev, i32, make_scan, oracle, scan_k, scan_slack, scan_tensors

pytestmark = pytest.mark.gpu


def check(x, dtype, cu=None, soft=True, drop=(), got=None, t=None):
    x = {k: None if k in drop else v for k, v in x.items()}
    if got is None:
        t = scan_tensors(x, dtype)
        got = drl.scan_fwd(*[t[k] for k in SCAN_IN], S0=t["S0"], cu_seqlens=None if cu is None else i32(cu), softplus=soft)
    a = [x[k] for k in SCAN_IN] + [x["S0"], cu, soft]
    (y, S), (my, mS) = oracle.scan(*a), oracle.scan(*a, magnitudes=True)
    N = x["A"].shape[1]
    end = y.shape[1] if cu is None else cu[-1]
    slack = scan_slack(dict(x, S0=x["S0"] if x["S0"] is not None else np.zeros(1), bias=x["bias"]), N, x["z"] is not None)
    close(got[0][:, :end], y[:, :end], my[:, :end], scan_k(y.shape[1], N), "y", slack)
    close(got[1], S, mS, scan_k(y.shape[1], N), "S_T", slack)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("block", ["1", "2"])  # waves along the tokens, or along the channels
@pytest.mark.parametrize("T,C,G", [(1, 1, 1), (7, 3, 3), (8, 64, 1), (9, 130, 2), (65, 65, 1), (130, 128, 2), (300, 40, 1)])
def test_rows(T, C, G, block, N, dtype, monkeypatch):
    monkeypatch.setenv("DR_SCAN_BLOCK", block)
    check(make_scan(seed_of("scan", T, C, G, N, dtype), 2, T, C, G, N, dtype), dtype)


@pytest.mark.parametrize("drop", [("D",), ("z",), ("bias",), ("S0",), ("D", "z", "bias", "S0")])
@pytest.mark.parametrize("soft", [True, False])
def test_optional_inputs(drop, soft):
    check(make_scan(seed_of("drop", drop), 2, 21, 70, 1, 16, "f32", soft=soft), "f32", soft=soft, drop=drop)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [0, 8, 40])
@pytest.mark.parametrize("N", [16, 64])
@pytest.mark.parametrize("block", ["1", "2"])
@pytest.mark.parametrize("cu", [[0, 0, 1, 3, 3, 40, 41, 90, 90], [0, 64, 72, 72, 75], [0], [0, 0]])
def test_packed(cu, block, N, seg, dtype, monkeypatch):
    monkeypatch.setenv("DR_SCAN_BLOCK", block)
    if seg:
        monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    x = make_scan(seed_of("packed", cu, N, dtype), 1, 97, 70, 2, N, dtype, n=len(cu) - 1)
    t = scan_tensors(x, dtype)
    y, S = torch.full_like(t["x"], 7.0), torch.empty_like(t["S0"])
    drl.dr_scan_fwd(*[t[k] for k in SCAN_IN], t["S0"], i32(cu), y, S)
    check(x, dtype, cu, got=(y, S))
    assert (y[:, cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [8, 16, 48])
@pytest.mark.parametrize("block", ["1", "2"])
@pytest.mark.parametrize("T", [8, 47, 48, 49, 200])
def test_segments(T, block, seg, dtype, monkeypatch):
    monkeypatch.setenv("DR_SCAN_BLOCK", block)
    monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    check(make_scan(seed_of("seg", T, seg), 2, T, 70, 1, 16, dtype), dtype)


def test_small_steps_keep_their_precision():
    # steps around 1e-6 over a long row: the state is a plain sum, to 2e-6 of itself
    x = make_scan(12, 1, 900, 64, 1, 16, "f32")
    x["bias"][:] = -13.8
    check(x, "f32")


def test_views_and_pools():
    # x and z as halves of one projection, dt, B and C split from another; states out of a pool, in place
    B, T, C, G, N = 3, 40, 72, 1, 16
    x = make_scan(5, B, T, C, G, N, "bf16", n=6)
    t = scan_tensors(x, "bf16")
    xz = torch.zeros(B, T + 3, 2 * C, dtype=torch.bfloat16, device="cuda")[:, 2:T + 2]
    low = torch.zeros(B, T, C + 8 + 2 * N, dtype=torch.bfloat16, device="cuda")
    v = dict(t, x=xz[..., :C], z=xz[..., C:], dt=low[..., :C], B=low[..., C:C + N].unflatten(-1, (1, N)), C=low[..., C + N:C + 2 * N].unflatten(-1, (1, N)))
    for k in ("x", "z", "dt", "B", "C"):
        v[k].copy_(t[k])
    pool, idx = t["S0"].clone(), [4, 17, 1]
    y, out = drl.scan_fwd(*[v[k] for k in SCAN_IN], S0=pool, state_idx=i32(idx))
    assert out is pool
    first = np.stack([x["S0"][4], np.zeros((C, N), np.float32), x["S0"][1]])
    dense = drl.scan_fwd(*[t[k] for k in SCAN_IN], S0=dev(first))
    assert torch.equal(y, dense[0]) and torch.equal(pool[[4, 1]], dense[1][[0, 2]])
    assert torch.equal(pool[[0, 2, 3, 5]], t["S0"][[0, 2, 3, 5]])
    check(dict(x, S0=first), "bf16", got=dense)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,C,G", [(16, 1, 1, 1), (16, 5, 130, 2), (32, 3, 65, 1), (64, 4, 48, 3), (16, 70, 64, 1), (16, 4099, 66, 1), (64, 2600, 40, 2)])
def test_step(N, S, C, G, dtype):
    # four tokens one by one from rows of a pool, against the definition over all of them
    T = 4
    x = make_scan(seed_of("step", N, S, C, dtype), S, T, C, G, N, dtype, n=S + 3)
    t = scan_tensors(x, dtype)
    idx = np.random.default_rng(5).permutation(S + 3)[:S]
    pool = t["S0"].clone()
    ys = []
    for k in range(T):
        one = {m: (t[m] if m in ("A", "D", "bias") else t[m][:, k]) for m in SCAN_IN}  # (views: every T-th row)
        ys.append(drl.scan_step(one["x"], one["dt"], one["A"], one["B"], one["C"], pool, D=one["D"], z=one["z"], dt_bias=one["bias"], state_idx=i32(idx)))
    check(dict(x, S0=x["S0"][idx]), dtype, got=(torch.stack(ys, 1), pool[torch.from_numpy(idx).cuda()]))
    rest = np.setdiff1d(np.arange(S + 3), idx)
    assert np.array_equal(pool.cpu().numpy()[rest], x["S0"][rest])
    before = pool.clone()
    y = drl.scan_step(*[one[m] for m in ("x", "dt", "A", "B", "C")], pool, state_idx=i32([-1] * S))
    assert not y.any() and torch.equal(pool, before)


# ------------------------------------------------------------------------------------------------ gradients
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")


def check_grad(x, dtype, cu=None, soft=True, drop=(), got=None):
    x = {k: None if k in drop else v for k, v in x.items()}
    t = scan_tensors(x, dtype)
    if got is None:
        got = drl.scan_bwd(*[t[k] for k in SCAN_IN], S0=t["S0"], cu_seqlens=None if cu is None else i32(cu), softplus=soft, dy=t["dy"], dS_T=t["dS"])
    a = [x[k] for k in SCAN_IN] + [x["S0"], cu, soft, x["dy"], x["dS"]]
    want, mag = oracle.scan_grad(*a), oracle.scan_grad(*a, magnitudes=True)
    B, T, _ = x["x"].shape
    N = x["A"].shape[1]
    end = T if cu is None else cu[-1]
    for n in NAMES:
        if {"dD": "D", "dz": "z", "ddt_bias": "bias"}.get(n) in drop:
            assert got[n] is None, n
            continue
        g, w, m = got[n], want[n], mag[n]
        if n in ("dx", "ddt", "dB", "dC", "dz"):
            g, w, m = g[:, :end], w[:, :end], m[:, :end]
        # twice a state's roundings (states and their gradients), and the sums over tokens and channels; the exponents' errors (see
        # scan_slack) of the same kind, taken against the largest magnitude
        tokens = B * T if n in ("dA", "dD", "ddt_bias") else x["x"].shape[2]
        close(g, w, m, 2 * scan_k(T, N) + tokens, n, slack=6 * 2.0 ** -23 * float(m.max() if m.size else 0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("T,C,G", [(1, 1, 1), (7, 3, 3), (8, 64, 1), (9, 130, 2), (65, 65, 1), (100, 160, 1)])
def test_gradients(T, C, G, N, dtype):
    check_grad(make_scan(seed_of("grad", T, C, G, N, dtype), 2, T, C, G, N, dtype), dtype)


@pytest.mark.parametrize("drop", [("D",), ("z",), ("bias",), ("S0",), ("dS",), ("D", "z", "bias", "S0", "dS")])
@pytest.mark.parametrize("soft", [True, False])
def test_gradients_optional_inputs(drop, soft):
    check_grad(make_scan(seed_of("dropg", drop), 2, 21, 70, 1, 16, "f32", soft=soft), "f32", soft=soft, drop=drop)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [0, 8, 40])
@pytest.mark.parametrize("N", [16, 64])
@pytest.mark.parametrize("cu", [[0, 0, 1, 3, 3, 40, 41, 90, 90], [0, 64, 72, 72, 75], [0], [0, 0]])
def test_gradients_packed(cu, N, seg, dtype, monkeypatch):
    if seg:
        monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    x = make_scan(seed_of("packedg", cu, N, dtype), 1, 97, 70, 2, N, dtype, n=len(cu) - 1)
    t = scan_tensors(x, dtype)
    like = {"dx": "x", "ddt": "dt", "dA": "A", "dB": "B", "dC": "C", "dD": "D", "dz": "z", "ddt_bias": "bias", "dS0": "S0"}
    g = {n: torch.full_like(t[like[n]], 7.0) for n in NAMES}
    drl.dr_scan_bwd(*[t[k] for k in SCAN_IN], t["S0"], i32(cu), t["dy"], t["dS"], *[g[n] for n in NAMES])
    check_grad(x, dtype, cu, got=g)
    for n in ("dx", "ddt", "dB", "dC", "dz"):
        assert (g[n][:, cu[-1]:] == 7.0).all(), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [8, 48])
@pytest.mark.parametrize("T", [8, 47, 49, 120])
def test_gradients_segments(T, seg, dtype, monkeypatch):
    monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    check_grad(make_scan(seed_of("segg", T, seg), 2, T, 70, 1, 16, dtype), dtype)


def test_gradients_through_autograd():
    x = make_scan(3, 2, 30, 40, 2, 16, "f32")
    t = scan_tensors(x, "f32")
    leaves = [t[k].requires_grad_() for k in SCAN_IN] + [t["S0"].requires_grad_()]
    y, S = drl.selective_scan(*leaves)
    ((y * t["dy"]).sum() + (S * t["dS"]).sum()).backward()
    check_grad(x, "f32", got=dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0"), (a.grad for a in leaves))))


def test_gradients_by_differences():
    # the loss moves by what the gradients say: both sides of a step of 2^-7 along a random direction evaluated by the kernel in
    # float32; third-order parts and roundings together below 2e-3 of the sum of magnitudes
    x = make_scan(8, 1, 50, 64, 1, 16, "f32")
    t = scan_tensors(x, "f32")

    def loss(ins):
        y, S = drl.scan_fwd(*ins[:8], S0=ins[8])
        return (y.double() * t["dy"].double()).sum() + (S.double() * t["dS"].double()).sum()

    ins = [t[k] for k in SCAN_IN] + [t["S0"]]
    g = drl.scan_bwd(*ins[:8], S0=ins[8], dy=t["dy"], dS_T=t["dS"])
    for i, n in enumerate(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dS0")):
        v = torch.randn(ins[i].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        h = 2.0 ** -7
        up, dn = ([a if j != i else a + s * v for j, a in enumerate(ins)] for s in (h, -h))
        num, ana = (loss(up) - loss(dn)) / (2 * h), (g[n].double() * v.double()).sum()
        assert abs(num - ana) <= 2e-3 * (g[n].double().abs() * v.double().abs()).sum(), (n, float(num), float(ana))


def test_the_same_call_gives_the_same_bits():
    t = scan_tensors(make_scan(4, 2, 300, 200, 1, 16, "bf16"), "bf16")
    run = lambda: drl.scan_bwd(*[t[k] for k in SCAN_IN], S0=t["S0"], dy=t["dy"], dS_T=t["dS"])  # noqa: E731
    a, b = run(), run()
    assert all(torch.equal(a[n], b[n]) for n in NAMES)
