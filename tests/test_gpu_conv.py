"""The short causal convolution on the GPU against its definition in float64."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from gpu_util import seed_of
from layer_util import CONV_K, close, dev, i32, make_conv, oracle

pytestmark = pytest.mark.gpu


def check_fwd(x, dtype, cu, act, state=True, bias=True, got=None):
    st, b = (x["state"] if state else None), (x["b"] if bias else None)
    if got is None:
        got = drl.conv_fwd(dev(x["x"], dtype), dev(x["w"]), dev(b), dev(st, dtype), None if cu is None else i32(cu), act)
    want, last = oracle.conv(x["x"], x["w"], b, st, cu, act)
    mag, _ = oracle.conv(x["x"], x["w"], b, st, cu, act, magnitudes=True)
    end = x["x"].shape[1] if cu is None else cu[-1]
    close(got[0][:, :end], want[:, :end], mag[:, :end], CONV_K, "y")
    assert np.array_equal(got[1].float().cpu().numpy(), last), "state"


def check_bwd(x, dtype, cu, act, state=True, bias=True, got=None):
    st, b = (x["state"] if state else None), (x["b"] if bias else None)
    if got is None:
        got = drl.conv_bwd(dev(x["x"], dtype), dev(x["w"]), dev(b), dev(st, dtype), None if cu is None else i32(cu), act,
                           dev(x["dy"], dtype), dev(x["dl"], dtype))
    a = (x["x"], x["w"], b, st, cu, act, x["dy"], x["dl"])
    want, mag = oracle.conv_grad(*a), oracle.conv_grad(*a, magnitudes=True)
    B, T, _ = x["x"].shape
    end = T if cu is None else cu[-1]
    close(got["dx"][:, :end], want["dx"][:, :end], mag["dx"][:, :end], CONV_K, "dx")
    close(got["dweight"], want["dweight"], mag["dweight"], CONV_K + B * T, "dweight")
    for n, given in (("dbias", bias), ("dstate", state)):
        if given:
            close(got[n], want[n], mag[n], CONV_K + B * T, n)
        else:
            assert got[n] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 33, 130])
@pytest.mark.parametrize("C", [1, 130, 256, 520])
def test_rows(C, T, W, dtype):
    x = make_conv(seed_of("conv", C, T, W, dtype), 2, T, C, W, dtype)
    act = ("silu", "none")[T % 2]
    check_fwd(x, dtype, None, act, state=T != 9, bias=T != 8)
    check_bwd(x, dtype, None, act, state=T != 9, bias=T != 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [65, 512])
@pytest.mark.parametrize("cu", [[0, 0, 1, 3, 3, 40, 41, 43, 43], [0, 64, 72, 72, 75], [0, 5], [0], [0, 0], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]])
def test_packed(cu, C, dtype):
    # empty sequences, sequences shorter than the window, ends inside a run; rows past the last sequence stay as they were
    T = 80
    x = make_conv(seed_of("packed", cu, C, dtype), 1, T, C, 4, dtype, n=len(cu) - 1)
    xd, st, off = dev(x["x"], dtype), dev(x["state"], dtype), i32(cu)
    y, last = torch.full_like(xd, 7.0), torch.empty_like(st)
    drl.dr_conv_fwd(xd, dev(x["w"]), dev(x["b"]), st, off, y, last)
    check_fwd(x, dtype, cu, "silu", got=(y, last))
    assert (y[:, cu[-1]:] == 7.0).all()
    g = dict(dx=torch.full_like(xd, 7.0), dweight=torch.full((C, 4), 7.0, device="cuda"), dbias=torch.full((C,), 7.0, device="cuda"), dstate=torch.empty_like(st))
    drl.dr_conv_bwd(xd, dev(x["w"]), dev(x["b"]), st, off, dev(x["dy"], dtype), dev(x["dl"], dtype), g["dx"], g["dweight"], g["dbias"], g["dstate"])
    check_bwd(x, dtype, cu, "silu", got=g)
    assert (g["dx"][:, cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [3, 512])
def test_views_and_pools(C, dtype):
    # a slice of a fused projection along both axes, states out of a pool, in place; a slot outside the pool starts at zero and
    # stores nothing, rows nobody names stay
    B, T, W = 3, 40, 4
    x = make_conv(seed_of("views", C, dtype), B, T, C, W, dtype, n=6)
    wide = torch.zeros(B, T + 8, 3 * C, dtype=dev(x["x"], dtype).dtype, device="cuda")
    view = wide[:, 4:T + 4, C:2 * C]
    view.copy_(dev(x["x"], dtype))
    pool = dev(x["state"], dtype)
    idx = [4, 17, 1]
    y, out = drl.conv_fwd(view, dev(x["w"]), dev(x["b"]), pool, state_idx=i32(idx))
    assert out is pool
    st = np.stack([x["state"][4], np.zeros((W - 1, C), np.float32), x["state"][1]])
    want, last = oracle.conv(x["x"], x["w"], x["b"], st)
    mag, _ = oracle.conv(x["x"], x["w"], x["b"], st, magnitudes=True)
    close(y, want, mag, CONV_K, "y")
    now = pool.float().cpu().numpy()
    assert np.array_equal(now[[4, 1]], last[[0, 2]]) and np.array_equal(now[[0, 2, 3, 5]], x["state"][[0, 2, 3, 5]])
    x["state"] = x["state"][:3]
    x["dl"] = x["dl"][:3]
    g = drl.conv_bwd(view, dev(x["w"]), dev(x["b"]), dev(x["state"], dtype), dy=dev(x["dy"], dtype), dstate_T=dev(x["dl"], dtype))
    check_bwd(x, dtype, None, "silu", got=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,C,W", [(1, 1, 2), (1, 512, 4), (5, 130, 3), (9, 264, 4), (70, 256, 4), (4099, 66, 4), (8195, 258, 3)])
def test_step(N, C, W, dtype):
    # tokens one by one equal the convolution of all of them, bit for bit; unnamed rows stay
    T = 6
    x = make_conv(seed_of("step", N, C, W, dtype), N, T, C, W, dtype, n=N + 3)
    xd, w, b = dev(x["x"], dtype), dev(x["w"]), dev(x["b"])
    idx = np.random.default_rng(5).permutation(N + 3)[:N]
    pool = dev(x["state"], dtype)
    first = pool[torch.from_numpy(idx).cuda()].clone()
    y, last = drl.conv_fwd(xd, w, b, first)
    wide = torch.zeros(N, 2 * C, dtype=xd.dtype, device="cuda")
    for t in range(T):
        wide[:, C:] = xd[:, t]
        got = drl.conv_step(wide[:, C:], w, pool, b, state_idx=i32(idx))
        assert torch.equal(got, y[:, t]), t
    assert torch.equal(pool[torch.from_numpy(idx).cuda()], last)
    rest = np.setdiff1d(np.arange(N + 3), idx)
    assert np.array_equal(pool.float().cpu().numpy()[rest], x["state"][rest])
    out = drl.conv_step(xd[:, 0].contiguous(), w, pool, b, state_idx=i32([N + 3] * N))
    assert not out.any()


def test_gradients_through_autograd():
    x = make_conv(3, 2, 30, 40, 4, "f32")
    leaves = [dev(x[k]).requires_grad_() for k in ("x", "w", "b", "state")]
    y, last = drl.causal_conv(*leaves)
    ((y * dev(x["dy"])).sum() + (last * dev(x["dl"])).sum()).backward()
    check_bwd(x, "f32", None, "silu", got=dict(zip(("dx", "dweight", "dbias", "dstate"), (t.grad for t in leaves))))
    # one output unused, and no state
    a, w = dev(x["x"]).requires_grad_(), dev(x["w"]).requires_grad_()
    drl.causal_conv(a, w)[0].sum().backward()
    b, v = dev(x["x"]).requires_grad_(), dev(x["w"]).requires_grad_()
    drl.causal_conv(b, v)[1].sum().backward()
    assert (b.grad[:, -3:] == 1).all() and not b.grad[:, :-3].any() and not v.grad.any()


def test_gradients_by_differences():
    # the loss moves by what the gradients say: a step of 2^-6 along a random direction, both sides evaluated by the
    # kernel in float32, the difference's third-order part below 1e-4 of it and its roundings below 4e-4
    x = make_conv(8, 1, 50, 64, 4, "f32")
    t = {k: dev(v) for k, v in x.items()}
    loss = lambda a, w, b, s: (lambda o: (o[0].double() * t["dy"].double()).sum() + (o[1].double() * t["dl"].double()).sum())(  # noqa: E731
        drl.conv_fwd(a, w, b, s))
    g = drl.conv_bwd(t["x"], t["w"], t["b"], t["state"], dy=t["dy"], dstate_T=t["dl"])
    ins = [t[k] for k in ("x", "w", "b", "state")]
    for i, name in enumerate(("dx", "dweight", "dbias", "dstate")):
        v = torch.randn(ins[i].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        h = 2.0 ** -6
        up, dn = ([a if j != i else a + s * v for j, a in enumerate(ins)] for s in (h, -h))
        num, ana = (loss(*up) - loss(*dn)) / (2 * h), (g[name].double() * v.double()).sum()
        scale = (g[name].double().abs() * v.double().abs()).sum()
        assert abs(num - ana) <= 1e-3 * scale, (name, float(num), float(ana))
