"""Pins of the layer oracle: closed forms, other programs' sums, differences."""
import numpy as np
import pytest

from oracle import decay, layer


def rnd(seed):
    r = np.random.default_rng(seed)
    return lambda *s: r.standard_normal(s)


def test_conv_is_numpys():
    f = rnd(0)
    x, w, b, st = f(1, 9, 3), f(3, 4), f(3), f(1, 3, 3)
    y, last = layer.conv(x, w, b, st, act="none")
    for c in range(3):
        e = np.concatenate([st[0, :, c], x[0, :, c]])
        assert np.allclose(y[0, :, c], np.convolve(e, w[c, ::-1], "valid") + b[c], atol=1e-14)
    assert np.array_equal(last[0], x[0, -3:])


def test_conv_state_of_short_sequences():
    f = rnd(1)
    x, st = f(1, 5, 2), f(3, 3, 2)
    _, last = layer.conv(x, f(2, 4), None, st, cu=[0, 1, 1, 5])
    assert np.array_equal(last[0], np.concatenate([st[0, 1:], x[0, :1]]))
    assert np.array_equal(last[1], st[1]) and np.array_equal(last[2], x[0, 2:5])


def test_scan_with_one_decay_is_decayed_attention():
    f = rnd(2)
    T, C, N = 12, 3, 16
    a = -np.exp(f(C))
    x, dt, B, Cm = f(1, T, C), f(1, T, C), f(1, T, 1, N), f(1, T, 1, N)
    y, S = layer.scan(x, dt, np.repeat(a[:, None], N, 1), B, Cm)
    d = layer.softplus(dt)
    v = (d * x)[..., None]
    o, ST = decay.forward(np.repeat(Cm, C, 2), np.repeat(B, C, 2), v, np.exp(d * a))
    assert np.allclose(y, o[..., 0], atol=1e-13) and np.allclose(S, ST[..., 0], atol=1e-13)


def test_scan_gate_and_skip():
    f = rnd(3)
    x, z, D = f(2, 4, 3), f(2, 4, 3), f(3)
    y, S = layer.scan(x, f(2, 4, 3), -np.ones((3, 16)), np.zeros((2, 4, 1, 16)), f(2, 4, 1, 16), D, z)
    assert np.allclose(y, D * x * z / (1 + np.exp(-z)), atol=1e-14) and not S.any()


def central(fn, a, g, eps=1e-6):
    for i in np.random.default_rng(9).permutation(a.size)[:6]:
        at = np.unravel_index(i, a.shape)
        old = a[at]
        a[at] = old + eps
        up = fn()
        a[at] = old - eps
        dn = fn()
        a[at] = old
        assert abs((up - dn) / (2 * eps) - g[at]) <= 1e-7 * (1 + abs(g[at])), at


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients_by_differences(W, act):
    f = rnd(4)
    cu = [0, 1, 1, 6]
    x, w, b, st, dy, dl = f(1, 6, 2), f(2, W), f(2), f(3, W - 1, 2), f(1, 6, 2), f(3, W - 1, 2)

    def loss():
        y, last = layer.conv(x, w, b, st, cu, act)
        return (y * dy).sum() + (last * dl).sum()

    g = layer.conv_grad(x, w, b, st, cu, act, dy, dl)
    for a, n in ((x, "dx"), (w, "dweight"), (b, "dbias"), (st, "dstate")):
        central(loss, a, g[n])


@pytest.mark.parametrize("soft", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradients_by_differences(gate, soft):
    f = rnd(5)
    cu, C, N, G = [0, 2, 2, 7], 4, 16, 2
    x, dt, A, B, Cm, D, bias = f(1, 7, C), f(1, 7, C), -np.exp(0.3 * f(C, N)), f(1, 7, G, N), f(1, 7, G, N), f(C), f(C)
    if not soft:
        dt, bias = np.abs(dt), np.abs(bias)
    z, S0, dy, dS = (f(1, 7, C) if gate else None), f(3, C, N), f(1, 7, C), f(3, C, N)

    def loss():
        y, S = layer.scan(x, dt, A, B, Cm, D, z, bias, S0, cu, soft)
        return (y * dy).sum() + (S * dS).sum()

    g = layer.scan_grad(x, dt, A, B, Cm, D, z, bias, S0, cu, soft, dy, dS)
    for a, n in ((x, "dx"), (dt, "ddt"), (A, "dA"), (B, "dB"), (Cm, "dC"), (D, "dD"), (bias, "ddt_bias"), (S0, "dS0"), (z, "dz")):
        if a is not None:
            central(loss, a, g[n])


def test_norm():
    f = rnd(6)
    h, w, dy, dh = f(3, 10), f(10), f(3, 10), f(3, 10)
    assert np.allclose((layer.norm(h, np.ones(10), 0.0) ** 2).mean(-1), 1.0)

    def loss():
        return (layer.norm(h, w) * dy).sum() + (h * dh).sum()

    g = layer.norm_grad(h, w, dy, dh)
    central(loss, h, g["dx"])
    central(loss, w, g["dweight"])


@pytest.mark.parametrize("fmt,far", [("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)])
def test_norm_in_8_bits(fmt, far):
    # int8: half a step of the row's largest; e4m3: half a step of each value, or of the least step of the scale
    f = rnd(7)
    h, w = f(4, 33).astype(np.float32), f(33).astype(np.float32)
    y, (v, s) = layer.norm(h, w), layer.norm(h, w, fmt=fmt)
    room = far * np.abs(y).max(-1, keepdims=True) if fmt == "int8" else np.maximum(far * np.abs(y), 2.0 ** -10 * s[:, None])
    assert (np.abs(v - y) <= room * (1 + 1e-6)).all()
