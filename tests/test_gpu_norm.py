"""The norm with residual and 8-bit output on the GPU against its definition in float64."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from gpu_util import seed_of
from layer_util import TYPES, close, dev, held, oracle

pytestmark = pytest.mark.gpu
# the sum of squares: 32 products a lane, 10 steps across lanes and waves, halved by the root; mean, rsq, two products
NORM_K = 32


def make(seed, R, C, dtype):
    r = np.random.default_rng(seed)
    f = lambda s=1.0: held(s * r.standard_normal((R, C)), dtype)  # noqa: E731
    x = dict(x=f(), r=f(3.0), w=(1 + 0.3 * r.standard_normal(C)).astype(np.float32), dy=f(), dh=f())
    # the sum in the type of x: in float32 first
    x["h"] = held(x["x"] + x["r"], dtype)
    return x


SIZES = [(1, 1), (3, 7), (5, 64), (2, 1531), (9, 2048), (2, 2056), (3, 8192), (2, 8200), (2, 32768), (1, 30001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", SIZES)
def test_values(R, C, dtype):
    x = make(seed_of("norm", R, C, dtype), R, C, dtype)
    y, h = drl.norm_fwd(dev(x["x"], dtype), dev(x["w"]), dev(x["r"], dtype))
    assert torch.equal(h, dev(x["h"], dtype))
    want = oracle.norm(x["h"], x["w"])
    close(y, want, np.abs(want), NORM_K, "y")
    alone = dev(x["x"], dtype)
    y, h = drl.norm_fwd(alone, dev(x["w"]), eps=0.5)
    assert h is alone
    want = oracle.norm(x["x"], x["w"], 0.5)
    close(y, want, np.abs(want), NORM_K, "y without residual")


def check_codes(got, h, w, fmt):
    codes, scales = got[0], got[1]
    values, want = oracle.norm(h, w, fmt=fmt)
    exact = values / want[:, None]
    assert np.array_equal(codes.float().cpu().numpy(), np.rint(exact) if fmt == "int8" else held(exact, "f32")), "codes"
    close(scales, want, np.abs(want), NORM_K, "scales")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("R,C", SIZES)
def test_codes(R, C, fmt, dtype):
    x = make(seed_of("codes", R, C, dtype), R, C, dtype)
    got = drl.norm_fwd(dev(x["x"], dtype), dev(x["w"]), dev(x["r"], dtype), fmt=fmt)
    check_codes(got, x["h"], x["w"], fmt)
    assert torch.equal(got[2], dev(x["h"], dtype))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_at_ties(fmt):
    # rows whose products lie on and next to halves of the code's steps
    k = np.arange(-127, 127, dtype=np.float32)
    rows = []
    for s in (1.0, 0.75, 3.0, 1.1, 2.0 ** -40, 2.0 ** 30):
        half = (k + np.float32(0.5)) * np.float32(s)
        for y in (half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf))):
            rows.append(np.concatenate([y, [np.float32(127) * np.float32(s), -np.float32(127) * np.float32(s)]]))
    rows += [np.linspace(-448, 448, 256), np.linspace(-1, 1, 256) ** 5, np.zeros(256), np.eye(256)[3] * 449]
    h = np.stack([np.asarray(r, np.float32) for r in rows])
    w = np.ones(256, np.float32)
    check_codes(drl.norm_fwd(dev(h), dev(w), fmt=fmt), h, w, fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_with_nan_or_infinity(fmt):
    h = np.random.default_rng(1).standard_normal((4, 64)).astype(np.float32)
    h[1, 5], h[2, 9] = np.nan, np.inf
    codes, scales, _ = drl.norm_fwd(dev(h), dev(np.ones(64, np.float32)), fmt=fmt)
    assert not codes[1:3].float().any() and scales[1:3].isnan().all() and scales[[0, 3]].isfinite().all()
    y, _ = drl.norm_fwd(dev(h), dev(np.ones(64, np.float32)))
    assert y[1].isnan().all() and y[[0, 3]].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 71])
def test_views_and_places(C, dtype):
    # rows of a wider tensor, three leading dimensions; the sum written over x and over the residual
    x = make(seed_of("views", C, dtype), 12, C, dtype)
    wide = torch.zeros(3, 4, 2 * C, dtype=TYPES[dtype], device="cuda")
    v = wide[..., C:]
    v.copy_(dev(x["x"], dtype).view(3, 4, C))
    want, h = drl.norm_fwd(dev(x["x"], dtype), dev(x["w"]), dev(x["r"], dtype))
    got, h2 = drl.norm_fwd(v, dev(x["w"]), dev(x["r"], dtype).view(3, 4, C))
    assert torch.equal(got.view(12, C), want) and torch.equal(h2.view(12, C), h)
    for place in ("x", "r"):
        t = {k: dev(x[k], dtype) for k in ("x", "r")}
        y = torch.empty_like(t["x"])
        drl.dr_norm_fwd(t["x"], t["r"], dev(x["w"]), y, None, t[place])
        assert torch.equal(t[place], h) and torch.equal(y, want)
    some = wide[:, 1:3, C:]
    with pytest.raises(ValueError):
        drl.norm_fwd(some, dev(x["w"]))


def check_bwd(x, dtype, dh=True, got=None):
    h, dh = x["h"], (x["dh"] if dh else None)
    if got is None:
        got = drl.norm_bwd(dev(h, dtype), dev(x["w"]), dev(x["dy"], dtype), dev(dh, dtype))
    want = oracle.norm_grad(h, x["w"], x["dy"], dh)
    h64 = h.astype(np.float64)
    r = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + 1e-5)
    wd = np.abs(x["w"] * x["dy"].astype(np.float64))
    mx = r * (wd + np.abs(h64) * r * r * (wd * np.abs(h64)).mean(-1, keepdims=True)) + (0 if dh is None else np.abs(dh))
    close(got["dx"], want["dx"], mx, 4 * NORM_K, "dx")
    close(got["dweight"], want["dweight"], np.abs(x["dy"] * h64 * r).sum(0), NORM_K + h.shape[0], "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", SIZES + [(700, 40), (2100, 72)])
def test_gradients(R, C, dtype):
    x = make(seed_of("grad", R, C, dtype), R, C, dtype)
    check_bwd(x, dtype)
    check_bwd(x, dtype, dh=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(257, 520), (257, 2047), (300, 2048), (257, 2056), (260, 8192)])
def test_more_rows_than_few(R, C, dtype):
    # (smaller calls of these widths give a row to more waves; below 2049 channels the forward pass does up to 8192 rows)
    x = make(seed_of("many", R, C, dtype), R, C, dtype)
    check_bwd(x, dtype)
    R = 8193 if C <= 2048 else R
    x = make(seed_of("many rows", R, C, dtype), R, C, dtype)
    y, h = drl.norm_fwd(dev(x["x"], dtype), dev(x["w"]), dev(x["r"], dtype))
    want = oracle.norm(x["h"], x["w"])
    close(y, want, np.abs(want), NORM_K, "y")
    assert torch.equal(h, dev(x["h"], dtype))
    for fmt in ("int8", "e4m3"):
        check_codes(drl.norm_fwd(h, dev(x["w"]), fmt=fmt), x["h"], x["w"], fmt)


def test_gradients_in_place_and_of_nothing():
    x = make(2, 33, 64, "bf16")
    dh, dw = dev(x["dh"], "bf16"), torch.empty(64, device="cuda")
    drl.dr_norm_bwd(dev(x["h"], "bf16"), dev(x["w"]), dev(x["dy"], "bf16"), dh, dh, dw)
    check_bwd(x, "bf16", got=dict(dx=dh, dweight=dw))
    none = torch.empty(0, 64, device="cuda")
    g = drl.norm_bwd(none, dev(x["w"]), none)
    assert g["dx"].shape == (0, 64) and not g["dweight"].any()
    y, h = drl.norm_fwd(none, dev(x["w"]), none)
    assert y.shape == h.shape == (0, 64)


def test_gradients_through_autograd():
    x = make(3, 40, 96, "f32")
    t = {k: dev(v) for k, v in x.items()}
    a, r, w = (t[k].requires_grad_() for k in ("x", "r", "w"))
    y, h = drl.rms_norm(a, w, r)
    ((y * t["dy"]).sum() + (h * t["dh"]).sum()).backward()
    check_bwd(x, "f32", got=dict(dx=a.grad, dweight=w.grad))
    assert torch.equal(a.grad, r.grad) and a.grad.data_ptr() != r.grad.data_ptr()
    a, w = dev(x["h"]).requires_grad_(), dev(x["w"]).requires_grad_()
    (drl.rms_norm(a, w) * t["dy"]).sum().backward()
    check_bwd(x, "f32", dh=False, got=dict(dx=a.grad, dweight=w.grad))
    a, r, w = (dev(x[k]).requires_grad_() for k in ("x", "r", "w"))
    drl.rms_norm(a, w, r)[1].sum().backward()  # only the sum used
    assert (a.grad == 1).all() and (r.grad == 1).all() and not w.grad.any()


def test_gradients_by_differences():
    x = make(5, 20, 64, "f32")
    t = {k: dev(v) for k, v in x.items()}
    g = drl.norm_bwd(t["h"], t["w"], t["dy"])
    for i, n in enumerate(("dx", "dweight")):
        v = torch.randn((20, 64)[i:], device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        s = 2.0 ** -6
        f = lambda k: (drl.norm_fwd(t["h"] + (k * v if i == 0 else 0), t["w"] + (k * v if i else 0))[0].double() * t["dy"].double()).sum()  # noqa: E731
        num, ana = (f(s) - f(-s)) / (2 * s), (g[n].double() * v.double()).sum()
        # third-order part below (2^-6)^2, roundings below 1e-4 of the magnitudes
        assert abs(num - ana) <= 1e-3 * (g[n].double().abs() * v.double().abs()).sum(), n
