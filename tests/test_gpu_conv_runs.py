"""The convolution where a wave's run of tokens is 16, 32 or 64 long, alone and with several packed ends in a run, and where
outputs are stored around the caches, against its definition in float64 (torch on the GPU)."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from gpu_util import seed_of
from layer_util import CONV_K, TYPES, ULP, i32

pytestmark = pytest.mark.gpu


def define(x, w, b, state, cu, act):
    """(y, state_T) in the type of the inputs, differentiable."""
    B, T, C = x.shape
    W = w.shape[1]
    if cu is None:
        start, seq, ends = torch.zeros(T, dtype=torch.long, device="cuda").expand(B, T), torch.arange(B, device="cuda")[:, None].expand(B, T), [(r, 0, T) for r in range(B)]
    else:
        lens = torch.tensor(np.diff(cu), device="cuda")
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)[None]
        start, ends = torch.tensor(cu[:-1], device="cuda")[seq], [(0, a, e) for a, e in zip(cu[:-1], cu[1:])]
        x, T = x[:, :cu[-1]], cu[-1]
    row = torch.arange(B, device="cuda")[:, None]
    t = torch.arange(T, device="cuda")[None]
    u = b
    for j in range(W):
        at = t - (W - 1) + j
        old = state[seq, (at - start + W - 1).clamp(0, W - 2)]
        u = u + w[:, j] * torch.where((at >= start)[..., None], x[row, at.clamp(min=0)], old)
    last = torch.stack([torch.cat([state[n], x[r, a:e]])[-(W - 1):] for n, (r, a, e) in enumerate(ends)])
    return (u * torch.sigmoid(u) if act == "silu" else u), last


def close(got, want, mag, k, what):
    half = 2.0 ** -8 * want.abs() if got.dtype == torch.bfloat16 else 0.0
    lim = (1 + 2.0 ** -8) * k * ULP * mag + half + 1e-37
    worst = ((got.double() - want).abs() / lim).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound"


def run(B, T, C, W, dtype, act, cu=None):
    g = torch.Generator("cuda").manual_seed(seed_of("runs", B, T, C, W, dtype) % 2 ** 31)
    n = B if cu is None else len(cu) - 1
    ty = TYPES[dtype]
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, state, dy, dl = (rnd(*s).to(ty) for s in ((B, T, C), (n, W - 1, C), (B, T, C), (n, W - 1, C)))
    w, b = rnd(C, W) / W ** 0.5, 0.2 * rnd(C)
    off = None if cu is None else i32(cu)
    end = T if cu is None else cu[-1]
    y, last = torch.full_like(x, 7.0), torch.empty_like(state)
    drl.dr_conv_fwd(x, w, b, state, off, y, last, act)
    got = dict(dx=torch.full_like(x, 7.0), dweight=torch.empty_like(w), dbias=torch.empty_like(b), dstate=torch.empty_like(state))
    drl.dr_conv_bwd(x, w, b, state, off, dy, dl, *got.values(), act)
    assert (y[:, end:] == 7.0).all() and (got["dx"][:, end:] == 7.0).all()

    ins = [a.double().requires_grad_() for a in (x, w, b, state)]
    want, wl = define(*ins, cu, act)
    grads = torch.autograd.grad([want, wl], ins, [dy[:, :end].double(), dl.double()])
    # magnitudes: the sums over absolute values, with an error of u of half of it in silu' (see the oracle)
    pos = [a.detach().abs().requires_grad_() for a in ins]
    mag, _ = define(*pos, cu, "none")
    slope = 1.1 + 0.5 * mag.detach() if act == "silu" else torch.ones_like(mag)
    gmag = torch.autograd.grad(list(define(*pos, cu, "none")), pos, [dy[:, :end].double().abs() * slope, dl.double().abs()])
    close(y[:, :end], want.detach(), mag.detach(), CONV_K, "y")
    assert torch.equal(last, wl.to(ty))
    # a weight's gradient: the tokens of a run, four waves, and the workgroups' sums sixteen at a time and then sixteen
    sums = 64 + 4 + B * -(-T // 8) // 64 + 1 + 16
    for name, a, want, m in zip(got, got.values(), grads, gmag):
        if name == "dx":
            a, want, m = a[:, :end], want[:, :end], m[:, :end]
        close(a, want, m, CONV_K + (sums if name in ("dweight", "dbias") else 0), name)


# Runs double from 8 while rows x halved runs x channel blocks (64 lanes, of 1 channel each where rows are not aligned, else of 16 bytes; backward
# 4 channels) stay at 4096, up to 32 forward and 64 backward.
@pytest.mark.parametrize("B,T,C,W,dtype,act", [
    (300, 70, 130, 4, "f32", "silu"), (300, 70, 130, 2, "bf16", "none"),    # 16 both
    (600, 70, 130, 3, "f32", "silu"), (600, 70, 130, 4, "bf16", "silu"),    # 32 both
    (2100, 70, 65, 4, "f32", "none"), (2100, 71, 65, 2, "bf16", "silu"),    # 32, 64
    (700, 140, 512, 4, "bf16", "silu"),                                     # 16 with 8 channels, 64 with 4; stored around the caches
    (1100, 130, 256, 3, "f32", "none"),                                     # 32 both with 4 channels; the same
])
def test_rows(B, T, C, W, dtype, act):
    run(B, T, C, W, dtype, act)


@pytest.mark.parametrize("T,C,W,dtype,act", [
    (2800, 1531, 3, "f32", "silu"), (5500, 1531, 2, "bf16", "none"),        # 16; 32
    (11000, 1531, 4, "f32", "silu"), (11000, 1531, 4, "bf16", "silu"),      # 32, 64
    (140000, 128, 4, "f32", "silu"), (140000, 128, 2, "f32", "none"),       # 32 both with 4 channels; stored around the caches
    (270000, 256, 4, "bf16", "silu"), (270000, 256, 3, "bf16", "none"),     # 32 with 8 channels, 64 with 4; the same
])
def test_packed(T, C, W, dtype, act):
    # sequences of none to 200 tokens, many of them within a run, and one of a tenth of the row; the row's last tokens are no one's
    r = np.random.default_rng(T + W)
    lens = r.choice([0, 1, 2, 3, 5, 9, 30, 200], T // 60)
    lens[len(lens) // 3] = T // 10
    lens = lens[np.cumsum(lens) <= T - 11]
    run(1, T, C, W, dtype, act, [0, *(int(a) for a in np.cumsum(lens))])
