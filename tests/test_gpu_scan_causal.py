"""Inputs of the selective scan that are not finite: no token before them, and no other channel, sees them."""
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from gpu_util import seed_of
from layer_util import SCAN_IN, i32, make_scan, scan_tensors

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def run(t, cu=None):
    return drl.scan_fwd(*[t[k] for k in SCAN_IN], S0=t["S0"], cu_seqlens=cu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,seg", [("1", 0), ("2", 0), ("2", 16), ("2", 24)])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("at", [0, 1, 20, 31, 32, 129, 149])
def test_earlier_tokens_and_other_channels_are_the_same_bits(at, N, block, seg, dtype, monkeypatch):
    monkeypatch.setenv("DR_SCAN_BLOCK", block)
    if seg:
        monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    T, C, ch = 150, 40, 7
    t = scan_tensors(make_scan(seed_of("causal", at, N, dtype), 1, T, C, 1, N, dtype), dtype)
    y, S = run(t)
    others = [c for c in range(C) if c != ch]
    for name, value in (("x", NAN), ("x", INF), ("x", -INF), ("dt", NAN), ("dt", INF), ("z", NAN)):
        bad = dict(t, **{name: t[name].clone()})
        bad[name][0, at, ch] = value
        yb, Sb = run(bad)
        assert torch.equal(yb[:, :at], y[:, :at]), (name, value)
        assert torch.equal(yb[..., others], y[..., others]) and torch.equal(Sb[:, others], S[:, others]), (name, value)
        if name == "z":
            assert torch.isnan(yb[0, at, ch]) and torch.equal(yb[0, at + 1:, ch], y[0, at + 1:, ch]) and torch.equal(Sb, S)
        else:  # the state is not finite from there on
            assert not torch.isfinite(yb[0, at:, ch]).any() and not torch.isfinite(Sb[0, ch]).any(), (name, value)
    for name in ("B", "C"):  # of the group: every channel, from this token on
        for value in (NAN, INF):
            bad = dict(t, **{name: t[name].clone()})
            bad[name][0, at, 0, 3] = value
            yb, Sb = run(bad)
            assert torch.equal(yb[:, :at], y[:, :at]), (name, value)
            rest = [n for n in range(N) if n != 3]
            assert torch.equal(Sb[..., rest], S[..., rest]), (name, value)
            if name == "C":
                assert torch.equal(yb[:, at + 1:], y[:, at + 1:]) and torch.equal(Sb, S)
            elif at == T - 1 and value == INF:
                assert torch.isinf(Sb[..., 3]).all()  # (d x is not zero here)
            else:
                assert not torch.isfinite(Sb[..., 3]).any()


@pytest.mark.parametrize("block", ["1", "2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_of_any_value(dtype, block, monkeypatch):
    # rows of several lengths padded with NaN: what stands before the padding is what the rows without it give
    monkeypatch.setenv("DR_SCAN_BLOCK", block)
    lens, T = (1, 14, 33, 64, 101), 101
    t = scan_tensors(make_scan(seed_of("pad", dtype), len(lens), T, 72, 1, 16, dtype), dtype)
    clean, _ = run(t)
    for b, n in enumerate(lens):
        for k in ("x", "dt", "B", "C", "z"):
            t[k][b, n:] = NAN
    y, S = run(t)
    for b, n in enumerate(lens):
        assert torch.equal(y[b, :n], clean[b, :n]) and torch.isnan(y[b, n:]).all(), n
    assert torch.isfinite(S[-1]).all()


def test_a_number_too_large_stays_in_its_sequence():
    # d x B beyond the type's range, in packed sequences
    t = scan_tensors(make_scan(5, 1, 60, 40, 1, 16, "f32", n=3), "f32")
    cu = i32([0, 21, 40, 60])
    y, S = run(t, cu)
    t["x"][0, 39, 3] = 3e38
    t["B"][0, 39] = 1e30
    yb, Sb = run(t, cu)
    assert torch.equal(yb[:, :39], y[:, :39]) and torch.equal(yb[:, 40:], y[:, 40:])
    assert torch.equal(Sb[[0, 2]], S[[0, 2]]) and not torch.isfinite(Sb[1, 3]).any()
