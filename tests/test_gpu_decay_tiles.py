"""The prefill's main pass at every width of its workgroups: column tiles of 16 forced from 1 up to all of a head's, and
shapes with enough heads for the plan to take the widest by itself; start states, segments, packed offsets, slots,
snapshots and strides at each, against the float64 oracle."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from decay_norm import close_in_norm
from decay_util import close, dev, make, oracle, tensors
from gpu_util import seed_of

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "alpha")
# (type, d_k, d_v, tiles): bf16 takes up to d_v / 16, fp32 up to two and with d_k = 128 one
WIDTHS = [("bf16", dk, dv, ct) for dk in (16, 32, 64, 128) for dv, ct in ((32, 2), (64, 4), (128, 4), (128, 8))]
WIDTHS += [("f32", dk, 64, 2) for dk in (16, 64)] + [("f32", 128, 128, 1)]
CU = [0, 70, 70, 71, 199, 263, 263, 300]  # empty sequences, one token, ends inside and on chunks; 10 rows behind


def compare(x, out, cu=None):
    args = [x[n] for n in NAMES]
    want, mag = oracle.forward(*args, x["S0"], cu), oracle.forward(*args, x["S0"], cu, magnitudes=True)
    T = x["v"].shape[1]
    end = T if cu is None else cu[-1]
    close(out[0][:, :end], want[0][:, :end], mag[0][:, :end], T, "o")
    close(out[1], want[1], mag[1], T, "S_T")
    close_in_norm(out[0][:, :end], want[0][:, :end], "o")
    close_in_norm(out[1], want[1], "S_T")


@pytest.fixture(params=WIDTHS, ids=lambda w: "-".join(map(str, w)))
def width(request, monkeypatch):
    dtype, dk, dv, ct = request.param
    monkeypatch.setenv("DR_DECAY_CT", str(ct))
    return request.param


@pytest.mark.parametrize("decay", ["signed", "head"])
@pytest.mark.parametrize("T", [1, 63, 65, 150])
def test_prefill(width, T, decay):
    dtype, dk, dv, ct = width
    x = make(seed_of("tiles", width, T, decay), 2, T, 4, 2, dk, dv, dtype, decay)
    t = tensors(x, dtype)
    compare(x, drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"]))


@pytest.mark.parametrize("seg", [64, 192])
def test_segments(width, seg, monkeypatch):
    dtype, dk, dv, ct = width
    monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("tiles seg", width, seg), 2, 333, 2, 1, dk, dv, dtype, "token")
    t = tensors(x, dtype)
    compare(x, drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"]))


@pytest.mark.parametrize("seg", [0, 64])
def test_packed(width, seg, monkeypatch):
    dtype, dk, dv, ct = width
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("tiles packed", width, seg), 1, 310, 6, 2, dk, dv, dtype, "signed", n=len(CU) - 1)
    t = tensors(x, dtype)
    for n in NAMES:
        t[n][:, 300:] = float("nan")  # rows that no sequence holds are not read
    o, S = torch.full((1, 310, 6, dv), 7.0, device="cuda"), torch.empty_like(t["S0"])
    drl.dr_decay_fwd(*[t[n] for n in NAMES], t["S0"], dev(np.asarray(CU, np.int32)), o, S)
    assert (o[:, 300:] == 7.0).all(), "rows behind the last sequence were written"
    compare(x, (o, S), CU)


@pytest.mark.parametrize("seg", [0, 128])
def test_snapshots_slots_and_strides(width, seg, monkeypatch):
    dtype, dk, dv, ct = width
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    B, T, H, pool = 2, 270, 2, 5
    x = make(seed_of("tiles snap", width, seg), B, T, H, H, dk, dv, dtype, "token", n=pool)
    t = tensors(x, dtype)
    # q, k and v as views whose rows carry other data too
    wide = {n: torch.full((B, T + 3, H * t[n].shape[3] + 16), float("nan"), device="cuda", dtype=t[n].dtype) for n in "qkv"}
    view = {}
    for n in "qkv":
        d = t[n].shape[3]
        view[n] = wide[n][:, 2:T + 2, 8:8 + H * d].unflatten(2, (H, d))
        view[n].copy_(t[n])
    slots = [3, 0]
    state, idx = t["S0"].clone(), dev(np.asarray(slots, np.int32))
    o, S, snaps = drl.decay_fwd(view["q"], view["k"], view["v"], t["alpha"], S0=state, state_idx=idx, snapshot_every=128)
    assert S is state and torch.equal(state[[1, 2, 4]], t["S0"][[1, 2, 4]])
    y = dict(x, S0=x["S0"][slots])
    compare(y, (o, S[slots]))
    for j in range(2):
        cut = dict(y, **{n: x[n][:, :128 * (j + 1)] for n in NAMES})
        want, mag = (oracle.forward(*[cut[n] for n in NAMES], cut["S0"], magnitudes=m)[1] for m in (False, True))
        close(snaps[j::2], want, mag, T, f"snapshot {j}")
        close_in_norm(snaps[j::2], want, f"snapshot {j}")
    # states alone
    again = t["S0"].clone()
    drl.dr_decay_fwd(view["q"], view["k"], view["v"], t["alpha"], again, None, None, again, state_idx=idx)
    assert torch.equal(again, state)


@pytest.mark.parametrize("dk,dv", [(16, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
def test_enough_heads_for_the_widest(dk, dv):
    x = make(seed_of("tiles many", dk, dv), 8, 100, 32, 8, dk, dv, "bf16", "token")
    t = tensors(x, "bf16")
    compare(x, drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"]))


def test_a_long_sequence_is_cut():
    # two heads leave most of the chip idle: the call takes room for the states of several segments
    import ctypes
    from delta_rule_linear_chunked_amd import _decay
    lib, n = drl.load_library(), ctypes.c_int64()
    d = _decay._DecayDims(1, 9000, 2, 1, 128, 128, 1, 1, 0, 0, 0)
    assert lib.dr_decay_workspace(ctypes.byref(d), 0, 0, ctypes.byref(n)) == 0
    assert n.value >= 2 * 2 * 128 * 128 * 4
