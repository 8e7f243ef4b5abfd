"""The decayed linear attention's prefill and step against the float64 token-by-token oracle."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from decay_util import close, dev, make, oracle, tensors
from gpu_util import seed_of

pytestmark = pytest.mark.gpu


def check(x, t, cu=None, **kw):
    """Runs the prefill and compares o and S_T (rows inside a sequence)."""
    T = x["v"].shape[1]
    cu_t = None if cu is None else dev(np.asarray(cu, np.int32))
    out = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"], cu_seqlens=cu_t, **kw)
    args = [x[n] for n in ("q", "k", "v", "alpha")]
    o, S = oracle.forward(*args, x["S0"], cu)
    mo, mS = oracle.forward(*args, x["S0"], cu, magnitudes=True)
    end = T if cu is None else cu[-1]
    close(out[0][:, :end], o[:, :end], mo[:, :end], T, "o")
    close(out[1], S, mS, T, "S_T")
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 128), (64, 32), (128, 16), (128, 64), (128, 128), (16, 128)])
@pytest.mark.parametrize("decay", ["token", "signed", "head"])
def test_prefill(dk, dv, dtype, decay):
    x = make(seed_of(dk, dv, dtype, decay), 2, 150, 4, 2, dk, dv, dtype, decay)
    check(x, tensors(x, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129])
def test_prefill_lengths(T, dtype):
    x = make(seed_of("len", T, dtype), 1, T, 2, 1, 64, 32, dtype, "signed")
    check(x, tensors(x, dtype))


@pytest.mark.parametrize("ct", [1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 64), (64, 64), (128, 128)])
def test_prefill_column_blocks(ct, dtype, dk, dv, monkeypatch):
    monkeypatch.setenv("DR_DECAY_CT", str(ct))
    x = make(seed_of("ct", ct, dtype, dk, dv), 1, 200, 3, 3, dk, dv, dtype, "small")
    check(x, tensors(x, dtype))


@pytest.mark.parametrize("seg", [64, 128, 192])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 32), (64, 128), (128, 128)])
def test_prefill_segments(seg, dtype, dk, dv, monkeypatch):
    monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("seg", seg, dtype, dk, dv), 2, 333, 2, 1, dk, dv, dtype, "token")
    t = tensors(x, dtype)
    check(x, t)
    x0 = dict(x, S0=None)
    check(x0, tensors(x0, dtype))


CU = [0, 70, 70, 71, 199, 263, 263, 300]  # empty sequences, one token, ends inside and on chunks; 10 rows behind


@pytest.mark.parametrize("seg", [0, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head", "signed"])
def test_packed(seg, dtype, decay, monkeypatch):
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(seed_of("packed", seg, dtype, decay), 1, 310, 6, 2, 64, 64, dtype, decay, n=len(CU) - 1)
    t = tensors(x, dtype)
    o = torch.full((1, 310, 6, 64), 7.0, device="cuda")
    S = torch.empty_like(t["S0"])
    drl.dr_decay_fwd(t["q"], t["k"], t["v"], t["alpha"], t["S0"], dev(np.asarray(CU, np.int32)), o, S)
    assert (o[:, 300:] == 7.0).all(), "rows behind the last sequence were written"
    check(x, t, cu=CU)


def test_packed_rows_behind_the_end_are_not_read():
    x = make(5, 1, 310, 2, 2, 64, 64, "bf16", "token", n=len(CU) - 1)
    for n in ("q", "k", "v", "alpha"):
        x[n][:, 300:] = np.nan
    check(x, tensors(x, "bf16"), cu=CU)


def test_many_sequences_of_one_token():
    n = 700
    x = make(6, 1, n, 2, 1, 32, 32, "bf16", "token", n=n)
    check(x, tensors(x, "bf16"), cu=list(range(n + 1)))


def test_offsets_out_of_range_touch_nothing_else():
    # malformed offsets: results are unspecified, but what is written stays inside the outputs
    x = make(7, 1, 130, 2, 2, 64, 64, "bf16", "token", n=3)
    t = tensors(x, "bf16")
    pad = torch.full((3 * 130 * 2 * 64,), 7.0, device="cuda")
    o = pad[130 * 2 * 64:2 * 130 * 2 * 64].view(1, 130, 2, 64)
    for cu in ([0, 90, 40, 500], [-5, 64, 1 << 30, 10], [130, 0, 0, 0]):
        drl.dr_decay_fwd(t["q"], t["k"], t["v"], t["alpha"], t["S0"], dev(np.asarray(cu, np.int32)), o,
                         torch.empty_like(t["S0"]))
    torch.cuda.synchronize()
    assert (pad[:130 * 2 * 64] == 7.0).all() and (pad[2 * 130 * 2 * 64:] == 7.0).all()


@pytest.mark.parametrize("seg", [0, 128])
def test_snapshots_and_slots(seg, monkeypatch):
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    x = make(8, 2, 333, 2, 2, 64, 64, "f32", "token")
    t = tensors(x, "f32")
    o, S, snaps = check(x, t, snapshot_every=128)
    for b in range(2):
        for j in range(2):
            cut = {n: x[n][b:b + 1, :128 * (j + 1)] for n in ("q", "k", "v", "alpha")}
            _, want = oracle.forward(*cut.values(), x["S0"][b:b + 1])
            _, mag = oracle.forward(*cut.values(), x["S0"][b:b + 1], magnitudes=True)
            close(snaps[2 * b + j], want[0], mag[0], 333, f"snapshot {b} {j}")
    # packed, with a pool: slots 4 and outside
    cu = [0, 200, 333]
    x = make(9, 1, 333, 2, 2, 64, 64, "f32", "token", n=6)
    t = tensors(x, "f32")
    pool = t["S0"].clone()
    idx = dev(np.asarray([4, -1], np.int32))
    o, pool, snaps = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=pool, cu_seqlens=dev(np.asarray(cu, np.int32)),
                                   state_idx=idx, snapshot_every=64)
    S0 = np.stack([x["S0"][4], np.zeros_like(x["S0"][0])])
    want_o, want_S = oracle.forward(x["q"], x["k"], x["v"], x["alpha"], S0, cu)
    mo, mS = oracle.forward(x["q"], x["k"], x["v"], x["alpha"], S0, cu, magnitudes=True)
    close(o, want_o, mo, 333, "o")
    close(pool[4], want_S[0], mS[0], 333, "slot 4")
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(pool[keep], t["S0"][keep]), "a slot that nobody names changed"
    assert snaps.shape[0] == 3 + 2
    cut = {n: x[n][:, 200:328] for n in ("q", "k", "v", "alpha")}
    close(snaps[4], oracle.forward(*cut.values())[1][0], oracle.forward(*cut.values(), magnitudes=True)[1][0], 333,
          "snapshot of the second sequence")


def test_final_state_in_place_and_states_only():
    x = make(10, 3, 100, 2, 1, 64, 32, "bf16", "token")
    t = tensors(x, "bf16")
    o, S = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"])
    S2 = t["S0"].clone()
    drl.dr_decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S2, None, None, S2)
    assert torch.equal(S, S2)
    o2, none = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"], output_final_state=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_views(dtype):
    # q, k, v as slices of one projection whose rows also carry something else, and a slice along T
    B, T, H, d = 2, 140, 4, 64
    x = make(11, B, T, H, H, d, d, dtype, "token")
    t = tensors(x, dtype)
    big = torch.full((B, T + 9, 4, H, d), float("nan"), device="cuda", dtype=t["q"].dtype)
    for i, n in enumerate("qkv"):
        big[:, 4:T + 4, i] = t[n]
    view = dict(t, **{n: big[:, 4:T + 4, i] for i, n in enumerate("qkv")})
    a = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"])
    b = drl.decay_fwd(view["q"], view["k"], view["v"], t["alpha"], S0=t["S0"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_empty():
    for B, T in ((2, 0), (0, 5)):
        x = make(12, B, T, 2, 2, 32, 32, "bf16", "token")
        t = tensors(x, "bf16")
        o, S = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"])
        assert torch.equal(S, t["S0"]) and o.shape == (B, T, 2, 32)


def test_long_sequence_with_segments():
    x = make(13, 1, 9000, 2, 1, 128, 128, "bf16", "token")
    assert 9000 > 512  # more than one segment for two heads
    check(x, tensors(x, "bf16"))


def test_other_heads_are_not_affected_by_nan():
    x = make(14, 2, 100, 4, 4, 64, 64, "bf16", "token")
    t = tensors(x, "bf16")
    o, S = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"])
    t["v"][0, 50, 1] = float("nan")
    o2, S2 = drl.decay_fwd(t["q"], t["k"], t["v"], t["alpha"], S0=t["S0"])
    keep = [0, 2, 3]
    assert torch.equal(o[:, :, keep], o2[:, :, keep]) and torch.equal(o[1], o2[1])
    assert torch.equal(S[:, keep], S2[:, keep]) and torch.isnan(o2[0, 50, 1]).any()


# ------------------------------------------------------------------------------------------------ step
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 7, 300])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (64, 32), (128, 128), (32, 64)])
def test_step(dk, dv, N, dtype):
    x = make(seed_of("step", dk, dv, N, dtype), 1, N, 4, 2, dk, dv, dtype, "signed", n=N)
    t = tensors(x, dtype)
    S = t["S0"].clone()
    one = lambda n: t[n][0]  # noqa: E731
    o = drl.decay_step(one("q"), one("k"), one("v"), one("alpha"), S)
    want_S, want_o = oracle.step(x["S0"], x["q"][0], x["k"][0], x["v"][0], x["alpha"][0])
    mS, mo = oracle.step(x["S0"], x["q"][0], x["k"][0], x["v"][0], x["alpha"][0], magnitudes=True)
    close(S, want_S, mS, 1, "S")
    close(o, want_o, mo, 1, "o")


def test_step_slots_strides_and_decay_per_head():
    N, H, d, pool = 5, 4, 64, 9
    x = make(21, 1, N, H, H, d, d, "bf16", "head", n=pool)
    t = tensors(x, "bf16")
    qkv = torch.stack([t["q"][0], t["k"][0], t["v"][0]], 1)  # [N, 3, H, d]
    slots = [3, 0, 99, 8, -1]
    S = t["S0"].clone()
    o = drl.decay_step(qkv[:, 0], qkv[:, 1], qkv[:, 2], t["alpha"], S, state_idx=dev(np.asarray(slots, np.int32)))
    live = [0, 1, 3]
    rows = [slots[n] for n in live]
    pick = lambda n: x[n][0][live]  # noqa: E731
    want_S, want_o = oracle.step(x["S0"][rows], pick("q"), pick("k"), pick("v"), x["alpha"])
    mS, mo = oracle.step(x["S0"][rows], pick("q"), pick("k"), pick("v"), x["alpha"], magnitudes=True)
    close(S[rows], want_S, mS, 1, "S")
    close(o[live], want_o, mo, 1, "o")
    assert (o[[2, 4]] == 0).all()
    keep = [r for r in range(pool) if r not in rows]
    assert torch.equal(S[keep], t["S0"][keep])


def test_prefill_then_steps_equals_one_prefill():
    # prompt, then tokens one by one, then another prompt from the state: as one long prefill
    x = make(22, 2, 90, 4, 2, 64, 64, "bf16", "token")
    t = tensors(x, "bf16")
    part = lambda a, b: [t[n][:, a:b].contiguous() for n in ("q", "k", "v", "alpha")]  # noqa: E731
    o1, S = drl.decay_fwd(*part(0, 70), S0=t["S0"])
    outs = [o1]
    for i in range(70, 75):
        outs.append(drl.decay_step(*[a[:, 0] for a in part(i, i + 1)], S)[:, None])
    o3, S = drl.decay_fwd(*part(75, 90), S0=S)
    o = torch.cat(outs + [o3], 1)
    args = [x[n] for n in ("q", "k", "v", "alpha")]
    want, wS = oracle.forward(*args, x["S0"])
    mo, mS = oracle.forward(*args, x["S0"], magnitudes=True)
    close(o, want, mo, 90 + 64 * 7, "o")
    close(S, wS, mS, 90 + 64 * 7, "S")
