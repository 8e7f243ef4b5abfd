"""The 8-bit state cache against its definition in float64: codes and scales exactly."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from decay_util import dev
from gpu_util import seed_of
from oracle import decay as oracle

pytestmark = pytest.mark.gpu


def states(seed, n, H, dk, dv):
    r = np.random.default_rng(seed)
    S = r.standard_normal((n, H, dk, dv)) * np.exp(2 * r.standard_normal((n, H, dk, 1)))
    return S.astype(np.float32)


def same(got, want, what):
    got = got.cpu().double().numpy()
    want = np.asarray(want, dtype=np.float64).astype(np.float32).astype(np.float64)  # code * scale, rounded once
    assert np.array_equal(got, want, equal_nan=True), f"{what}: {np.sum(got != want)} of {got.size} differ"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (64, 32), (32, 64), (128, 128)])
@pytest.mark.parametrize("n,H", [(1, 1), (5, 3), (40, 8)])
def test_round_trip(fmt, dk, dv, n, H):
    S = states(seed_of("cache", fmt, dk, dv, n), n, H, dk, dv)
    codes, scales = drl.state_pack(dev(S), fmt)
    held, sc = oracle.pack(S, fmt)
    same(scales, sc, "scales")
    same(drl.state_unpack(codes, scales), held, "values")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_borders(fmt):
    # rows of exact halves and of their neighbours, largest and smallest magnitudes, zeros, subnormals, one-hot rows
    rows = []
    k = np.arange(-127, 127, dtype=np.float32)
    for s in (1.0, 0.75, 3.0, 1.1, 2.0 ** -100, 2.0 ** 90):
        half = ((k + np.float32(0.5)) * np.float32(s))[:126]
        for y in (half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf))):
            row = np.zeros(128, np.float32)
            row[:126] = y
            row[126] = np.float32(127) * np.float32(s)
            row[127] = -row[126]
            rows.append(row)
    r = np.random.default_rng(3)
    big = np.finfo(np.float32).max
    rows += [np.zeros(128), np.full(128, big), np.full(128, -big), np.full(128, 2.0 ** -149), np.full(128, 2.0 ** -126),
             r.standard_normal(128) * 2.0 ** -130, r.standard_normal(128) * 1e-40, np.eye(128)[5] * 448, np.eye(128)[5] * 449,
             np.linspace(-448, 448, 128), np.linspace(-1, 1, 128) ** 5, 2.0 ** np.linspace(-30, 8, 128)]
    rows = np.stack([np.asarray(x, dtype=np.float32) for x in rows])
    S = np.zeros(((len(rows) + 15) // 16, 1, 16, 128), np.float32)
    S.reshape(-1, 128)[:len(rows)] = rows
    codes, scales = drl.state_pack(dev(S), fmt)
    held, sc = oracle.pack(S, fmt)
    same(scales, sc, "scales")
    same(drl.state_unpack(codes, scales), held, "values")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_with_nan_or_infinity(fmt):
    S = states(4, 2, 2, 16, 32)
    S[0, 1, 3, 7] = np.nan
    S[1, 0, 0, 0] = np.inf
    S[1, 1, 15, 31] = -np.inf
    codes, scales = drl.state_pack(dev(S), fmt)
    held, sc = oracle.pack(S, fmt)
    assert np.isnan(sc).sum() == 3
    same(scales, sc, "scales")
    same(drl.state_unpack(codes, scales), held, "values")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_slots(fmt):
    H, dk, dv, pool, slots = 2, 64, 64, 7, 9
    S = states(5, pool, H, dk, dv)
    t = dev(S)
    dtype = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    codes = torch.full((slots, H, dk, dv), 3, device="cuda", dtype=torch.int8).view(dtype)
    scales = torch.full((slots, H, dk), 5.0, device="cuda")
    before = codes.view(torch.int8).clone()
    rows = [6, 0, -2, 3, 2]      # -2: no stored state, held as zeros
    into = [8, 1, 4, 9, 0]       # 9: outside the cache, skipped
    i32 = lambda x: dev(np.asarray(x, np.int32))  # noqa: E731
    drl.dr_state_pack(t, codes, scales, slot_idx=i32(into), state_idx=i32(rows))
    held, sc = oracle.pack(np.stack([S[6], S[0], np.zeros_like(S[0]), S[2]]), fmt)
    named = [8, 1, 4, 0]
    same(scales[named], sc, "scales")
    rest = [s for s in range(slots) if s not in named]
    assert torch.equal(codes.view(torch.int8)[rest], before[rest]) and (scales[rest] == 5.0).all()
    # back: one slot into two rows, a slot outside (zeros), a row outside (skipped)
    out = torch.full((4, H, dk, dv), 9.0, device="cuda")
    drl.dr_state_unpack(codes, scales, out, slot_idx=i32([8, 8, 77, 0]), state_idx=i32([0, 2, 3, 4]))
    same(out[0], held[0], "row 0")
    same(out[2], held[0], "row 2")
    assert (out[3] == 0).all() and (out[1] == 9.0).all()


def test_offsets_past_32_bits():
    # the last slot's codes start past 2^32 bytes
    H, dk, dv = 16, 128, 128
    slots = (1 << 32) // (H * dk * dv) + 2
    S = states(6, 1, H, dk, dv)
    codes = torch.empty((slots, H, dk, dv), device="cuda", dtype=torch.int8)
    scales = torch.empty((slots, H, dk), device="cuda")
    idx = dev(np.asarray([slots - 1], np.int32))
    drl.dr_state_pack(dev(S), codes, scales, slot_idx=idx)
    held, _ = oracle.pack(S, "int8")
    same(drl.state_unpack(codes, scales, slot_idx=idx), held, "values")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_resumed_sequence(fmt):
    # prefill, park the state, resume from the cache: the outputs move by the cache's rounding, and equal the
    # prefill from the values that the cache holds bit for bit
    from decay_util import make, tensors
    x = make(7, 2, 128, 2, 1, 64, 64, "bf16", "token")
    t = tensors(x, "bf16")
    cut = lambda a, b: [t[n][:, a:b].contiguous() for n in ("q", "k", "v", "alpha")]  # noqa: E731
    _, S = drl.decay_fwd(*cut(0, 64), S0=t["S0"])
    codes, scales = drl.state_pack(S, fmt)
    back = drl.state_unpack(codes, scales)
    held, _ = oracle.pack(S.cpu().numpy(), fmt)
    same(back, held, "values")
    o, _ = drl.decay_fwd(*cut(64, 128), S0=back)
    o2, _ = drl.decay_fwd(*cut(64, 128), S0=dev(held.astype(np.float32)))
    assert torch.equal(o, o2)
    # half a step of the largest value per entry: 1/254 (int8), 2^-4 (e4m3)
    step = 1 / 254 if fmt == "int8" else 2.0 ** -4
    assert ((back - S).abs() <= step * S.abs().amax(-1, keepdim=True) * (1 + 2.0 ** -20)).all()
