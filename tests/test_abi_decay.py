"""The C ABI and the binding of the decayed linear attention and the state cache without a GPU: exported symbols and
refusals, all found on the host before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from delta_rule_linear_chunked_amd import _decay

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x100000, 0x100004  # never dereferenced: every call below is refused, or has nothing to do


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(drl.library_path()):
        from delta_rule_linear_chunked_amd import _build
        _build.build(verbose=False)
    return drl.load_library()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "deltarule_decay.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(dr_[a-z_]+)\s*\(", text)))
    assert names == ["dr_decay_bwd", "dr_decay_fwd", "dr_decay_step", "dr_decay_workspace", "dr_state_pack", "dr_state_unpack"]
    for name in names:
        assert hasattr(lib, name), name


def dims(B=1, T=8, H=4, Hk=2, dk=64, dv=64, N=None, dt=1, layout=0, strided=0, reserved=0, strides=()):
    return _decay._DecayDims(B, T, H, Hk, dk, dv, B if N is None else N, dt, layout, strided, reserved, *strides)


BAD_DIMS = [
    (dict(dk=48), -5), (dict(dv=256), -5), (dict(dt=7), -3), (dict(layout=2), -2), (dict(strided=2), -2),
    (dict(reserved=1), -2), (dict(T=-1), -2), (dict(H=0), -2), (dict(Hk=0), -2), (dict(H=4, Hk=3), -2),
    (dict(B=2, N=3), -2), (dict(B=1 << 16, T=1 << 16, N=1 << 16), -2), (dict(H=1 << 17, Hk=1), -5),
    (dict(B=1 << 40, N=1 << 40), -2),
    (dict(strided=1, strides=(-64, 0, 64, 0, 64, 0)), -2), (dict(strided=1, strides=(132, 0, 128, 0, 128, 0)), -4),
    (dict(strided=1, strides=((1 << 24) + 8, 0, 128, 0, 128, 0)), -4),
    (dict(strided=1, strides=(128, 1 << 41, 128, 0, 128, 0)), -4),
]


@pytest.mark.parametrize("case,expect", BAD_DIMS)
def test_sizes_are_checked(lib, case, expect):
    d = dims(**case)
    assert lib.dr_decay_fwd(FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, ctypes.byref(d), None, None, 0, None) == expect
    assert lib.dr_last_error()
    assert lib.dr_decay_bwd(*[FAKE] * 4, None, None, FAKE, None, *[FAKE] * 4, None, ctypes.byref(d), None, 0, None) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(q=None), -1), (dict(alpha=None), -1), (dict(v=ODD), -4), (dict(o=ODD), -4), (dict(S0=ODD), -4), (dict(S_T=ODD), -4),
    (dict(cu=ODD), -4), (dict(d=None), -1), (dict(cu=FAKE, d=dims(B=2, N=3)), -2),
])
def test_prefill_pointers_are_checked(lib, case, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, alpha=FAKE, S0=None, cu=None, o=FAKE, S_T=None, d=dims())
    a.update(case)
    d = a.pop("d")
    assert lib.dr_decay_fwd(*a.values(), ctypes.byref(d) if d is not None else None, None, None, 0, None) == expect


@pytest.mark.parametrize("i", [0, 1, 2, 3, 6, 8, 9, 10, 11])
def test_backward_pointers_are_checked(lib, i):
    a = [FAKE] * 4 + [None, None, FAKE, None] + [FAKE] * 4 + [None]
    for value, expect in ((None, -1), (ODD, -4)):
        b = list(a)
        b[i] = value
        assert lib.dr_decay_bwd(*b, ctypes.byref(dims()), None, 0, None) == expect, (i, value)


def opts(**kw):
    o = drl._Opts(None, 0, None, 0)
    for k, v in kw.items():
        setattr(o, k, v)
    return o


@pytest.mark.parametrize("o,expect", [
    (dict(l2norm_qk=1), -5), (dict(alpha_act=1), -5), (dict(gate_act=3), -5), (dict(alpha_dtype=1), -5),
    (dict(snapshots=FAKE, snapshot_every=100), -2), (dict(snapshots=FAKE, snapshot_every=0), -2),
    (dict(snapshots=ODD, snapshot_every=64), -4), (dict(state_idx=ODD, num_slots=3), -4), (dict(state_idx=FAKE, num_slots=-1), -2),
])
def test_options_are_checked(lib, o, expect):
    assert lib.dr_decay_fwd(*[FAKE] * 4, None, None, FAKE, None, ctypes.byref(dims()), ctypes.byref(opts(**o)), None, 0, None) == expect


def test_step_is_checked(lib):
    a = [FAKE] * 6
    assert lib.dr_decay_step(*a, ctypes.byref(dims(T=2)), None, None) == -2
    assert lib.dr_decay_step(*a, ctypes.byref(dims(T=1, N=3)), None, None) == -2
    assert lib.dr_decay_step(FAKE, FAKE, FAKE, FAKE, None, FAKE, ctypes.byref(dims(T=1)), None, None) == -1
    assert lib.dr_decay_step(*a, ctypes.byref(dims(T=1)), ctypes.byref(opts(snapshots=FAKE, snapshot_every=64)), None) == -2


def need(lib, d, packed=0, backward=0):
    n = ctypes.c_int64(-1)
    assert lib.dr_decay_workspace(ctypes.byref(d), packed, backward, ctypes.byref(n)) == 0
    return n.value


def test_workspace_sizes(lib, monkeypatch):
    assert need(lib, dims(T=8)) == 0  # one segment
    state = 64 * 64 * 4
    assert need(lib, dims(T=200, H=4, Hk=4), backward=1) >= 2 * 4 * 4 * state  # states and gradients of 4 chunks
    shared = need(lib, dims(T=200), backward=1) - need(lib, dims(T=200, H=4, Hk=4), backward=1)
    assert 2 * 200 * 4 * 64 * 4 <= shared < 2 * 200 * 4 * 64 * 4 + 1024
    assert 0 < need(lib, dims(T=100, N=5), packed=1) < 4096
    monkeypatch.setenv("DR_DECAY_SEG", "64")
    assert need(lib, dims(T=200)) >= 4 * 4 * state
    n = ctypes.c_int64()
    assert lib.dr_decay_workspace(ctypes.byref(dims(dk=48)), 0, 0, ctypes.byref(n)) == -5
    assert lib.dr_decay_workspace(ctypes.byref(dims(B=2, N=5)), 0, 0, ctypes.byref(n)) == -2
    assert lib.dr_decay_workspace(ctypes.byref(dims(B=2, N=5)), 1, 0, ctypes.byref(n)) == -2
    assert lib.dr_decay_workspace(ctypes.byref(dims()), 0, 0, None) == -1
    assert lib.dr_decay_workspace(None, 0, 0, ctypes.byref(n)) == -1


def test_workspace_is_checked(lib):
    d = dims(T=200)
    n = need(lib, d, backward=1)
    a = [FAKE] * 4 + [None, None, FAKE, None] + [FAKE] * 4 + [None]
    assert lib.dr_decay_bwd(*a, ctypes.byref(d), FAKE, n - 1, None) == -2
    assert lib.dr_decay_bwd(*a, ctypes.byref(d), ODD, n, None) == -4
    d = dims(T=200, N=3)
    n = need(lib, d, packed=1)
    b = [FAKE] * 4 + [None, FAKE, FAKE, None]
    assert lib.dr_decay_fwd(*b, ctypes.byref(d), None, FAKE, n - 1, None) == -2
    assert lib.dr_decay_fwd(*b, ctypes.byref(d), None, ODD, n, None) == -4


def test_nothing_to_do(lib):
    assert lib.dr_decay_fwd(*[FAKE] * 4, None, None, FAKE, None, ctypes.byref(dims(B=0)), None, None, 0, None) == 0
    assert lib.dr_decay_step(*[FAKE] * 6, ctypes.byref(dims(B=0, T=1)), None, None) == 0
    assert lib.dr_decay_bwd(*[FAKE] * 4, None, None, FAKE, None, *[FAKE] * 4, None, ctypes.byref(dims(B=0)), None, 0, None) == 0
    d = _decay._CacheDims(0, 3, 3, 2, 64, 64, 0, 0)
    assert lib.dr_state_pack(FAKE, None, FAKE, FAKE, None, ctypes.byref(d), None) == 0


@pytest.mark.parametrize("args,expect", [
    ((1, 3, 3, 2, 48, 64, 0, 0), -5), ((1, 3, 3, 2, 64, 64, 2, 0), -3), ((1, 3, 3, 2, 64, 64, 0, 1), -2),
    ((-1, 3, 3, 2, 64, 64, 0, 0), -2), ((4, 3, 9, 2, 64, 64, 0, 0), -2), ((4, 9, 3, 2, 64, 64, 0, 0), -2),
    ((1, 1 << 40, 3, 2, 64, 64, 0, 0), -5), ((1 << 30, 1 << 30, 1 << 30, 16, 64, 64, 0, 0), -5),
])
def test_cache_sizes_are_checked(lib, args, expect):
    d = _decay._CacheDims(*args)
    assert lib.dr_state_pack(FAKE, None, FAKE, FAKE, None, ctypes.byref(d), None) == expect
    assert lib.dr_state_unpack(FAKE, FAKE, None, FAKE, None, ctypes.byref(d), None) == expect


def test_cache_pointers_are_checked(lib):
    d = _decay._CacheDims(1, 3, 3, 2, 64, 64, 0, 0)
    assert lib.dr_state_pack(None, None, FAKE, FAKE, None, ctypes.byref(d), None) == -1
    assert lib.dr_state_pack(FAKE, None, ODD, FAKE, None, ctypes.byref(d), None) == -4
    assert lib.dr_state_unpack(FAKE, FAKE, ODD, FAKE, None, ctypes.byref(d), None) == -4


# ----------------------------------------------------------------- the binding's own checks (CPU tensors)
def inputs(B=1, T=10, H=4, Hk=2, d=32):
    z = lambda *s: torch.zeros(s)  # noqa: E731
    return dict(q=z(B, T, Hk, d), k=z(B, T, Hk, d), v=z(B, T, H, d), alpha=z(B, T, H))


@pytest.mark.parametrize("change,message", [
    (dict(k=torch.zeros(1, 10, 4, 32)), "k has shape"), (dict(v=torch.zeros(1, 9, 4, 32)), "v has shape"),
    (dict(v=torch.zeros(1, 10, 3, 32)), "not a multiple"), (dict(q=torch.zeros(10, 2, 32)), "dimensions"),
    (dict(alpha=torch.zeros(1, 10, 2)), "alpha has shape"), (dict(alpha=torch.zeros(2)), "alpha has shape"),
    (dict(alpha=torch.zeros(1, 10, 4).double()), "alpha has dtype"), (dict(alpha=None), "alpha is required"),
    (dict(q=torch.zeros(1, 10, 2, 32).half()), "not float32 or bfloat16"), (dict(k=torch.zeros(1, 10, 2, 32).bfloat16()), "k has dtype"),
    (dict(v=torch.zeros(1, 10, 32, 4).transpose(2, 3)), "must be dense"),
    (dict(S0=torch.zeros(2, 4, 32, 32)), "S0 has shape"), (dict(cu_seqlens=torch.zeros(3)), "cu_seqlens has dtype"),
    (dict(cu_seqlens=torch.zeros(2, 2, dtype=torch.int32)), "vector"), (dict(state_idx=torch.zeros(1, dtype=torch.int32)), "needs the pool"),
    (dict(), "on a GPU"),
])
def test_binding_checks_the_prefill(change, message):
    with pytest.raises(ValueError, match=message):
        drl.decay_fwd(**{**inputs(), **change})


def test_binding_checks_step_backward_and_cache():
    a = inputs(B=3, T=1)
    tok = {n: t[:, 0].contiguous() for n, t in a.items()}
    with pytest.raises(ValueError, match="S has shape"):
        drl.decay_step(**tok, S=torch.zeros(2, 4, 32, 32))
    with pytest.raises(ValueError, match="state_idx has dtype"):
        drl.decay_step(**tok, S=torch.zeros(2, 4, 32, 32), state_idx=torch.zeros(3))
    with pytest.raises(ValueError, match="dO is required"):
        drl.decay_bwd(**inputs())
    with pytest.raises(ValueError, match="dS_T has shape"):
        drl.decay_bwd(**inputs(), dO=torch.zeros(1, 10, 4, 32), dS_T=torch.zeros(1, 4, 32, 16))
    S, codes, scales = torch.zeros(2, 4, 32, 32), torch.zeros(3, 4, 32, 32, dtype=torch.int8), torch.zeros(3, 4, 32)
    with pytest.raises(ValueError, match="give state_idx or slot_idx"):
        drl.dr_state_pack(S, codes, scales)
    with pytest.raises(ValueError, match="expected int8"):
        drl.dr_state_pack(S, codes.float(), scales)
    with pytest.raises(ValueError, match="scales has shape"):
        drl.dr_state_pack(S, codes, scales[:2])
    with pytest.raises(ValueError, match="slot_idx has shape"):
        drl.dr_state_unpack(codes, scales, S, slot_idx=torch.zeros(3, dtype=torch.int32), state_idx=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="unknown cache format"):
        drl.state_pack(S, "int4")
