"""Calls whose launches would not fit are refused on the host, before the first of them: a kernel's work items along an
axis are a 32-bit number."""
import ctypes
import os

import pytest

import delta_rule_linear_chunked_amd as drl
from delta_rule_linear_chunked_amd import _decay

FAKE = 0x100000  # never dereferenced: every call below is refused
UNSUPPORTED = -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(drl.library_path()):
        from delta_rule_linear_chunked_amd import _build
        _build.build(verbose=False)
    return drl.load_library()


def dims(N, H, dk=16, dv=16, T=1, dt=1, Hk=None, B=None):
    return _decay._DecayDims(N if B is None else B, T, H, Hk or H, dk, dv, N, dt, 0, 0, 0)


@pytest.mark.parametrize("d,packed", [
    (dims(349526, 16), False),          # 5592416 workgroups of 768
    (dims(1 << 15, 256), False),
    (dims(349526, 16, B=1, T=349526), True),
    (dims(1 << 16, 16, dk=128, dv=128, dt=0), False),  # eight column blocks a head
])
def test_prefill(lib, d, packed):
    cu = FAKE if packed else None
    assert lib.dr_decay_fwd(*[FAKE] * 4, None, cu, FAKE, FAKE, ctypes.byref(d), None, FAKE, 1 << 60, None) == UNSUPPORTED
    assert b"work items" in lib.dr_last_error()


@pytest.mark.parametrize("d", [
    dims(524288, 16),                    # 8388608 chunks of heads, 512 threads each
    dims(1, 64, T=64 * 131072),
    dims(1, 64, T=32 * 131072, dt=0),
    dims(1 << 21, 4, dk=128, dv=128, Hk=1),
])
def test_gradients(lib, d):
    a = [FAKE] * 4 + [None, None, FAKE, None] + [FAKE] * 4 + [None]
    assert lib.dr_decay_bwd(*a, ctypes.byref(d), FAKE, 1 << 60, None) == UNSUPPORTED
    assert b"work items" in lib.dr_last_error()


@pytest.mark.parametrize("d", [dims(1 << 20, 16, dk=16, dv=128), dims(1 << 20, 16, dk=128, dv=128), dims(1 << 26, 1)])
def test_step(lib, d):
    assert lib.dr_decay_step(*[FAKE] * 6, ctypes.byref(d), None, None) == UNSUPPORTED
    assert b"work items" in lib.dr_last_error()


@pytest.mark.parametrize("count,H,dk,dv", [(1 << 20, 16, 16, 16), (1 << 20, 4, 128, 128), (1 << 23, 2, 64, 64)])
def test_cache(lib, count, H, dk, dv):
    d = _decay._CacheDims(count, count, count, H, dk, dv, 0, 0)
    assert lib.dr_state_pack(FAKE, None, FAKE, FAKE, None, ctypes.byref(d), None) == UNSUPPORTED
    assert lib.dr_state_unpack(FAKE, FAKE, None, FAKE, None, ctypes.byref(d), None) == UNSUPPORTED
