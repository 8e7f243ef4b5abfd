"""The prefill's and the backward's workspace entry points without a GPU: sizes, and refusals found on the host before
anything is launched."""
import ctypes
import os

import pytest

import delta_rule_linear_chunked_amd as drl

FAKE, ODD = 0x100000, 0x100010  # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(drl.library_path()):
        from delta_rule_linear_chunked_amd import _build
        _build.build(verbose=False)
    return drl.load_library()


def dims(B=1, T=200, H=2, dk=64, dv=64, N=None, dt=1):
    return drl._Dims(B, T, H, dk, dv, B if N is None else N, dt, 0)


def need(lib, d, variant="kda", packed=0, backward=0):
    n = ctypes.c_int64(-1)
    assert lib.dr_chunk_workspace(ctypes.byref(d), drl.VARIANTS[variant], packed, backward, ctypes.byref(n)) == 0, lib.dr_last_error()
    return n.value


@pytest.mark.parametrize("variant", list(drl.VARIANTS))
def test_sizes(lib, variant):
    d = dims()
    assert need(lib, d, variant) == drl.chunk_fwd_plan_ex(1, 200, 2, 64, 64, variant=variant)["workspace"] > 0
    packed = dims(N=5)
    assert need(lib, packed, variant, 1) == drl.chunk_fwd_plan_ex(1, 200, 2, 64, 64, num_seqs=5, variant=variant)["workspace"]
    for x, p in ((d, 0), (packed, 1)):
        own, given = need(lib, x, variant, p, 1), need(lib, x, variant, p, 2)
        # the forward's records and three 64-step states a head are left out with the caller's checkpoints
        assert own - given >= need(lib, x, variant, p) // 2 and given > 0
        # the walk's partial sums: four rows of d_k for every step, head and block of 32 value columns
        steps = 200 * (2 if variant == "product2" else 1)
        assert given >= steps * 2 * (64 // 32) * 4 * 64 * 4


def test_queries_are_checked(lib):
    n = ctypes.c_int64()
    q = lambda d, variant=0, packed=0, backward=0, out=ctypes.byref(n): lib.dr_chunk_workspace(  # noqa: E731
        None if d is None else ctypes.byref(d), variant, packed, backward, out)
    assert q(None) == -1 and q(dims(), out=None) == -1
    assert q(dims(dk=48)) == -5 and q(dims(), variant=9) == -6
    assert q(dims(B=2, N=3)) == -2 and q(dims(B=2, N=3), packed=1) == -2
    assert q(dims(), backward=3) == -2 and q(dims(), backward=-1) == -2
    assert q(dims(T=1 << 30), variant=4) == -2


def test_a_workspace_is_checked(lib):
    d = dims()
    fwd = [FAKE] * 5 + [None, 0, None, None, FAKE, None, ctypes.byref(d), None]
    n = need(lib, d)
    assert lib.dr_chunk_fwd_ws(*fwd, FAKE, n - 1, None) == -2
    assert lib.dr_chunk_fwd_ws(*fwd, ODD, n, None) == -4
    bwd = [FAKE] * 5 + [None, 0, None, None, FAKE, None] + [FAKE] * 5 + [None, None]
    for ck, kind in ((None, 1), (FAKE, 2)):
        n = need(lib, d, backward=kind)
        assert lib.dr_chunk_bwd_ws(*bwd, ck, ctypes.byref(d), FAKE, n - 1, None) == -2
        assert lib.dr_chunk_bwd_ws(*bwd, ck, ctypes.byref(d), ODD, n, None) == -4
