"""The C ABI and the binding of the selective scan, the convolution and the norm without a GPU: exported symbols, workspace
sizes and refusals, all found on the host before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from delta_rule_linear_chunked_amd import _scan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x100000, 0x100001  # never dereferenced: every call below is refused, or has nothing to do
NULL, SHAPE, DTYPE, LAYOUT, UNSUPPORTED = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(drl.library_path()):
        from delta_rule_linear_chunked_amd import _build
        _build.build(verbose=False)
    return drl.load_library()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "deltarule_scan.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(dr_[a-z_]+)\s*\(", text)))
    assert names == ["dr_conv_bwd", "dr_conv_fwd", "dr_conv_step", "dr_conv_workspace", "dr_norm_bwd", "dr_norm_fwd",
                     "dr_norm_workspace", "dr_scan_bwd", "dr_scan_fwd", "dr_scan_step", "dr_scan_workspace"]
    for name in names:
        assert hasattr(lib, name), name


def ref(d):
    return None if d is None else ctypes.byref(d)


def conv(B=1, T=8, C=64, W=4, N=None, ts=64, bs=512, dt=1, act=1):
    return _scan._ConvDims(B, T, C, W, B if N is None else N, ts, bs, dt, act)


def scan(B=1, T=8, C=64, G=1, S=16, N=None, dt=1, soft=1, **strides):
    st = dict(x=(C, T * C), dt_=(C, T * C), b=(G * S, T * G * S), c=(G * S, T * G * S), z=(C, T * C))
    st.update(strides)
    return _scan._ScanDims(B, T, C, G, S, B if N is None else N, *st["x"], *st["dt_"], *st["b"], *st["c"], *st["z"], dt, soft)


def norm(rows=8, C=64, xs=64, rs=64, dt=1, out=0, eps=1e-5, reserved=0):
    return _scan._NormDims(rows, C, xs, rs, dt, out, eps, reserved)


def conv_fwd(lib, d, opts=None, **kw):
    a = dict(x=FAKE, w=FAKE, b=FAKE, state=FAKE, cu=None, y=FAKE, out=FAKE)
    a.update(kw)
    return lib.dr_conv_fwd(*a.values(), ref(d), ref(opts), None)


def conv_step(lib, d, opts=None, **kw):
    a = dict(x=FAKE, w=FAKE, b=FAKE, state=FAKE, y=FAKE)
    a.update(kw)
    return lib.dr_conv_step(*a.values(), ref(d), ref(opts), None)


def conv_bwd(lib, d, ws=None, n=0, **kw):
    a = dict(x=FAKE, w=FAKE, b=FAKE, state=FAKE, cu=None, dy=FAKE, dout=FAKE, dx=FAKE, dw=FAKE, db=FAKE, dstate=FAKE)
    a.update(kw)
    return lib.dr_conv_bwd(*a.values(), ref(d), ws, n, None)


IN = ("x", "dt", "A", "B", "C", "D", "z", "bias")


def scan_fwd(lib, d, opts=None, ws=None, n=0, **kw):
    a = dict({k: FAKE for k in IN}, S0=FAKE, cu=None, y=FAKE, ST=FAKE)
    a.update(kw)
    return lib.dr_scan_fwd(*a.values(), ref(d), ref(opts), ws, n, None)


def scan_step(lib, d, opts=None, **kw):
    a = dict({k: FAKE for k in IN}, S=FAKE, y=FAKE)
    a.update(kw)
    return lib.dr_scan_step(*a.values(), ref(d), ref(opts), None)


def scan_bwd(lib, d, ws=None, n=0, **kw):
    a = dict({k: FAKE for k in IN}, S0=FAKE, cu=None, dy=FAKE, dST=FAKE,
             **{k: FAKE for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dS0")})
    a.update(kw)
    return lib.dr_scan_bwd(*a.values(), ref(d), ws, n, None)


def norm_fwd(lib, d, **kw):
    a = dict(x=FAKE, r=FAKE, w=FAKE, y=FAKE, scales=None, h=FAKE)
    a.update(kw)
    return lib.dr_norm_fwd(*a.values(), ref(d), None)


def norm_bwd(lib, d, ws=None, n=0, **kw):
    a = dict(h=FAKE, w=FAKE, dy=FAKE, dh=FAKE, dx=FAKE, dw=FAKE)
    a.update(kw)
    return lib.dr_norm_bwd(*a.values(), ref(d), ws, n, None)


TOKENS = [
    (dict(dt=7), DTYPE), (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(C=0), SHAPE), (dict(C=(1 << 20) + 32), UNSUPPORTED),
    (dict(B=2, N=3), SHAPE), (dict(B=1 << 16, T=1 << 16), SHAPE), (dict(B=1 << 40), SHAPE), (dict(T=(1 << 31) - 1023), SHAPE),
]


@pytest.mark.parametrize("case,expect", TOKENS + [
    (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED), (dict(act=2), UNSUPPORTED), (dict(ts=-64), SHAPE), (dict(bs=-64), SHAPE),
    (dict(ts=(1 << 24) + 1), LAYOUT), (dict(bs=(1 << 40) + 1), LAYOUT),
])
def test_convolution_sizes_are_checked(lib, case, expect):
    d = conv(**case)
    assert conv_fwd(lib, d) == expect and lib.dr_last_error()
    assert conv_bwd(lib, d) == expect
    n = ctypes.c_int64()
    assert lib.dr_conv_workspace(ref(d), 0, ctypes.byref(n)) == expect


@pytest.mark.parametrize("case,expect", TOKENS + [
    (dict(S=8), UNSUPPORTED), (dict(S=128), UNSUPPORTED), (dict(G=0), SHAPE), (dict(G=3), SHAPE), (dict(C=1 << 18, G=1 << 18), UNSUPPORTED),
    (dict(soft=2), SHAPE), (dict(x=(-1, 0)), SHAPE), (dict(dt_=((1 << 24) + 8, 0)), LAYOUT), (dict(b=(20, 0)), LAYOUT),
    (dict(c=(16, 12)), LAYOUT), (dict(z=(64, (1 << 40) + 8)), LAYOUT), (dict(dt=0, b=(18, 0)), LAYOUT),
])
def test_scan_sizes_are_checked(lib, case, expect):
    d = scan(**case)
    assert scan_fwd(lib, d) == expect and lib.dr_last_error()
    assert scan_bwd(lib, d) == expect
    n = ctypes.c_int64()
    assert lib.dr_scan_workspace(ref(d), 0, 0, ctypes.byref(n)) == expect
    assert lib.dr_scan_workspace(ref(d), 0, 1, ctypes.byref(n)) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(dt=7), DTYPE), (dict(rows=-1), SHAPE), (dict(C=0), SHAPE), (dict(C=32769), UNSUPPORTED), (dict(rows=(1 << 40) + 1), UNSUPPORTED),
    (dict(xs=-1), SHAPE), (dict(rs=-1), SHAPE), (dict(xs=(1 << 40) + 1), LAYOUT), (dict(out=3), DTYPE), (dict(out=-1), DTYPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(reserved=1), SHAPE),
])
def test_norm_sizes_are_checked(lib, case, expect):
    d = norm(**case)
    assert norm_fwd(lib, d) == expect and lib.dr_last_error()
    assert norm_bwd(lib, d) == expect
    n = ctypes.c_int64()
    assert lib.dr_norm_workspace(ref(d), ctypes.byref(n)) == expect


@pytest.mark.parametrize("call,dims,needed,free", [
    (conv_fwd, conv(), "x w y", "b state out"), (conv_bwd, conv(), "x w dy dx dw", "b state dout db dstate"),
    (conv_step, conv(T=1, B=3), "x w state y", "b"),
    (scan_fwd, scan(), "x dt A B C y", "D z bias S0 ST"), (scan_step, scan(T=1, B=3), "x dt A B C S y", "D z bias"),
    (scan_bwd, scan(), "x dt A B C dy dx ddt dA dB dC dD dz dbias", "D z bias S0 dST dS0"),
    (norm_fwd, norm(), "x w y", "r h"), (norm_bwd, norm(), "h w dy dx dw", "dh"),
])
def test_pointers_are_checked(lib, call, dims, needed, free):
    for name in needed.split():
        assert call(lib, dims, **{name: None}) == NULL, name
    for name in (needed + " " + free).split():
        assert call(lib, dims, **{name: ODD}) == LAYOUT, name
    assert call(lib, None) == NULL
    for name in ("w", "A", "D", "bias", "B", "C", "S0", "S", "ST", "dA", "dS0", "db", "dw"):  # 16 bytes
        if name in (needed + " " + free).split():
            assert call(lib, dims, **{name: FAKE + 8}) == LAYOUT, name


def test_packed_sequences_are_checked(lib):
    assert conv_fwd(lib, conv(B=2, N=3), cu=FAKE) == SHAPE and conv_fwd(lib, conv(N=3), cu=ODD) == LAYOUT
    assert scan_fwd(lib, scan(B=2, N=3), cu=FAKE) == SHAPE and scan_fwd(lib, scan(N=3), cu=ODD) == LAYOUT
    assert scan_bwd(lib, scan(B=2, N=3), cu=FAKE) == SHAPE and conv_bwd(lib, conv(B=2, N=3), cu=FAKE) == SHAPE


def opts(**kw):
    o = drl._Opts(None, 0, None, 0)
    for k, v in kw.items():
        setattr(o, k, v)
    return o


@pytest.mark.parametrize("o,expect", [
    (dict(l2norm_qk=1), UNSUPPORTED), (dict(alpha_act=1), UNSUPPORTED), (dict(gate_act=3), UNSUPPORTED), (dict(alpha_dtype=1), UNSUPPORTED),
    (dict(snapshots=FAKE, snapshot_every=64), UNSUPPORTED), (dict(state_idx=ODD, num_slots=3), LAYOUT),
    (dict(state_idx=FAKE, num_slots=-1), SHAPE), (dict(state_idx=FAKE, num_slots=1 << 31), UNSUPPORTED),
])
def test_options_are_checked(lib, o, expect):
    for call, d in ((conv_fwd, conv()), (scan_fwd, scan()), (conv_step, conv(T=1)), (scan_step, scan(T=1))):
        assert call(lib, d, opts(**o)) == expect


def test_steps_are_checked(lib):
    for call, make in ((conv_step, conv), (scan_step, scan)):
        assert call(lib, make(T=2)) == SHAPE
        assert call(lib, make(T=1, B=2, N=3)) == SHAPE


def test_norm_outputs_are_checked(lib):
    assert norm_fwd(lib, norm(), scales=FAKE) == SHAPE  # values have no scales
    assert norm_fwd(lib, norm(out=1)) == NULL           # codes need them
    assert norm_fwd(lib, norm(out=1), scales=FAKE + 4) == LAYOUT
    assert norm_fwd(lib, norm(), r=None) == SHAPE       # no sum to write
    assert norm_bwd(lib, norm(out=2)) == UNSUPPORTED


def need(lib, entry, d, *args):
    n = ctypes.c_int64(-1)
    assert getattr(lib, entry)(ref(d), *args, ctypes.byref(n)) == 0
    return n.value


def test_workspace_sizes(lib, monkeypatch):
    assert need(lib, "dr_scan_workspace", scan(), 0, 0) == 0  # one segment
    assert need(lib, "dr_scan_workspace", scan(), 0, 1) >= 64 * 16 * 4 + 8 * 16 * 8
    monkeypatch.setenv("DR_SCAN_SEG", "16")
    assert need(lib, "dr_scan_workspace", scan(T=100), 0, 0) == 7 * 64 * 16 * 4 + 7 * 64 * 4  # states and sums of seven segments
    assert need(lib, "dr_scan_workspace", scan(T=100, N=5), 1, 0) > 11 * 64 * 17 * 4          # at most six and one a sequence
    monkeypatch.delenv("DR_SCAN_SEG")
    assert need(lib, "dr_conv_workspace", conv(T=100), 0) >= 2 * 5 * 64 * 4
    assert need(lib, "dr_norm_workspace", norm()) == 8 * 64 * 4 or need(lib, "dr_norm_workspace", norm()) == 2 * 64 * 4
    for entry, d, more in (("dr_scan_workspace", scan(), (0, 0)), ("dr_conv_workspace", conv(), (0,)), ("dr_norm_workspace", norm(), ())):
        assert getattr(lib, entry)(ref(d), *more, None) == NULL
        assert getattr(lib, entry)(None, *more, ctypes.byref(ctypes.c_int64())) == NULL


def test_workspace_is_checked(lib, monkeypatch):
    monkeypatch.setenv("DR_SCAN_SEG", "16")
    for call, d, n in ((conv_bwd, conv(), need(lib, "dr_conv_workspace", conv(), 0)), (norm_bwd, norm(), need(lib, "dr_norm_workspace", norm())),
                       (scan_fwd, scan(T=100), need(lib, "dr_scan_workspace", scan(T=100), 0, 0)),
                       (scan_bwd, scan(T=100), need(lib, "dr_scan_workspace", scan(T=100), 0, 1))):
        assert n > 0
        assert call(lib, d, ws=FAKE, n=n - 1) == SHAPE
        assert call(lib, d, ws=ODD, n=n) == LAYOUT


def test_nothing_to_do(lib):
    assert conv_fwd(lib, conv(B=0)) == 0 and conv_fwd(lib, conv(N=0), cu=FAKE) == 0
    assert scan_fwd(lib, scan(B=0)) == 0 and scan_fwd(lib, scan(N=0), cu=FAKE) == 0
    assert conv_step(lib, conv(B=0, T=1)) == 0 and scan_step(lib, scan(B=0, T=1)) == 0
    assert norm_fwd(lib, norm(rows=0)) == 0


# A launch has at most 2^32 - 1 work items. (No workspace of these sizes exists: the sizes are refused first.)
def test_launch_sizes_are_checked(lib):
    big = 1 << 60
    for call, d in (
            (conv_fwd, conv(T=1 << 30, C=1025, ts=1025)), (conv_bwd, conv(T=1 << 30, C=1025, ts=1025)), (conv_step, conv(B=1 << 28, T=1, C=65)),
            (scan_fwd, scan(B=1 << 20, T=1, C=1 << 12)), (scan_fwd, scan(B=1 << 26, T=1, C=32, S=64)), (scan_step, scan(B=1 << 20, T=1, C=1 << 16)),
            (scan_bwd, scan(B=1 << 20, T=1, C=1 << 12)), (scan_bwd, scan(B=1, T=1 << 28, C=32))):
        kw = {} if call in (conv_fwd, conv_step, scan_step) else dict(ws=FAKE, n=big)
        assert call(lib, d, **kw) == UNSUPPORTED, (call, d)
        assert b"work items" in lib.dr_last_error()


# ----------------------------------------------------------------- the binding's own checks (CPU tensors)
def z(*s):
    return torch.zeros(s)


def conv_args(**kw):
    return {**dict(x=z(1, 10, 8), weight=z(8, 4), bias=z(8)), **kw}


@pytest.mark.parametrize("change,message", [
    (dict(x=z(10, 8)), "x must have 3 dimensions"), (dict(weight=z(8)), "weight must have 2"), (dict(weight=z(7, 4)), "weight has shape"),
    (dict(bias=z(7)), "bias has shape"), (dict(bias=z(8).bfloat16()), "bias has dtype"), (dict(x=z(1, 10, 8).half()), "not float32 or bfloat16"),
    (dict(state=z(1, 4, 8)), "state has shape"), (dict(state=z(1, 3, 8).bfloat16()), "state has dtype"), (dict(activation="gelu"), "unknown activation"),
    (dict(cu_seqlens=z(3)), "cu_seqlens has dtype"), (dict(cu_seqlens=torch.zeros(2, 2, dtype=torch.int32)), "vector"),
    (dict(state_idx=torch.zeros(1, dtype=torch.int32)), "needs the pool"), (dict(x=z(1, 8, 10).transpose(1, 2)), "must be dense"),
    (dict(), "on a GPU"),
])
def test_binding_checks_the_convolution(change, message):
    with pytest.raises(ValueError, match=message):
        drl.conv_fwd(**conv_args(**change))


def scan_args(T=10, **kw):
    return {**dict(x=z(1, T, 8), dt=z(1, T, 8), A=z(8, 16), B=z(1, T, 2, 16), C=z(1, T, 2, 16)), **kw}


@pytest.mark.parametrize("change,message", [
    (dict(x=z(10, 8)), "x must have 3 dimensions"), (dict(A=z(8)), "A must have 2"), (dict(B=z(1, 10, 16)), "B must have 4"),
    (dict(dt=z(1, 9, 8)), "dt has shape"), (dict(dt=z(1, 10, 8).bfloat16()), "dt has dtype"), (dict(A=z(7, 16)), "A has shape"),
    (dict(A=z(8, 16).double()), "A has dtype"), (dict(B=z(1, 10, 3, 16)), "not a multiple of 3 groups"), (dict(C=z(1, 10, 1, 16)), "C has shape"),
    (dict(D=z(7)), "D has shape"), (dict(z=z(1, 10, 7)), "z has shape"), (dict(dt_bias=z(8).bfloat16()), "dt_bias has dtype"),
    (dict(S0=z(2, 8, 16)), "S0 has shape"), (dict(cu_seqlens=z(3)), "cu_seqlens has dtype"), (dict(state_idx=torch.zeros(1, dtype=torch.int32)), "needs the pool"),
    (dict(x=z(1, 10, 8).half()), "not float32 or bfloat16|dt has dtype"), (dict(B=z(1, 10, 16, 2).transpose(2, 3)), "must be dense"), (dict(), "on a GPU"),
])
def test_binding_checks_the_scan(change, message):
    with pytest.raises(ValueError, match=message):
        drl.scan_fwd(**scan_args(**change))


def test_binding_checks_steps_and_gradients():
    with pytest.raises(ValueError, match="state has shape"):
        drl.conv_step(z(3, 8), z(8, 4), z(2, 3, 8))
    with pytest.raises(ValueError, match="state must have 3"):
        drl.conv_step(z(3, 8), z(8, 4), z(3, 8))
    with pytest.raises(ValueError, match="state_idx has dtype"):
        drl.conv_step(z(3, 8), z(8, 4), z(2, 3, 8), state_idx=z(3))
    tok = dict(x=z(3, 8), dt=z(3, 8), A=z(8, 16), B=z(3, 1, 16), C=z(3, 1, 16))
    with pytest.raises(ValueError, match="S has shape"):
        drl.scan_step(**tok, S=z(2, 8, 16))
    with pytest.raises(ValueError, match="state_idx has shape"):
        drl.scan_step(**tok, S=z(2, 8, 16), state_idx=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="dy is required"):
        drl.scan_bwd(**scan_args())
    with pytest.raises(ValueError, match="dy is required"):
        drl.conv_bwd(**conv_args())
    with pytest.raises(ValueError, match="dS_T has shape"):
        drl.scan_bwd(**scan_args(), dy=z(1, 10, 8), dS_T=z(1, 8, 15))


@pytest.mark.parametrize("change,message", [
    (dict(weight=z(7)), "weight has shape"), (dict(weight=z(8).bfloat16()), "weight has dtype"), (dict(residual=z(3, 7)), "residual has shape"),
    (dict(residual=z(3, 8).bfloat16()), "residual has dtype"), (dict(x=z(3, 0)), "no channels"), (dict(x=z()), "at least 1 dimension"),
    (dict(x=z(3, 8).half()), "not float32 or bfloat16"), (dict(fmt="int4"), "unknown format"), (dict(x=z(8, 3).t()), "must be dense"),
    (dict(x=z(4, 5, 8)[:, :3]), "evenly spaced"), (dict(), "on a GPU"),
])
def test_binding_checks_the_norm(change, message):
    with pytest.raises(ValueError, match=message):
        drl.norm_fwd(**{**dict(x=z(3, 8), weight=z(8)), **change})


def test_binding_checks_the_norms_outputs():
    x, w = z(3, 8), z(8)
    with pytest.raises(ValueError, match="y has dtype"):
        drl.dr_norm_fwd(x, None, w, x.bfloat16(), None, None)
    with pytest.raises(ValueError, match="scales is required|scales has shape"):
        drl.dr_norm_fwd(x, None, w, x.to(torch.int8), None, None)
    with pytest.raises(ValueError, match="scales are an output"):
        drl.dr_norm_fwd(x, None, w, x.clone(), z(3), None)
    with pytest.raises(ValueError, match="dy has shape"):
        drl.norm_bwd(x, w, z(3, 7))
