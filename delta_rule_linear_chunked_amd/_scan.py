"""Binding of the selective scan, the short causal convolution and the norm (``include/deltarule_scan.h``).

Argument marshalling only, as for the recurrences: shapes, dtypes and layouts are checked, raw pointers and the current
stream go to the library, a non-zero status raises. The ``dr_*`` functions write into the caller's tensors;
``conv_fwd``, ``scan_fwd``, ``norm_fwd``, their steps and gradients allocate; ``causal_conv``, ``selective_scan`` and
``rms_norm`` wire both directions into torch autograd.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _DT, _Opts, _check, _dense, _need_rows, load_library
from ._decay import CACHE_FORMATS, _addr, _call, _like, _require

CONV_ACTS = {None: 0, "none": 0, "silu": 1}  # dr_conv_act
_NORM_OUT = {None: 0, "int8": 1, "e4m3": 2}  # dr_norm_out
_I64, _I32 = ctypes.c_int64, ctypes.c_int32


class _ConvDims(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("channels", _I64), ("width", _I64), ("num_seqs", _I64),
                ("x_token_stride", _I64), ("x_batch_stride", _I64), ("in_dtype", _I32), ("activation", _I32)]


class _ScanDims(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("channels", _I64), ("groups", _I64), ("state_dim", _I64), ("num_seqs", _I64),
                ("x_token_stride", _I64), ("x_batch_stride", _I64), ("dt_token_stride", _I64), ("dt_batch_stride", _I64),
                ("b_token_stride", _I64), ("b_batch_stride", _I64), ("c_token_stride", _I64), ("c_batch_stride", _I64),
                ("z_token_stride", _I64), ("z_batch_stride", _I64), ("in_dtype", _I32), ("softplus", _I32)]


class _NormDims(ctypes.Structure):
    _fields_ = [("rows", _I64), ("channels", _I64), ("x_row_stride", _I64), ("residual_row_stride", _I64),
                ("in_dtype", _I32), ("out", _I32), ("eps", ctypes.c_float), ("reserved", _I32)]


def declare(lib):
    """Signatures of this part of the library."""
    vp, ip, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    op, out = ctypes.POINTER(_Opts), ctypes.POINTER(i64)
    cp, sp, np_ = ctypes.POINTER(_ConvDims), ctypes.POINTER(_ScanDims), ctypes.POINTER(_NormDims)
    for name, args in (("dr_conv_fwd", [vp] * 7 + [cp, op, vp]), ("dr_conv_step", [vp] * 5 + [cp, op, vp]),
                       ("dr_conv_workspace", [cp, ip, out]), ("dr_conv_bwd", [vp] * 11 + [cp, vp, i64, vp]),
                       ("dr_scan_workspace", [sp, ip, ip, out]), ("dr_scan_fwd", [vp] * 12 + [sp, op, vp, i64, vp]),
                       ("dr_scan_step", [vp] * 10 + [sp, op, vp]), ("dr_scan_bwd", [vp] * 21 + [sp, vp, i64, vp]),
                       ("dr_norm_fwd", [vp] * 6 + [np_, vp]), ("dr_norm_workspace", [np_, out]),
                       ("dr_norm_bwd", [vp] * 6 + [np_, vp, i64, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ip


def _space(lib, entry, dev, *args):
    """A call's workspace from torch's allocator (a captured call's then belongs to its graph) and its size."""
    n = _I64()
    _check(lib, getattr(lib, entry)(*args, ctypes.byref(n)), entry)
    return (torch.empty(n.value, dtype=torch.uint8, device=dev), n.value) if n.value else (None, 0)


# The short ways below are for the usual case, dense inner dimensions (these calls are made once per token and layer with little
# GPU work behind them); anything else goes to the checks that say what is wrong.
def _strides(t, name, shape, dtype, dev):
    """(token, batch) strides of [B, T, C] or [B, T, G, n]."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == dev:
        s = t.stride()
        if s[-1] == 1 and (len(s) == 3 or s[2] == shape[3] or shape[2] == 1):
            return (s[1] if shape[1] != 1 else 0), (s[0] if shape[0] != 1 else 0)
    s = _need_rows(t, name, shape, 2, dtype, dev)
    return s[1], s[0]


def _strides1(t, name, shape, dtype, dev):
    """(0, stride between sequences) of a step's [N, C] or [N, G, n]."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == dev:
        s = t.stride()
        if s[-1] == 1 and (len(s) == 2 or s[1] == shape[2] or shape[1] == 1):
            return 0, (s[0] if shape[0] != 1 else 0)
    return 0, _need_rows(t, name, shape, 1, dtype, dev)[0]


def _type(x, name="x"):
    if x.dtype not in _DT:
        raise ValueError(f"{name} dtype {x.dtype} is not float32 or bfloat16")
    return _DT[x.dtype]


def _optional(t, name, shape, dtype, dev):
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev):
        _require(t, name, shape, dtype, dev)


def _seqs(cu_seqlens, B, dev):
    """Number of sequences; ``cu_seqlens`` checked."""
    if cu_seqlens is None:
        return B
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a vector of num_seqs + 1 offsets")
    _require(cu_seqlens, "cu_seqlens", (cu_seqlens.shape[0],), torch.int32, dev)
    return cu_seqlens.shape[0] - 1


def _slots(state_idx, N, pools, dev):
    """Rows of the state buffers and the options block."""
    if state_idx is None:
        return N, None
    _require(state_idx, "state_idx", (N,), torch.int32, dev)
    rows = next((t.shape[0] for t in pools if t is not None), 0)
    return rows, ctypes.byref(_Opts(state_idx.data_ptr(), rows))


def _rank(t, name, n):
    if t is None or t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {None if t is None else t.dim()}")


# ------------------------------------------------------------------------------------------------ convolution
def _conv_inputs(x, weight, bias, activation, lead):
    _rank(x, "x", lead + 1)
    _rank(weight, "weight", 2)
    if activation not in CONV_ACTS:
        raise ValueError(f"unknown activation {activation!r}")
    dev, C, W = x.device, x.shape[-1], weight.shape[1]
    B, T = (x.shape[0], x.shape[1]) if lead == 2 else (x.shape[0], 1)
    d = _ConvDims(B, T, C, W, B, 0, 0, _type(x), CONV_ACTS[activation])
    d.x_token_stride, d.x_batch_stride = (_strides if lead == 2 else _strides1)(x, "x", x.shape, x.dtype, dev)
    _require(weight, "weight", (C, W), torch.float32, dev)
    _optional(bias, "bias", (C,), torch.float32, dev)
    return d


def dr_conv_fwd(x, weight, bias, state, cu_seqlens, y, state_T, activation="silu", state_idx=None) -> None:
    """The convolution of ``x`` [B,T,C] (fp32 or bf16, a view with free batch and token strides) with ``weight`` [C,width]
    (and ``bias`` [C]; fp32) into ``y`` [B,T,C]. ``state`` and ``state_T`` [N,width-1,C] hold the inputs before and the
    last inputs of each sequence (x's dtype, either may be None, they may be the same); ``state_idx`` [N] int32 names
    their rows in pools."""
    lib = load_library()
    d = _conv_inputs(x, weight, bias, activation, 2)
    dev, B, T, C, W = x.device, d.batch, d.seqlen, d.channels, d.width
    d.num_seqs = N = _seqs(cu_seqlens, B, dev)
    rows, opts = _slots(state_idx, N, (state, state_T), dev)
    _optional(state, "state", (rows, W - 1, C), x.dtype, dev)
    _optional(state_T, "state_T", (rows, W - 1, C), x.dtype, dev)
    _require(y, "y", (B, T, C), x.dtype, dev)
    _call(lib, "dr_conv_fwd", dev, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(state), _addr(cu_seqlens),
          y.data_ptr(), _addr(state_T), ctypes.byref(d), opts)


def conv_fwd(x, weight, bias=None, state=None, cu_seqlens=None, activation="silu", output_final_state: bool = True,
             state_idx=None):
    """Allocates ``y`` (and the final state) and runs ``dr_conv_fwd``. Returns (y, state_T or None). With ``state_idx``,
    ``state`` is a pool that is updated in place and returned. Rows of ``y`` past the last packed sequence are not
    written."""
    _rank(x, "x", 3)
    _rank(weight, "weight", 2)
    state_T = None
    if state_idx is not None:
        if state is None:
            raise ValueError("state_idx needs the pool of states as state")
        state_T = state
    elif output_final_state:
        N = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        state_T = torch.empty((N, weight.shape[1] - 1, x.shape[2]), dtype=x.dtype, device=x.device)
    y = _like(x, x.dtype)
    dr_conv_fwd(x, weight, bias, state, cu_seqlens, y, state_T, activation, state_idx)
    return y, state_T


def dr_conv_step(x, weight, bias, state, y, activation="silu", state_idx=None) -> None:
    """One token for each sequence: ``x`` [N,C] into ``y`` [N,C], ``state`` [N,width-1,C] (or with ``state_idx`` the rows
    it names of a pool) updated in place."""
    lib = load_library()
    d = _conv_inputs(x, weight, bias, activation, 1)
    dev, N, C = x.device, d.batch, d.channels
    _rank(state, "state", 3)
    rows, opts = _slots(state_idx, N, (state,), dev)
    _require(state, "state", (rows, d.width - 1, C), x.dtype, dev)
    _require(y, "y", (N, C), x.dtype, dev)
    _call(lib, "dr_conv_step", dev, x.data_ptr(), weight.data_ptr(), _addr(bias), state.data_ptr(), y.data_ptr(),
          ctypes.byref(d), opts)


def conv_step(x, weight, state, bias=None, activation="silu", state_idx=None):
    """Allocates ``y`` and runs ``dr_conv_step`` (state, or its rows ``state_idx``, updated in place). Returns y."""
    y = _like(x, x.dtype)
    dr_conv_step(x, weight, bias, state, y, activation, state_idx)
    return y


def dr_conv_bwd(x, weight, bias, state, cu_seqlens, dy, dstate_T, dx, dweight, dbias, dstate, activation="silu") -> None:
    """Gradients of ``dr_conv_fwd`` for ``dy`` [B,T,C] and ``dstate_T`` [N,width-1,C] (None: zero), both of x's dtype and
    dense: ``dx`` [B,T,C] and ``dstate`` [N,width-1,C] (or None) in x's dtype, ``dweight`` [C,width] and ``dbias`` [C] (or None)
    in fp32."""
    lib = load_library()
    d = _conv_inputs(x, weight, bias, activation, 2)
    dev, B, T, C, W = x.device, d.batch, d.seqlen, d.channels, d.width
    d.num_seqs = N = _seqs(cu_seqlens, B, dev)
    for t, name in ((state, "state"), (dstate_T, "dstate_T"), (dstate, "dstate")):
        _optional(t, name, (N, W - 1, C), x.dtype, dev)
    _require(dy, "dy", (B, T, C), x.dtype, dev)
    _require(dx, "dx", (B, T, C), x.dtype, dev)
    _require(dweight, "dweight", (C, W), torch.float32, dev)
    _optional(dbias, "dbias", (C,), torch.float32, dev)
    ws, n = _space(lib, "dr_conv_workspace", dev, ctypes.byref(d), cu_seqlens is not None)
    _call(lib, "dr_conv_bwd", dev, *map(_addr, (x, weight, bias, state, cu_seqlens, dy, dstate_T, dx, dweight, dbias, dstate)),
          ctypes.byref(d), _addr(ws), n)


def conv_bwd(x, weight, bias=None, state=None, cu_seqlens=None, activation="silu", dy=None, dstate_T=None):
    """Allocates the gradients and runs ``dr_conv_bwd``. Returns a dict with dx, dweight, dbias (None without bias) and
    dstate (None without state). Rows past the last packed sequence are not written."""
    g = dict(dx=_like(x, x.dtype), dweight=_like(weight), dbias=None if bias is None else _like(bias),
             dstate=None if state is None else _like(state, state.dtype))
    dr_conv_bwd(x, weight, bias, state, cu_seqlens, dy, dstate_T, g["dx"], g["dweight"], g["dbias"], g["dstate"], activation)
    return g


class _CausalConv(torch.autograd.Function):
    """``conv_fwd`` as an autograd node; both directions are the library's kernels."""

    @staticmethod
    def forward(ctx, x, weight, bias, state, cu_seqlens, activation):
        ctx.set_materialize_grads(False)  # an output that the loss does not use gets no gradient
        N = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        # rows that no packed sequence holds are zeros, and so are their gradients
        new = torch.empty if cu_seqlens is None else torch.zeros
        y = new(tuple(x.shape), dtype=x.dtype, device=x.device)
        state_T = torch.empty((N, weight.shape[1] - 1, x.shape[2]), dtype=x.dtype, device=x.device)
        dr_conv_fwd(x, weight, bias, state, cu_seqlens, y, state_T, activation)
        ctx.save_for_backward(x, weight, bias, state, cu_seqlens)
        ctx.activation = activation
        return y, state_T

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dstate_T):
        x, weight, bias, state, cu_seqlens = ctx.saved_tensors
        new = torch.empty if cu_seqlens is None else torch.zeros
        dy = torch.zeros(tuple(x.shape), dtype=x.dtype, device=x.device) if dy is None else _dense(dy)
        dx, dw = new(tuple(x.shape), dtype=x.dtype, device=x.device), _like(weight)
        db, ds = None if bias is None else _like(bias), None if state is None else _like(state, state.dtype)
        dr_conv_bwd(x, weight, bias, state, cu_seqlens, dy, _dense(dstate_T), dx, dw, db, ds, ctx.activation)
        return dx, dw, db, ds, None, None


def causal_conv(x, weight, bias=None, state=None, cu_seqlens=None, activation="silu"):
    """The convolution with gradients through torch autograd: returns (y, state_T) as ``conv_fwd``; ``backward()`` fills
    the ``.grad`` of x, weight, bias and state. In a graph capture take forward and backward together, on leaves that no
    eager graph holds."""
    return _CausalConv.apply(x, weight, bias, state, cu_seqlens, activation)


# ------------------------------------------------------------------------------------------------ selective scan
def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, lead):
    _rank(x, "x", lead + 1)
    _rank(A, "A", 2)
    _rank(B, "B", lead + 2)
    dev, dtype, shape = x.device, x.dtype, x.shape
    Ch, N, G = shape[-1], A.shape[1], B.shape[-2]
    bs, T = (shape[0], shape[1]) if lead == 2 else (shape[0], 1)
    if G == 0 or Ch % G != 0:
        raise ValueError(f"{Ch} channels are not a multiple of {G} groups")
    bc = (bs, T, G, N) if lead == 2 else (bs, G, N)
    st = _strides if lead == 2 else _strides1
    d = _ScanDims(bs, T, Ch, G, N, bs, *st(x, "x", shape, dtype, dev), *st(dt, "dt", shape, dtype, dev), *st(B, "B", bc, dtype, dev),
                  *st(C, "C", bc, dtype, dev), *((0, 0) if z is None else st(z, "z", shape, dtype, dev)), _type(x), 1 if softplus else 0)
    _require(A, "A", (Ch, N), torch.float32, dev)
    _optional(D, "D", (Ch,), torch.float32, dev)
    _optional(dt_bias, "dt_bias", (Ch,), torch.float32, dev)
    return d


def dr_scan_fwd(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, y, S_T, softplus: bool = True, state_idx=None) -> None:
    """The selective scan into ``y`` [B,T,Ch] and ``S_T`` [N,Ch,n] (fp32, may be None, may be S0). x, dt, z [B,T,Ch] and B, C
    [B,T,G,n] of one dtype (fp32 or bf16), views with free batch and token strides; A [Ch,n], D [Ch], dt_bias [Ch] fp32; D,
    z, dt_bias and ``S0`` [N,Ch,n] may be None. ``state_idx`` [N] int32 names the states' rows in pools."""
    lib = load_library()
    d = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, 2)
    dev = x.device
    d.num_seqs = N = _seqs(cu_seqlens, d.batch, dev)
    rows, opts = _slots(state_idx, N, (S0, S_T), dev)
    _optional(S0, "S0", (rows, d.channels, d.state_dim), torch.float32, dev)
    _optional(S_T, "S_T", (rows, d.channels, d.state_dim), torch.float32, dev)
    _require(y, "y", x.shape, x.dtype, dev)
    ws, n = _space(lib, "dr_scan_workspace", dev, ctypes.byref(d), cu_seqlens is not None, 0)
    _call(lib, "dr_scan_fwd", dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z),
          _addr(dt_bias), _addr(S0), _addr(cu_seqlens), y.data_ptr(), _addr(S_T), ctypes.byref(d), opts, _addr(ws), n)


def scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, S0=None, cu_seqlens=None, softplus: bool = True,
             output_final_state: bool = True, state_idx=None):
    """Allocates ``y`` (and the final states) and runs ``dr_scan_fwd``. Returns (y, S_T or None). With ``state_idx``, S0 is a
    pool that is updated in place and returned. Rows of ``y`` past the last packed sequence are not written."""
    _rank(x, "x", 3)
    _rank(A, "A", 2)
    S_T = None
    if state_idx is not None:
        if S0 is None:
            raise ValueError("state_idx needs the pool of states as S0")
        S_T = S0
    elif output_final_state:
        N = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        S_T = torch.empty((N,) + tuple(A.shape), dtype=torch.float32, device=x.device)
    y = _like(x, x.dtype)
    dr_scan_fwd(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, y, S_T, softplus, state_idx)
    return y, S_T


def dr_scan_step(x, dt, A, B, C, D, z, dt_bias, S, y, softplus: bool = True, state_idx=None) -> None:
    """One token for each sequence: x, dt, z [N,Ch], B, C [N,G,n] into ``y`` [N,Ch], the states ``S`` [N,Ch,n] fp32 (or with
    ``state_idx`` the rows it names of a pool) updated in place."""
    lib = load_library()
    d = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, 1)
    dev = x.device
    _rank(S, "S", 3)
    rows, opts = _slots(state_idx, d.batch, (S,), dev)
    _require(S, "S", (rows, d.channels, d.state_dim), torch.float32, dev)
    _require(y, "y", x.shape, x.dtype, dev)
    _call(lib, "dr_scan_step", dev, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z),
          _addr(dt_bias), S.data_ptr(), y.data_ptr(), ctypes.byref(d), opts)


def scan_step(x, dt, A, B, C, S, D=None, z=None, dt_bias=None, softplus: bool = True, state_idx=None):
    """Allocates ``y`` and runs ``dr_scan_step`` (S, or its rows ``state_idx``, updated in place). Returns y."""
    y = _like(x, x.dtype)
    dr_scan_step(x, dt, A, B, C, D, z, dt_bias, S, y, softplus, state_idx)
    return y


def dr_scan_bwd(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, dy, dS_T, dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dS0,
                softplus: bool = True) -> None:
    """Gradients of ``dr_scan_fwd`` for ``dy`` [B,T,Ch] (x's dtype) and ``dS_T`` [N,Ch,n] (fp32, None: zero) into dense tensors of
    the inputs' shapes: dx, ddt, dB, dC and dz in x's dtype, dA, dD, ddt_bias and dS0 in fp32 (dD, dz and ddt_bias None
    without their inputs, dS0 None where it is not wanted)."""
    lib = load_library()
    d = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, 2)
    dev = x.device
    d.num_seqs = N = _seqs(cu_seqlens, d.batch, dev)
    states = (N, d.channels, d.state_dim)
    for t, name in ((S0, "S0"), (dS_T, "dS_T"), (dS0, "dS0")):
        _optional(t, name, states, torch.float32, dev)
    for t, name, like in ((dy, "dy", x), (dx, "dx", x), (ddt, "ddt", x), (dB, "dB", B), (dC, "dC", B), (dz, "dz", z)):
        if like is not None:
            _require(t, name, tuple(like.shape), x.dtype, dev)
    for t, name, like in ((dA, "dA", A), (dD, "dD", D), (ddt_bias, "ddt_bias", dt_bias)):
        if like is not None:
            _require(t, name, tuple(like.shape), torch.float32, dev)
    ws, n = _space(lib, "dr_scan_workspace", dev, ctypes.byref(d), cu_seqlens is not None, 1)
    _call(lib, "dr_scan_bwd", dev, *map(_addr, (x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, dy, dS_T, dx, ddt, dA, dB, dC, dD,
                                                dz, ddt_bias, dS0)), ctypes.byref(d), _addr(ws), n)


def scan_bwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, S0=None, cu_seqlens=None, softplus: bool = True, dy=None,
             dS_T=None, need_dS0: bool = True):
    """Allocates the gradients and runs ``dr_scan_bwd``. Returns a dict with dx, ddt, dA, dB, dC, dD, dz, ddt_bias (None
    without their inputs) and dS0 (None unless ``need_dS0``). Rows past the last packed sequence are not written."""
    _rank(x, "x", 3)
    _rank(A, "A", 2)
    N = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
    like = lambda t: None if t is None else _like(t, t.dtype)  # noqa: E731
    g = dict(dx=like(x), ddt=like(dt), dA=like(A), dB=like(B), dC=like(C), dD=like(D), dz=like(z), ddt_bias=like(dt_bias),
             dS0=torch.empty((N,) + tuple(A.shape), dtype=torch.float32, device=x.device) if need_dS0 else None)
    dr_scan_bwd(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, dy, dS_T, g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"],
                g["dz"], g["ddt_bias"], g["dS0"], softplus)
    return g


class _SelectiveScan(torch.autograd.Function):
    """``scan_fwd`` as an autograd node; both directions are the library's kernels."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, softplus):
        ctx.set_materialize_grads(False)
        N = x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        new = torch.empty if cu_seqlens is None else torch.zeros
        y = new(tuple(x.shape), dtype=x.dtype, device=x.device)
        S_T = torch.empty((N,) + tuple(A.shape), dtype=torch.float32, device=x.device)
        dr_scan_fwd(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, y, S_T, softplus)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens)
        ctx.softplus = softplus
        return y, S_T

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dS_T):
        x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens = ctx.saved_tensors
        new = torch.empty if cu_seqlens is None else torch.zeros
        rows = lambda t: None if t is None else new(tuple(t.shape), dtype=t.dtype, device=t.device)  # noqa: E731
        like = lambda t: None if t is None else _like(t)  # noqa: E731
        dy = torch.zeros(tuple(x.shape), dtype=x.dtype, device=x.device) if dy is None else _dense(dy)
        g = [rows(x), rows(dt), like(A), rows(B), rows(C), like(D), rows(z), like(dt_bias)]
        dS0 = _like(S0) if S0 is not None and ctx.needs_input_grad[8] else None
        dr_scan_bwd(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, dy, _dense(dS_T), *g, dS0, ctx.softplus)
        return (*g, dS0, None, None)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, S0=None, cu_seqlens=None, softplus: bool = True):
    """The scan with gradients through torch autograd: returns (y, S_T) as ``scan_fwd``; ``backward()`` fills the ``.grad`` of
    every input. In a graph capture take forward and backward together, on leaves that no eager graph holds."""
    return _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, S0, cu_seqlens, softplus)


# ------------------------------------------------------------------------------------------------ norm
def _norm_rows(t, name, shape, dtype, dev):
    """Element stride between the rows of a tensor [..., C]: its channels dense, its other dimensions evenly spaced."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev:
        return shape[-1]
    _need_rows(t, name, shape, len(shape) - 1, dtype, dev)
    if t.numel() == 0:
        return 0
    step = None
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] == 1:
            continue
        if step is None:
            step = span = t.stride(i)
        elif t.stride(i) != span:
            raise ValueError(f"{name}: its rows must be evenly spaced, got strides {tuple(t.stride())}")
        span *= t.shape[i]
    return 0 if step is None else step


def _norm_dims(x, weight, residual, eps, out):
    if x.dim() < 1:
        raise ValueError("x must have at least 1 dimension")
    dev, shape, C = x.device, x.shape, x.shape[-1]
    if C == 0:
        raise ValueError("x has no channels")
    rows = x.numel() // C
    d = _NormDims(rows, C, _norm_rows(x, "x", shape, x.dtype, dev),
                  0 if residual is None else _norm_rows(residual, "residual", shape, x.dtype, dev), _type(x), out, eps, 0)
    _require(weight, "weight", (C,), torch.float32, dev)
    return d


def dr_norm_fwd(x, residual, weight, y, scales, h, eps: float = 1e-5) -> None:
    """``x`` [..., C] (plus ``residual``, or None) normalised into ``y``: of x's dtype with scales None, or int8 or float8_e4m3fn
    codes with ``scales`` [...] fp32 (y stands for code * scale). ``h``, the sum in x's dtype, is written with a residual (None:
    not wanted; it may be x or residual)."""
    lib = load_library()
    fmt = next((k for k, v in CACHE_FORMATS.items() if v[1] is y.dtype), None)
    if fmt is None and y.dtype is not x.dtype:
        raise ValueError(f"y has dtype {y.dtype}, expected {x.dtype}, int8 or float8_e4m3fn")
    d = _norm_dims(x, weight, residual, eps, _NORM_OUT[fmt])
    dev = x.device
    _require(y, "y", x.shape, y.dtype, dev)
    _optional(h, "h", x.shape, x.dtype, dev)
    if fmt is not None:
        _require(scales, "scales", x.shape[:-1], torch.float32, dev)
    elif scales is not None:
        raise ValueError("scales are an output of the 8-bit formats")
    _call(lib, "dr_norm_fwd", dev, x.data_ptr(), _addr(residual), weight.data_ptr(), y.data_ptr(), _addr(scales), _addr(h),
          ctypes.byref(d))


def norm_fwd(x, weight, residual=None, eps: float = 1e-5, fmt=None):
    """Allocates the outputs and runs ``dr_norm_fwd``. Returns (y, h), or with ``fmt`` ("int8" or "e4m3") (codes, scales, h); h is x
    itself without a residual."""
    if fmt is not None and fmt not in CACHE_FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    y = _like(x, x.dtype if fmt is None else CACHE_FORMATS[fmt][1])
    scales = None if fmt is None else torch.empty(tuple(x.shape[:-1]), dtype=torch.float32, device=x.device)
    h = None if residual is None else _like(x, x.dtype)
    dr_norm_fwd(x, residual, weight, y, scales, h, eps)
    h = x if residual is None else h
    return (y, h) if fmt is None else (y, scales, h)


def dr_norm_bwd(h, weight, dy, dh, dx, dweight, eps: float = 1e-5) -> None:
    """Gradients of the norm at ``h`` [..., C] for ``dy`` and (or None) ``dh``, what reaches h itself, both of h's dtype and dense:
    ``dx`` in h's dtype (of x and of the residual alike; it may be dh) and ``dweight`` [C] fp32."""
    lib = load_library()
    d = _norm_dims(h, weight, None, eps, 0)
    dev = h.device
    _require(dy, "dy", h.shape, h.dtype, dev)
    _optional(dh, "dh", h.shape, h.dtype, dev)
    _require(dx, "dx", h.shape, h.dtype, dev)
    _require(dweight, "dweight", (d.channels,), torch.float32, dev)
    ws, n = _space(lib, "dr_norm_workspace", dev, ctypes.byref(d))
    _call(lib, "dr_norm_bwd", dev, *map(_addr, (h, weight, dy, dh, dx, dweight)), ctypes.byref(d), _addr(ws), n)


def norm_bwd(h, weight, dy, dh=None, eps: float = 1e-5):
    """Allocates the gradients and runs ``dr_norm_bwd``. Returns a dict with dx and dweight."""
    g = dict(dx=_like(h, h.dtype), dweight=_like(weight))
    dr_norm_bwd(h, weight, dy, dh, g["dx"], g["dweight"], eps)
    return g


class _RmsNorm(torch.autograd.Function):
    """``norm_fwd`` as an autograd node; both directions are the library's kernels."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        y, h = norm_fwd(x, weight, residual, eps)
        ctx.save_for_backward(h, weight)
        ctx.eps, ctx.summed = eps, residual is not None
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        if dy is None:  # only the sum was used
            return dh, torch.zeros_like(weight), dh, None
        g = norm_bwd(h, weight, _dense(dy), _dense(dh), ctx.eps)
        return g["dx"], g["dweight"], g["dx"] if ctx.summed else None, None


def rms_norm(x, weight, residual=None, eps: float = 1e-5):
    """The norm with gradients through torch autograd: y, or with a residual (y, h) as ``norm_fwd``; ``backward()`` fills the
    ``.grad`` of x, weight and residual. In a graph capture take forward and backward together, on leaves that no eager
    graph holds."""
    return _RmsNorm.apply(x, weight, residual, eps)
