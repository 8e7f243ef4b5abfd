"""Binding of the decayed linear attention and the 8-bit state cache (``include/deltarule_decay.h``).

Argument marshalling only, as for the gated delta rule: shapes, dtypes and layouts are checked, raw pointers and
the current stream go to the library, a non-zero status raises. The ``dr_*`` functions write into the
caller's tensors; ``decay_fwd``, ``decay_step``, ``decay_bwd``, ``state_pack`` and ``state_unpack`` allocate;
``decay_attention`` wires the prefill and its backward into torch autograd.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _DT, _Opts, _capturing, _check, _dense, _need, _need_rows, check_offsets, load_library, snapshot_count

# code types of the state cache (dr_cache_format)
CACHE_FORMATS = {"int8": (0, torch.int8), "e4m3": (1, torch.float8_e4m3fn)}


class _DecayDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("num_heads", ctypes.c_int64),
                ("num_k_heads", ctypes.c_int64), ("head_dim_k", ctypes.c_int64), ("head_dim_v", ctypes.c_int64),
                ("num_seqs", ctypes.c_int64), ("in_dtype", ctypes.c_int32), ("decay_layout", ctypes.c_int32),
                ("strided", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("q_token_stride", ctypes.c_int64), ("q_batch_stride", ctypes.c_int64),
                ("k_token_stride", ctypes.c_int64), ("k_batch_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_batch_stride", ctypes.c_int64)]


class _CacheDims(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("num_states", ctypes.c_int64), ("num_slots", ctypes.c_int64),
                ("num_heads", ctypes.c_int64), ("head_dim_k", ctypes.c_int64), ("head_dim_v", ctypes.c_int64),
                ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def declare(lib):
    """Signatures of this part of the library."""
    vp, ip = ctypes.c_void_p, ctypes.c_int
    dp, op, cp = ctypes.POINTER(_DecayDims), ctypes.POINTER(_Opts), ctypes.POINTER(_CacheDims)
    lib.dr_decay_workspace.argtypes = [dp, ip, ip, ctypes.POINTER(ctypes.c_int64)]
    lib.dr_decay_fwd.argtypes = [vp] * 8 + [dp, op, vp, ctypes.c_int64, vp]
    lib.dr_decay_step.argtypes = [vp] * 6 + [dp, op, vp]
    lib.dr_state_pack.argtypes = [vp] * 5 + [cp, vp]
    lib.dr_state_unpack.argtypes = [vp] * 5 + [cp, vp]
    lib.dr_decay_bwd.argtypes = [vp] * 13 + [dp, vp, ctypes.c_int64, vp]
    for f in (lib.dr_decay_workspace, lib.dr_decay_fwd, lib.dr_decay_step, lib.dr_decay_bwd, lib.dr_state_pack, lib.dr_state_unpack):
        f.restype = ip


# These calls are made once per token and layer with little GPU work behind them: what the checks cost on the host
# counts. The common case (dense tensors of the right kind on the current device) takes the short ways below;
# anything else goes to the checks that say what is wrong.
def _is(t, shape, dtype, device) -> bool:
    return t is not None and t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()


def _require(t, name, shape, dtype, device):
    if not _is(t, shape, dtype, device):
        _need(t, name, shape, dtype, device)


def _call(lib, entry, device, *args):
    """Calls an entry point with the device's current stream, on that device."""
    index = device.index
    if device.type != "cuda":  # the library has nothing to launch on
        raise ValueError(f"{entry}: tensors must be on a GPU, got {device}")
    fn = getattr(lib, entry)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):  # the library launches on the current device
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        _check(lib, st, entry)


def _workspace(lib, d, dev, packed, backward):
    """A call's workspace from torch's allocator: a captured call's then belongs to its graph."""
    n = ctypes.c_int64()
    _check(lib, lib.dr_decay_workspace(ctypes.byref(d), packed, backward, ctypes.byref(n)), "dr_decay_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=dev) if n.value else None


def _like(t, dtype=torch.float32):
    """An uninitialised dense tensor of t's shape (a third of the time of ``torch.empty``)."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _addr(t):
    return None if t is None else t.data_ptr()


def _options(state_idx, rows, snapshots=None, every=0):
    if state_idx is None and snapshots is None:
        return None
    return ctypes.byref(_Opts(_addr(state_idx), rows, _addr(snapshots), int(every or 0)))


def _ranks(q, v, alpha, lead):
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError(f"q and v must have {lead + 2} dimensions, got {q.dim()} and {v.dim()}")
    if alpha is None:
        raise ValueError("alpha is required")


def _inputs(q, k, v, alpha, lead):
    """Checks q, k, v, alpha with ``lead`` leading dimensions (2: batch and token, 1: sequence) and returns the sizes
    block, num_seqs that of unpacked inputs."""
    _ranks(q, v, alpha, lead)
    dev, dtype, qs, vs = q.device, q.dtype, q.shape, v.shape
    if lead == 2:
        B, T, Hk, dk = qs
        vB, vT, H, dv = vs
        first = (B, T)
    else:
        B, Hk, dk = qs
        vB, H, dv = vs
        T = vT = 1
        first = (B,)
    if dtype not in _DT:
        raise ValueError(f"q dtype {dtype} is not float32 or bfloat16")
    if Hk == 0 or H % Hk != 0:
        raise ValueError(f"{H} value heads are not a multiple of {Hk} query/key heads")
    strides = None
    if not (vB == B and vT == T and q.is_contiguous() and v.is_contiguous() and v.dtype is dtype and v.device == dev
            and _is(k, qs, dtype, dev)):
        strides = (_need_rows(q, "q", first + (Hk, dk), lead, dtype, dev),
                   _need_rows(k, "k", first + (Hk, dk), lead, dtype, dev),
                   _need_rows(v, "v", first + (H, dv), lead, dtype, dev))
    per_head = alpha.dim() == 1
    _require(alpha, "alpha", (H,) if per_head else first + (H,), torch.float32, dev)
    d = _DecayDims(B, T, H, Hk, dk, dv, B, _DT[dtype], int(per_head), 0, 0)
    if strides is not None:
        d.strided = 1
        (d.q_token_stride, d.q_batch_stride), (d.k_token_stride, d.k_batch_stride), \
            (d.v_token_stride, d.v_batch_stride) = [((s[1], s[0]) if lead == 2 else (0, s[0])) for s in strides]
    return d


def _offsets(cu_seqlens, d, dev):
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be a vector of num_seqs + 1 offsets")
        _require(cu_seqlens, "cu_seqlens", (cu_seqlens.shape[0],), torch.int32, dev)
        d.num_seqs = cu_seqlens.shape[0] - 1


def dr_decay_fwd(q, k, v, alpha, S0, cu_seqlens, o, S_T, state_idx=None, snapshots=None,
                 snapshot_every: int = 0) -> None:
    """Prefill of the decayed linear attention into ``o`` [B,T,H,dv] and ``S_T`` [N,H,dk,dv] (fp32, either may be
    None). q, k [B,T,Hk,dk] and v [B,T,H,dv] (fp32 or bf16, views with free batch and token strides), alpha fp32
    [B,T,H] or [H]. ``S0``, ``cu_seqlens``, ``state_idx`` and ``snapshots`` as for ``dr_chunk_fwd_ex``; the offsets
    are clamped on the device and not read on the host."""
    lib = load_library()
    d = _inputs(q, k, v, alpha, 2)
    dev, B, T, H, dk, dv = q.device, d.batch, d.seqlen, d.num_heads, d.head_dim_k, d.head_dim_v
    _offsets(cu_seqlens, d, dev)
    rows = d.num_seqs
    if state_idx is not None:
        _require(state_idx, "state_idx", (d.num_seqs,), torch.int32, dev)
        pools = [t for t in (S0, S_T) if t is not None]
        rows = pools[0].shape[0] if pools else 0
    for t, name in ((S0, "S0"), (S_T, "S_T")):
        if t is not None:
            _require(t, name, (rows, H, dk, dv), torch.float32, dev)
    if snapshots is not None:
        if not snapshot_every or snapshot_every <= 0:
            raise ValueError("snapshots need a positive snapshot_every")
        if cu_seqlens is None:
            rows_s = B * (T // int(snapshot_every))
        elif not _capturing():
            rows_s = snapshot_count(check_offsets(cu_seqlens, T), snapshot_every)
        else:
            rows_s = snapshots.shape[0]
        _require(snapshots, "snapshots", (rows_s, H, dk, dv), torch.float32, dev)
    if o is not None:
        _require(o, "o", (B, T, H, dv), torch.float32, dev)
    ws = _workspace(lib, d, dev, cu_seqlens is not None, False)
    _call(lib, "dr_decay_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), _addr(S0),
          _addr(cu_seqlens), _addr(o), _addr(S_T), ctypes.byref(d), _options(state_idx, rows, snapshots, snapshot_every),
          _addr(ws), 0 if ws is None else ws.numel())


def decay_fwd(q, k, v, alpha, S0=None, cu_seqlens=None, output_final_state: bool = True, state_idx=None,
              snapshot_every: Optional[int] = None, output: bool = True):
    """Allocates ``o`` (and ``S_T``) and runs ``dr_decay_fwd``. Returns (o, S_T or None), plus the snapshots when
    ``snapshot_every`` is given. With ``state_idx``, S0 is a pool that is updated in place and returned as S_T.
    Rows of ``o`` past the last packed sequence are not written."""
    _ranks(q, v, alpha, 2)
    B, T, _, dk = q.shape
    H, dv = v.shape[-2:]
    N = B if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if state_idx is not None and S0 is None:
        raise ValueError("state_idx needs the pool of states as S0")
    S_T = None
    if state_idx is not None:
        S_T = S0
    elif output_final_state:
        S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device) if S0 is None else _like(S0)
    snaps = None
    if snapshot_every is not None:
        if cu_seqlens is None:
            lens = [T] * B
        elif _capturing():
            raise ValueError("snapshots of packed sequences need cu_seqlens on the host: not inside a graph capture")
        else:
            lens = check_offsets(cu_seqlens, T)
        snaps = torch.empty((snapshot_count(lens, snapshot_every), H, dk, dv), dtype=torch.float32, device=q.device)
    o = _like(v) if output else None
    dr_decay_fwd(q, k, v, alpha, S0, cu_seqlens, o, S_T, state_idx, snaps, snapshot_every or 0)
    return (o, S_T) if snapshot_every is None else (o, S_T, snaps)


def dr_decay_step(q, k, v, alpha, S, o, state_idx=None) -> None:
    """One token for each sequence, in place on ``S`` [N,H,dk,dv] fp32 (or, with ``state_idx`` [N] int32, on the rows
    it names of a pool); writes ``o`` [N,H,dv] fp32. q, k [N,Hk,dk]; v [N,H,dv]; alpha fp32 [N,H] or [H]."""
    lib = load_library()
    d = _inputs(q, k, v, alpha, 1)
    dev, N, H, dk, dv = q.device, d.batch, d.num_heads, d.head_dim_k, d.head_dim_v
    rows = N
    if state_idx is not None:
        _require(state_idx, "state_idx", (N,), torch.int32, dev)
        rows = S.shape[0]
    _require(S, "S", (rows, H, dk, dv), torch.float32, dev)
    _require(o, "o", (N, H, dv), torch.float32, dev)
    _call(lib, "dr_decay_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), S.data_ptr(),
          o.data_ptr(), ctypes.byref(d), _options(state_idx, rows))


def decay_step(q, k, v, alpha, S, state_idx=None):
    """Allocates ``o`` and runs ``dr_decay_step`` (S, or its rows ``state_idx``, updated in place). Returns o."""
    o = _like(v)
    dr_decay_step(q, k, v, alpha, S, o, state_idx)
    return o


def dr_decay_bwd(q, k, v, alpha, S0, cu_seqlens, dO, dS_T, dq, dk, dv, dalpha, dS0) -> None:
    """Gradients of ``dr_decay_fwd`` into caller-provided fp32 tensors: dq, dk [B,T,Hk,dk] (summed over the value heads
    that share them), dv [B,T,H,dv], dalpha in alpha's shape, dS0 [N,H,dk,dv] or None; dS_T may be None (zero)."""
    lib = load_library()
    d = _inputs(q, k, v, alpha, 2)
    dev, B, T, H, dk_, dv_ = q.device, d.batch, d.seqlen, d.num_heads, d.head_dim_k, d.head_dim_v
    _offsets(cu_seqlens, d, dev)
    for t, name in ((S0, "S0"), (dS_T, "dS_T"), (dS0, "dS0")):
        if t is not None:
            _require(t, name, (d.num_seqs, H, dk_, dv_), torch.float32, dev)
    for t, name, shape in ((dO, "dO", (B, T, H, dv_)), (dq, "dq", tuple(q.shape)), (dk, "dk", tuple(q.shape)),
                           (dv, "dv", (B, T, H, dv_)), (dalpha, "dalpha", tuple(alpha.shape))):
        _require(t, name, shape, torch.float32, dev)
    ws = _workspace(lib, d, dev, cu_seqlens is not None, True)
    _call(lib, "dr_decay_bwd", dev, *map(_addr, (q, k, v, alpha, S0, cu_seqlens, dO, dS_T, dq, dk, dv, dalpha, dS0)),
          ctypes.byref(d), _addr(ws), 0 if ws is None else ws.numel())


def decay_bwd(q, k, v, alpha, S0=None, cu_seqlens=None, dO=None, dS_T=None, need_dS0: bool = True):
    """Allocates the gradients and runs ``dr_decay_bwd``. Returns a dict with dq, dk, dv, dalpha and dS0 (None unless
    ``need_dS0``). Rows past the last packed sequence are not written."""
    _ranks(q, v, alpha, 2)
    dS0 = None
    if need_dS0 and S0 is not None:
        dS0 = _like(S0)
    elif need_dS0:
        N = q.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        dS0 = torch.empty((N, v.shape[2], q.shape[3], v.shape[3]), dtype=torch.float32, device=q.device)
    g = dict(dq=_like(q), dk=_like(k), dv=_like(v), dalpha=_like(alpha), dS0=dS0)
    dr_decay_bwd(q, k, v, alpha, S0, cu_seqlens, dO, dS_T, g["dq"], g["dk"], g["dv"], g["dalpha"], g["dS0"])
    return g


class _DecayAttention(torch.autograd.Function):
    """``decay_fwd`` as an autograd node; both directions are the library's kernels."""

    @staticmethod
    def forward(ctx, q, k, v, alpha, S0, cu_seqlens):
        ctx.set_materialize_grads(False)  # an output that the loss does not use gets no gradient
        N = q.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        # rows that no packed sequence holds are zeros, and so are their gradients
        new = torch.empty if cu_seqlens is None else torch.zeros
        o = new(tuple(v.shape), dtype=torch.float32, device=q.device)
        S_T = torch.empty((N, v.shape[2], q.shape[3], v.shape[3]), dtype=torch.float32, device=q.device)
        dr_decay_fwd(q, k, v, alpha, S0, cu_seqlens, o, S_T)
        ctx.save_for_backward(q, k, v, alpha, S0, cu_seqlens)
        return o, S_T

    @staticmethod
    @once_differentiable
    def backward(ctx, dO, dS_T):
        q, k, v, alpha, S0, cu_seqlens = ctx.saved_tensors
        new = torch.empty if cu_seqlens is None else torch.zeros
        like = lambda x: new(tuple(x.shape), dtype=torch.float32, device=x.device)  # noqa: E731
        dO = torch.zeros(tuple(v.shape), dtype=torch.float32, device=q.device) if dO is None else _dense(dO)
        dq, dk, dv, da = like(q), like(k), like(v), like(alpha)
        dS0 = torch.empty_like(S0) if S0 is not None and ctx.needs_input_grad[4] else None
        dr_decay_bwd(q, k, v, alpha, S0, cu_seqlens, dO, _dense(dS_T), dq, dk, dv, da, dS0)
        return dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype), da, dS0, None


def decay_attention(q, k, v, alpha, S0=None, cu_seqlens=None):
    """The prefill with gradients through torch autograd: returns (o, S_T) as ``decay_fwd``; ``backward()`` fills the
    ``.grad`` of q, k, v, alpha and S0 (gradients of bf16 inputs are computed in fp32 and returned in bf16). In a graph capture take forward and backward
    together, on leaves that no eager graph holds (torch would accumulate into those on the other stream)."""
    return _DecayAttention.apply(q, k, v, alpha, S0, cu_seqlens)


def _cache_dims(S, codes, scales, state_idx, slot_idx):
    if S.dim() != 4 or codes.dim() != 4:
        raise ValueError("S and codes must have 4 dimensions: rows, heads, d_k, d_v")
    dev = S.device
    rows, H, dk, dv = S.shape
    slots = codes.shape[0]
    fmt = 0 if codes.dtype is torch.int8 else 1 if codes.dtype is torch.float8_e4m3fn else None
    if fmt is None:
        raise ValueError(f"codes have dtype {codes.dtype}, expected int8 or float8_e4m3fn")
    _require(S, "S", (rows, H, dk, dv), torch.float32, dev)
    _require(codes, "codes", (slots, H, dk, dv), codes.dtype, dev)
    _require(scales, "scales", (slots, H, dk), torch.float32, dev)
    count = None
    for t, name in ((state_idx, "state_idx"), (slot_idx, "slot_idx")):
        if t is not None:
            if t.dim() != 1:
                raise ValueError(f"{name} must be a vector")
            _require(t, name, (t.shape[0] if count is None else count,), torch.int32, dev)
            count = t.shape[0]
    if count is None and rows != slots:
        raise ValueError(f"{rows} states and {slots} slots: give state_idx or slot_idx")
    return _CacheDims(rows if count is None else count, rows, slots, H, dk, dv, fmt, 0)


def dr_state_pack(S, codes, scales, slot_idx=None, state_idx=None) -> None:
    """Writes states ``S`` [R,H,dk,dv] fp32 (rows ``state_idx``) in 8 bits to the rows ``slot_idx`` of the cache:
    ``codes`` [P,H,dk,dv] int8 or float8_e4m3fn, ``scales`` [P,H,dk] fp32. A state row outside S is the zero state, a
    slot outside the cache is skipped; other slots are left as they are."""
    lib = load_library()
    d = _cache_dims(S, codes, scales, state_idx, slot_idx)
    _call(lib, "dr_state_pack", S.device, S.data_ptr(), _addr(state_idx), codes.data_ptr(), scales.data_ptr(),
          _addr(slot_idx), ctypes.byref(d))


def dr_state_unpack(codes, scales, S, slot_idx=None, state_idx=None) -> None:
    """Reads the rows ``slot_idx`` of the cache into the rows ``state_idx`` of ``S``: the inverse of
    ``dr_state_pack``. A slot outside the cache gives the zero state, a state row outside S is skipped."""
    lib = load_library()
    d = _cache_dims(S, codes, scales, state_idx, slot_idx)
    _call(lib, "dr_state_unpack", S.device, codes.data_ptr(), scales.data_ptr(), _addr(slot_idx), S.data_ptr(),
          _addr(state_idx), ctypes.byref(d))


def state_pack(S, fmt: str = "int8"):
    """``S`` [N,H,dk,dv] in 8 bits: (codes, scales), a cache of N slots."""
    if fmt not in CACHE_FORMATS:
        raise ValueError(f"unknown cache format {fmt!r}")
    codes = _like(S, CACHE_FORMATS[fmt][1])
    scales = torch.empty(tuple(S.shape[:-1]), dtype=torch.float32, device=S.device)
    dr_state_pack(S, codes, scales)
    return codes, scales


def state_unpack(codes, scales, slot_idx=None):
    """The states held by a cache (or by its rows ``slot_idx``), fp32."""
    rows = codes.shape[0] if slot_idx is None else slot_idx.shape[0]
    S = torch.empty((rows,) + tuple(codes.shape[1:]), dtype=torch.float32, device=codes.device)
    dr_state_unpack(codes, scales, S, slot_idx=slot_idx)
    return S
