"""Captured prefills and gradients of the gated delta rule: their workspace is the caller's (from Python torch's
allocator), never the library's pool, whose memory nodes two graphs must not hold."""
import ctypes

import pytest
import torch

import delta_rule_linear_chunked_amd as drl
import synth
from gpu_util import prefill_inputs, seed_of

pytestmark = pytest.mark.gpu


def workload(variant, packed, i):
    make = synth.make_prefill if variant != "product2" else lambda _, *a, **kw: synth.make_product("kda", *a, **kw)
    sizes = (1, 0) if packed else (2, 150)
    lengths = [70, 0, 130, 64] if packed else None
    return prefill_inputs(make(variant, *sizes, 2, 64, 64, in_dtype="bf16", seed=seed_of("ws", variant, i), lengths=lengths))


def fwd_args(a, o, S):
    return [a[n] for n in ("q", "k", "v", "alpha", "erase", "write")] + [a["variant"], a["S0"], a["cu_seqlens"], o, S]


@pytest.mark.parametrize("variant", ["kda", "gdn2", "product2"])
@pytest.mark.parametrize("packed", [False, True])
def test_two_graphs_of_prefill_and_backward_replayed_in_turn(variant, packed):
    xs = [workload(variant, packed, i) for i in range(2)]
    dO = torch.randn(xs[0]["q"].shape[:3] + (64,), device="cuda")

    def run(a):
        # prefill, gradients that form the states themselves, gradients from the prefill's checkpoints
        o = torch.zeros(a["q"].shape[:3] + (64,), device="cuda")
        N = a["S0"].shape[0]
        S = torch.zeros((N, 2, 64, 64), device="cuda")
        drl.dr_chunk_fwd(*fwd_args(a, o, S))
        kw = dict(S0=a["S0"], cu_seqlens=a["cu_seqlens"], dO=dO)
        args = [a[n] for n in ("q", "k", "v", "alpha", "erase", "write")] + [a["variant"]]
        g = drl.chunk_bwd(*args, **kw)
        out = dict(o=o, S=S, **{n: x for n, x in g.items() if x is not None})
        if not packed:
            ck = drl.chunk_fwd(*args, S0=a["S0"], snapshot_every=32 if variant == "product2" else 64)[2]
            g = drl.chunk_bwd(*args, checkpoints=ck, **kw)
            out.update({n + " from checkpoints": x for n, x in g.items() if x is not None})
        return out

    want = [{n: x.clone() for n, x in run(a).items()} for a in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(a))
        torch.cuda.synchronize()
        graphs.append(g)
    for r in range(3):
        for i in (0, 1):
            graphs[i].replay()
            eager = run(xs[1 - i])
            torch.cuda.synchronize()
            for n in want[i]:
                assert torch.equal(outs[i][n], want[i][n]), f"replay {r} of graph {i}: {n}"
                assert torch.equal(eager[n], want[1 - i][n]), f"eager {1 - i}: {n}"


def test_the_caller_s_workspace_of_the_stated_size_is_enough():
    # between guard bands, filled with NaN bits: the same bits as with the pool
    lib = drl.load_library()
    ptr = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    for packed in (False, True):
        a = workload("kda", packed, 3)
        B, T, H, _ = a["q"].shape
        N = a["S0"].shape[0]
        d = drl._Dims(B, T, H, 64, 64, N, 1, 0)
        dO = torch.randn(B, T, H, 64, device="cuda")
        ins = [ptr(a[n]) for n in ("q", "k", "v", "alpha", "erase", "write")] + [0, ptr(a["S0"]), ptr(a["cu_seqlens"])]
        got = []
        for own in (True, False):
            o, S = torch.zeros(B, T, H, 64, device="cuda"), torch.zeros(N, H, 64, 64, device="cuda")
            g = [torch.zeros(x.shape, device="cuda") for x in (a["q"], a["k"], a["v"], a["alpha"], a["erase"])]
            for kind in (0, 1):
                n = ctypes.c_int64()
                assert lib.dr_chunk_workspace(ctypes.byref(d), 0, int(packed), kind, ctypes.byref(n)) == 0
                buf = torch.full((n.value + (2 << 20),), 255, dtype=torch.uint8, device="cuda")
                ws = (None, 0) if own else (buf.data_ptr() + (1 << 20), n.value)
                stream = torch.cuda.current_stream().cuda_stream
                if kind:
                    st = lib.dr_chunk_bwd_ws(*ins, ptr(dO), None, *map(ptr, g), None, None, None, ctypes.byref(d), *ws, stream)
                else:
                    st = lib.dr_chunk_fwd_ws(*ins, ptr(o), ptr(S), ctypes.byref(d), None, *ws, stream)
                assert st == 0, lib.dr_last_error()
                torch.cuda.synchronize()
                assert (buf[:1 << 20] == 255).all() and (buf[(1 << 20) + n.value:] == 255).all()
            got.append([o, S] + g)
        assert all(torch.equal(x, y) for x, y in zip(*got))


def test_a_captured_call_without_a_workspace_is_refused():
    lib = drl.load_library()
    a = workload("kda", False, 4)
    B, T, H, _ = a["q"].shape
    d = drl._Dims(B, T, H, 64, 64, B, 1, 0)
    o = torch.zeros(B, T, H, 64, device="cuda")
    g = [torch.zeros(x.shape, device="cuda") for x in (a["q"], a["k"], a["v"], a["alpha"], a["erase"])]
    ins = [x if x is None or isinstance(x, int) else x.data_ptr()
           for x in [a[n] for n in ("q", "k", "v", "alpha", "erase", "write")] + [0, a["S0"], None]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stream = torch.cuda.current_stream().cuda_stream
        one = lib.dr_chunk_fwd_ex(*ins, o.data_ptr(), None, ctypes.byref(d), None, stream)
        said = lib.dr_last_error()
        two = lib.dr_chunk_bwd_ex(*ins, o.data_ptr(), None, *[x.data_ptr() for x in g], None, None, None, ctypes.byref(d), stream)
        o.add_(1.0)  # (a graph with no node in it makes torch warn)
    assert one == two == -5 and b"workspace" in said and b"workspace" in lib.dr_last_error()
