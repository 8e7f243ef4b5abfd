"""The decayed linear attention and the state cache as a program uses them: captured graphs, several streams and
threads, rows guarded on both sides, and a serving run of all of them together."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from delta_rule_linear_chunked_amd import _decay
from decay_util import close, dev, make, oracle, tensors
from gpu_util import seed_of

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "alpha")


def i32(x):
    return dev(np.asarray(x, np.int32))


def call_lib(entry, args, d, ws, nbytes, opts=()):
    lib = drl.load_library()
    ptr = [None if a is None else a.data_ptr() for a in args]
    return getattr(lib, entry)(*ptr, ctypes.byref(d), *opts, ws, nbytes, torch.cuda.current_stream().cuda_stream)


def need(d, packed, backward):
    n = ctypes.c_int64()
    assert drl.load_library().dr_decay_workspace(ctypes.byref(d), packed, backward, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("seg", [0, 64])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_a_workspace_of_the_stated_size_is_enough(seg, packed, decay, monkeypatch):
    # the caller's workspace between guard bands, filled with NaN bits before the call; the same results as with the
    # library's own pool
    if seg:
        monkeypatch.setenv("DR_DECAY_SEG", str(seg))
    T, H, Hk, dk, dv = 200, 4, 2, 32, 64
    cu = i32([0, 70, 70, 71, 199]) if packed else None
    x = make(seed_of("space", seg, packed, decay), 1, T, H, Hk, dk, dv, "bf16", decay, n=4 if packed else 1)
    t = tensors(x, "bf16")
    N = t["S0"].shape[0]
    d = _decay._DecayDims(1, T, H, Hk, dk, dv, N, 1, int(decay == "head"), 0, 0)
    dO = torch.randn(1, T, H, dv, device="cuda")
    outs = []
    for own in (False, True):
        o, S = torch.zeros(1, T, H, dv, device="cuda"), torch.zeros(N, H, dk, dv, device="cuda")
        g = [torch.zeros(tuple(a.shape), device="cuda") for a in (t["q"], t["k"], t["v"], t["alpha"], t["S0"])]
        ins = [t[n] for n in NAMES] + [t["S0"], cu]
        for entry, args, backward, opts in (("dr_decay_fwd", ins + [o, S], 0, (None,)), ("dr_decay_bwd", ins + [dO, None] + g, 1, ())):
            n = need(d, int(packed), backward)
            buf = torch.full((n + (2 << 20),), 255, dtype=torch.uint8, device="cuda")
            assert call_lib(entry, args, d, None if own or not n else buf.data_ptr() + (1 << 20), 0 if own else n, opts) == 0
            torch.cuda.synchronize()
            assert (buf[:1 << 20] == 255).all() and (buf[(1 << 20) + n:] == 255).all()
        outs.append([o, S] + g)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_several_threads_and_streams():
    # each thread on a stream of its own, its calls repeated; every result equals the call made alone
    cases = []
    for i, (T, H, Hk, dk, dv, dtype) in enumerate([(1300, 2, 1, 64, 64, "bf16"), (700, 3, 3, 32, 16, "f32"),
                                                   (2000, 2, 2, 128, 128, "bf16"), (65, 4, 2, 16, 32, "f32")]):
        t = tensors(make(50 + i, 2, T, H, Hk, dk, dv, dtype, "token"), dtype)
        t["dO"] = torch.randn_like(t["v"], dtype=torch.float32)
        cases.append(t)

    def run(t):
        o, S = drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"])
        g = drl.decay_bwd(*[t[n] for n in NAMES], S0=t["S0"], dO=t["dO"])
        return [o, S, drl.state_unpack(*drl.state_pack(S, "e4m3"))] + list(g.values())

    want = [run(t) for t in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                got = run(cases[i])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
                    return

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 63, 130])
def test_nothing_outside_the_outputs_is_written(T, dtype):
    # every output lies between guard bands
    x = make(seed_of("guards", T, dtype), 2, T, 3, 3, 32, 16, dtype, "token")
    t = tensors(x, dtype)
    bands = []

    def guarded(shape):
        n = int(np.prod(shape))
        buf = torch.full((n + 4096,), 7.0, device="cuda")
        bands.append((buf, n))
        return buf[2048:2048 + n].view(shape)

    o, S = guarded((2, T, 3, 16)), guarded((2, 3, 32, 16))
    snaps = guarded((2 * (T // 64), 3, 32, 16)) if T >= 64 else None
    drl.dr_decay_fwd(*[t[n] for n in NAMES], t["S0"], None, o, S, snapshots=snaps, snapshot_every=64)
    g = [guarded(s) for s in (x["q"].shape, x["k"].shape, x["v"].shape, x["alpha"].shape, x["S0"].shape)]
    drl.dr_decay_bwd(*[t[n] for n in NAMES], t["S0"], None, torch.randn(2, T, 3, 16, device="cuda"), None, *g)
    one = [t[n][:, 0].contiguous() for n in NAMES]
    drl.dr_decay_step(*one, S, guarded((2, 3, 16)))
    drl.dr_state_unpack(*drl.state_pack(S), guarded((2, 3, 32, 16)))
    torch.cuda.synchronize()
    for buf, n in bands:
        assert (buf[:2048] == 7.0).all() and (buf[2048 + n:] == 7.0).all()


def test_serving_run():
    # four users: a shared prefix of 128 tokens prefilled once with snapshots, parked in the cache, resumed into the
    # users' slots, each with a prompt of its own (packed), then decoded token by token; against one long evaluation
    # from the values that the cache holds
    H, Hk, d, users, steps = 4, 2, 64, 4, 6
    x = make(60, 1, 128, H, Hk, d, d, "bf16", "token", s0=False)
    t = tensors(x, "bf16")
    _, _, snaps = drl.decay_fwd(*[t[n] for n in NAMES], snapshot_every=64)
    codes = torch.zeros(5, H, d, d, dtype=torch.int8, device="cuda")
    scales = torch.zeros(5, H, d, device="cuda")
    drl.dr_state_pack(snaps, codes, scales, slot_idx=i32([4, 2]))
    pool = torch.full((6, H, d, d), 9.0, device="cuda")
    rows = [5, 0, 3, 1]
    drl.dr_state_unpack(codes, scales, pool, slot_idx=i32([2] * users), state_idx=i32(rows))
    held = oracle.pack(snaps[1:].cpu().numpy(), "int8")[0].astype(np.float32)
    cu = [0, 30, 31, 131, 190]
    y = make(61, 1, 190, H, Hk, d, d, "bf16", "token", s0=False)
    u = tensors(y, "bf16")
    o, pool = drl.decay_fwd(*[u[n] for n in NAMES], S0=pool, cu_seqlens=i32(cu), state_idx=i32(rows))
    z = make(62, steps, users, H, Hk, d, d, "bf16", "token", s0=False)
    w = tensors(z, "bf16")
    outs = [drl.decay_step(*[w[n][s] for n in NAMES], pool, state_idx=i32(rows)) for s in range(steps)]
    for n in range(users):
        seq = [np.concatenate([y[m][:, cu[n]:cu[n + 1]], z[m][:, n][None]], 1) for m in NAMES]
        want, wS = oracle.forward(*seq, held)
        mo, mS = oracle.forward(*seq, held, magnitudes=True)
        L = cu[n + 1] - cu[n]
        close(o[0, cu[n]:cu[n + 1]], want[0, :L], mo[0, :L], 190, f"prompt {n}")
        for s in range(steps):
            close(outs[s][n], want[0, L + s], mo[0, L + s], 190 + 64 * steps, f"user {n} step {s}")
        close(pool[rows[n]], wS[0], mS[0], 190 + 64 * steps, f"state {n}")
    assert (pool[[2, 4]] == 9.0).all()


def test_training_step_beside_the_delta_rule():
    # a layer whose output mixes both recurrences, its loss differentiated through both autograd nodes
    B, T, H, d = 2, 96, 2, 32
    x = make(63, B, T, H, H, d, d, "f32", "token")
    leaves = {n: a.requires_grad_() for n, a in tensors(x, "f32").items()}
    beta = torch.full((B, T, H), 0.5, device="cuda")
    wide = leaves["alpha"][..., None].expand(B, T, H, d).contiguous()
    o1, _ = drl.decay_attention(*[leaves[n] for n in NAMES], leaves["S0"])
    o2, _ = drl.delta_rule(leaves["q"], leaves["k"], leaves["v"], wide, beta, variant="kda")
    w = torch.randn_like(o1)
    ((o1 + o2) * w).sum().backward()
    g = drl.decay_bwd(*[leaves[n].detach() for n in NAMES], S0=leaves["S0"].detach(), dO=w)
    e = drl.chunk_bwd(leaves["q"].detach(), leaves["k"].detach(), leaves["v"].detach(), wide.detach(), beta, variant="kda", dO=w)
    assert torch.equal(leaves["v"].grad, g["dv"] + e["dv"]) or torch.allclose(leaves["v"].grad, g["dv"] + e["dv"], rtol=1e-6, atol=1e-6)
    # two gradients summed by autograd in either order, each rounded once more
    want = g["dalpha"] + e["dalpha"].sum(-1)
    assert (leaves["alpha"].grad - want).abs().max() <= 64 * 2.0 ** -24 * (g["dalpha"].abs() + e["dalpha"].abs().sum(-1)).max()
    assert torch.equal(leaves["S0"].grad, g["dS0"])


def test_calls_run_on_the_callers_stream():
    x = make(64, 1, 40, 2, 2, 32, 32, "f32", "token")
    t = tensors(x, "f32")
    want = drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"])[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"])[0]
        doubled = got * 2  # ordered behind the call on the same stream
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(doubled, want * 2)


def test_a_captured_call_without_a_workspace_is_refused():
    x = make(65, 1, 100, 2, 2, 32, 32, "bf16", "token")
    t = tensors(x, "bf16")
    d = _decay._DecayDims(1, 100, 2, 2, 32, 32, 1, 1, 0, 0, 0)
    g = [torch.zeros(tuple(a.shape), device="cuda") for a in (t["q"], t["k"], t["v"], t["alpha"], t["S0"])]
    dO = torch.randn(1, 100, 2, 32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = call_lib("dr_decay_bwd", [t[n] for n in NAMES] + [t["S0"], None, dO, None] + g, d, None, 0)
        dO.add_(1.0)  # (a graph with no node in it makes torch warn)
    assert st == -5 and b"workspace" in drl.load_library().dr_last_error()


def test_step_and_cache_in_a_graph():
    x = make(41, 1, 6, 4, 2, 64, 64, "bf16", "token", n=8)
    t = tensors(x, "bf16")
    q, k, v, a = (t[n][0] for n in NAMES)
    idx, slots = i32([7, 0, 3, 5, 1, 2]), i32([1, 2, 0, 4, 3, 5])
    pool, back = t["S0"].clone(), torch.zeros_like(t["S0"])
    codes, scales = drl.state_pack(pool)

    def run():
        o = drl.decay_step(q, k, v, a, pool, state_idx=idx)
        drl.dr_state_pack(pool, codes, scales, slot_idx=slots, state_idx=idx)
        drl.dr_state_unpack(codes, scales, back, slot_idx=slots, state_idx=idx)
        return o

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = run()
    pool.copy_(t["S0"])
    S = t["S0"].clone()
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        want = drl.decay_step(q, k, v, a, S, state_idx=idx)
        held = drl.state_unpack(*drl.state_pack(S[idx.long()]))
        assert torch.equal(o, want) and torch.equal(pool, S) and torch.equal(back[idx.long()], held), i


@pytest.mark.parametrize("packed", [False, True])
def test_two_graphs_replayed_among_eager_calls(packed):
    # prefill (in segments: it takes a workspace) and backward captured twice, for two inputs; replays of both in
    # turn, with eager calls and synchronisations between them
    T = 1500
    cu = i32([0, 700, 701, T - 3]) if packed else None
    xs = [tensors(make(seed_of("graph", packed, i), 1, T, 2, 1, 64, 64, "bf16", "token", n=3 if packed else 1), "bf16") for i in range(2)]
    dO, dS = torch.randn_like(xs[0]["v"], dtype=torch.float32), torch.randn_like(xs[0]["S0"])

    def run(t):
        out = dict(zip(("o", "S"), drl.decay_fwd(*[t[n] for n in NAMES], S0=t["S0"], cu_seqlens=cu)))
        return {**out, **drl.decay_bwd(*[t[n] for n in NAMES], S0=t["S0"], cu_seqlens=cu, dO=dO, dS_T=dS)}

    want = [{n: a.clone() for n, a in run(t).items()} for t in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(t))
        torch.cuda.synchronize()
        graphs.append(g)
    end = T - 3 if packed else T
    cut = lambda n, a: a[:, :end] if n not in ("S", "dS0") else a  # noqa: E731
    for _ in range(3):
        for i in (0, 1):
            graphs[i].replay()
            eager = run(xs[1 - i])
            torch.cuda.synchronize()
            for n in want[i]:
                assert torch.equal(cut(n, outs[i][n]), cut(n, want[i][n])), f"graph {i}: {n}"
                assert torch.equal(cut(n, eager[n]), cut(n, want[1 - i][n])), f"eager {1 - i}: {n}"


def test_captured_gradients():
    # forward and backward through autograd in one graph, on leaves of their own
    x = make(66, 2, 150, 4, 2, 32, 64, "bf16", "token")
    leaves = [a.requires_grad_() for a in tensors(x, "bf16").values()]
    w, wS = torch.randn(2, 150, 4, 64, device="cuda"), torch.randn(2, 4, 32, 64, device="cuda")

    def run():
        return torch.autograd.grad(drl.decay_attention(*leaves), leaves, (w, wS))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [a.clone() for a in run()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    torch.cuda.synchronize()
    for r in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {r}"
        again = [a.detach().requires_grad_() for a in leaves]  # eager work between the replays
        eager = torch.autograd.grad(drl.decay_attention(*again), again, (w, wS))
        assert all(torch.equal(a, b) for a, b in zip(eager, want)), f"eager {r}"


def test_second_derivatives_are_refused():
    x = make(67, 1, 20, 2, 2, 16, 16, "f32", "token")
    leaves = [a.requires_grad_() for a in tensors(x, "f32").values()]
    o, _ = drl.decay_attention(*leaves)
    g, = torch.autograd.grad(o.square().sum(), leaves[:1], create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_offsets_past_32_bits(monkeypatch):
    # 2^31 elements of v, of the outputs and of the pool lie before what is checked: the last tokens of a long row that
    # is zero up to them, and the last slots of a pool
    H, Hk, d, tail = 128, 2, 128, 150
    T = 64 * 2049 + tail
    x = make(70, 1, tail, H, Hk, d, d, "bf16", "token", s0=False)
    t = tensors(x, "bf16")
    big = {n: torch.zeros((1, T) + tuple(t[n].shape[2:]), dtype=t[n].dtype, device="cuda") for n in NAMES}
    for n in NAMES:
        big[n][:, T - tail:] = t[n]
    assert big["v"].numel() - tail * H * d > 2 ** 31
    heads = [0, 1, H - 1]
    pick = lambda a, hk: a[:, :, [h // (H // Hk) for h in heads]] if hk else a[:, :, heads]  # noqa: E731
    small = [pick(x["q"], True), pick(x["k"], True), pick(x["v"], False), pick(x["alpha"], False)]
    zero = np.zeros((1, len(heads), d, d), np.float32)
    o, S = drl.decay_fwd(*[big[n] for n in NAMES])
    want, wS = oracle.forward(*small, zero)
    mo, mS = oracle.forward(*small, zero, magnitudes=True)
    close(o[:, T - tail:, heads], want, mo, tail, "o")
    close(S[:, heads], wS, mS, tail, "S")
    del o
    dO = torch.zeros(1, T, H, d, device="cuda")
    dO[:, T - tail:] = torch.randn(1, tail, H, d, device="cuda")
    monkeypatch.setenv("DR_DECAY_SEG", str(1 << 20))  # one segment: the tail's chunks are then the same work in both
    g = drl.decay_bwd(*[big[n] for n in NAMES], dO=dO)
    part = drl.decay_bwd(*[t[n] for n in NAMES], S0=torch.zeros(1, H, d, d, device="cuda"), dO=dO[:, T - tail:].contiguous())
    for n in ("dv", "dq", "dk", "dalpha"):
        assert torch.equal(g[n][:, T - tail:], part[n]), n
        assert (g[n][:, :T - tail] == 0).all(), n
    del g, dO, big
    slots = 4 + 2 ** 31 // (32 * d * d)
    pool = torch.zeros(slots, 32, d, d, device="cuda")
    idx = i32([slots - 1, 0, slots - 2])
    y = make(71, 1, 3, 32, 32, d, d, "bf16", "token", n=3)
    u = tensors(y, "bf16")
    pool[idx.long()] = u["S0"]
    one = [u[n][0] for n in NAMES]
    S1 = u["S0"].clone()
    assert torch.equal(drl.decay_step(*one, pool, state_idx=idx), drl.decay_step(*one, S1))
    assert torch.equal(pool[idx.long()], S1)
    codes = torch.zeros(slots, 32, d, d, dtype=torch.int8, device="cuda")
    scales = torch.zeros(slots, 32, d, device="cuda")
    drl.dr_state_pack(pool, codes, scales, slot_idx=idx, state_idx=idx)
    back = torch.zeros(3, 32, d, d, device="cuda")
    drl.dr_state_unpack(codes, scales, back, slot_idx=idx, state_idx=i32([0, 1, 2]))
    assert torch.equal(back, drl.state_unpack(*drl.state_pack(S1)))
