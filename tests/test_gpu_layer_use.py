"""The norm, the convolution and the selective scan as a program uses them: captured graphs, several streams and threads,
guarded memory, large offsets, and a serving and a training run of all of them together."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from delta_rule_linear_chunked_amd import _scan
from gpu_util import seed_of
from layer_util import CONV_K, SCAN_IN, close, dev, i32, make_conv, make_scan, oracle, scan_k, scan_slack, scan_tensors

pytestmark = pytest.mark.gpu
GRADS = {"dx": "x", "ddt": "dt", "dA": "A", "dB": "B", "dC": "C", "dD": "D", "dz": "z", "ddt_bias": "bias", "dS0": "S0"}


class Layer:
    """Inputs of the three operators and every call of them, forward and backward, with a workspace of the caller's choice."""

    def __init__(self, seed, T, C, N, dtype, cu=None, rows=40):
        n = 1 if cu is None else len(cu) - 1
        self.scan = scan_tensors(make_scan(seed, 1, T, C, 1, N, dtype, n=n), dtype)
        c = make_conv(seed + 1, 1, T, C, 4, dtype, n=n)
        self.conv = {k: dev(v, "f32" if k in "wb" else dtype) for k, v in c.items()}
        r = np.random.default_rng(seed + 2)
        self.norm = {k: dev(r.standard_normal((rows, C)), dtype) for k in ("x", "r", "dy", "dh")}
        self.norm["w"] = dev(r.standard_normal(C))
        self.cu = None if cu is None else i32(cu)
        self.end = T if cu is None else cu[-1]

    def run(self, new=torch.zeros_like):
        """All calls through the binding (torch's allocator for workspaces); ``new(tensor)`` makes an output like it."""
        s, c, m, out = self.scan, self.conv, self.norm, {}
        out["scan y"], out["scan S"] = new(s["x"]), new(s["S0"])
        drl.dr_scan_fwd(*[s[k] for k in SCAN_IN], s["S0"], self.cu, out["scan y"], out["scan S"])
        g = {k: new(s[v]) for k, v in GRADS.items()}
        drl.dr_scan_bwd(*[s[k] for k in SCAN_IN], s["S0"], self.cu, s["dy"], s["dS"], *g.values())
        out.update({"scan " + k: v for k, v in g.items()})
        out["conv y"], out["conv S"] = new(c["x"]), new(c["state"])
        drl.dr_conv_fwd(c["x"], c["w"], c["b"], c["state"], self.cu, out["conv y"], out["conv S"])
        g = {k: new(c[v]) for k, v in dict(dx="x", dw="w", db="b", dstate="state").items()}
        drl.dr_conv_bwd(c["x"], c["w"], c["b"], c["state"], self.cu, c["dy"], c["dl"], *g.values())
        out.update({"conv " + k: v for k, v in g.items()})
        out["norm y"], out["norm h"] = new(m["x"]), new(m["x"])
        drl.dr_norm_fwd(m["x"], m["r"], m["w"], out["norm y"], None, out["norm h"])
        out["norm dx"], out["norm dw"] = new(m["x"]), new(m["w"])
        drl.dr_norm_bwd(out["norm h"], m["w"], m["dy"], m["dh"], out["norm dx"], out["norm dw"])
        return out

    def rows(self, out):
        """The outputs without the rows that no sequence holds."""
        return {k: v[:, :self.end] if k[:4] != "norm" and v.dim() > 2 and v.shape[1] == self.scan["x"].shape[1] else v for k, v in out.items()}


def same(a, b, what=""):
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), f"{what} {k}"


def call_lib(entry, args, d, ws, nbytes, opts=()):
    ptr = [None if a is None else a.data_ptr() for a in args]
    return getattr(drl.load_library(), entry)(*ptr, ctypes.byref(d), *opts, ws, nbytes, torch.cuda.current_stream().cuda_stream)


def need(entry, d, *args):
    n = ctypes.c_int64()
    assert getattr(drl.load_library(), entry)(ctypes.byref(d), *args, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("seg", [0, 16])
@pytest.mark.parametrize("cu", [None, [0, 70, 70, 71, 147]])
@pytest.mark.parametrize("N", [16, 64])
def test_a_workspace_of_the_stated_size_is_enough(N, cu, seg, monkeypatch):
    # the caller's workspace between guard bands, filled with NaN bits before the call; the same results as with the
    # library's own pool
    if seg:
        monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    T, C = 150, 72
    L = Layer(seed_of("space", N, cu, seg), T, C, N, "bf16", cu)
    s, c, m, packed = L.scan, L.conv, L.norm, int(cu is not None)
    ds = _scan._scan_inputs(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], True, 2)
    dc = _scan._conv_inputs(c["x"], c["w"], c["b"], "silu", 2)
    ds.num_seqs = dc.num_seqs = s["S0"].shape[0]
    dn = _scan._norm_dims(m["x"], m["w"], None, 1e-5, 0)
    outs = []
    for own in (False, True):
        y, S = torch.zeros_like(s["x"]), torch.zeros_like(s["S0"])
        g = [torch.zeros_like(s[v]) for v in GRADS.values()]
        gc = [torch.zeros_like(c[v]) for v in ("x", "w", "b", "state")]
        gn = [torch.zeros_like(m["x"]), torch.zeros_like(m["w"])]
        ins = [s[k] for k in SCAN_IN] + [s["S0"], L.cu]
        for entry, args, d, n, opts in (
                ("dr_scan_fwd", ins + [y, S], ds, need("dr_scan_workspace", ds, packed, 0), (None,)),
                ("dr_scan_bwd", ins + [s["dy"], s["dS"]] + g, ds, need("dr_scan_workspace", ds, packed, 1), ()),
                ("dr_conv_bwd", [c["x"], c["w"], c["b"], c["state"], L.cu, c["dy"], c["dl"]] + gc, dc, need("dr_conv_workspace", dc, packed), ()),
                ("dr_norm_bwd", [m["x"], m["w"], m["dy"], m["dh"]] + gn, dn, need("dr_norm_workspace", dn), ())):
            buf = torch.full((n + (2 << 20),), 255, dtype=torch.uint8, device="cuda")
            assert call_lib(entry, args, d, None if own or not n else buf.data_ptr() + (1 << 20), 0 if own else n, opts) == 0, entry
            torch.cuda.synchronize()
            assert (buf[:1 << 20] == 255).all() and (buf[(1 << 20) + n:] == 255).all(), entry
        outs.append([y, S] + g + gc + gn)
    for i, (a, b) in enumerate(zip(*outs)):
        assert torch.equal(a, b) and not torch.isnan(a).any(), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,C", [(1, 1), (9, 65), (33, 264)])
def test_nothing_outside_the_outputs_is_written(T, C, dtype):
    # every output lies between guard bands, and every element of it is written
    bands = []

    def guarded(like):
        n = like.numel()
        buf = torch.full((n + 4096,), float("nan"), device="cuda", dtype=like.dtype)
        bands.append((buf, n))
        return buf[2048:2048 + n].view(like.shape)

    L = Layer(seed_of("guards", T, C, dtype), T, C, 16, dtype)
    L.run(guarded)
    m, one = L.norm, {k: (L.scan[k] if k in ("A", "D", "bias") else L.scan[k][:, 0]) for k in SCAN_IN}
    S, e = guarded(L.scan["S0"]), guarded(L.conv["state"])
    S.copy_(L.scan["S0"])
    e.copy_(L.conv["state"])
    drl.dr_scan_step(*one.values(), S, guarded(one["x"]))
    drl.dr_conv_step(L.conv["x"][:, 0], L.conv["w"], L.conv["b"], e, guarded(one["x"]))
    for fmt in (torch.int8, torch.float8_e4m3fn):
        buf = torch.full((m["x"].numel() + 4096,), 77, dtype=torch.uint8, device="cuda")
        codes = buf[2048:2048 + m["x"].numel()].view(fmt).view(m["x"].shape)
        drl.dr_norm_fwd(m["x"], m["r"], m["w"], codes, guarded(m["x"][:, 0].float()), guarded(m["x"]))
        torch.cuda.synchronize()
        assert (buf[:2048] == 77).all() and (buf[2048 + m["x"].numel():] == 77).all()
    torch.cuda.synchronize()
    for i, (buf, n) in enumerate(bands):
        assert buf[:2048].isnan().all() and buf[2048 + n:].isnan().all() and not buf[2048:2048 + n].isnan().any(), i


def test_several_threads_and_streams():
    # each thread on a stream of its own, its calls repeated; every result equals the call made alone
    cases = [Layer(50, 900, 128, 16, "bf16"), Layer(60, 300, 65, 32, "f32", [0, 100, 100, 290]), Layer(70, 64, 520, 64, "bf16", [0, 1, 64]),
             Layer(80, 40, 3, 16, "f32")]
    want = [L.rows(L.run()) for L in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                got = cases[i].rows(cases[i].run())
                s.synchronize()
                if not all(torch.equal(got[k], want[i][k]) for k in got):
                    wrong.append(i)
                    return

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_calls_run_on_the_callers_stream():
    L = Layer(90, 200, 72, 16, "bf16")
    want = {k: v * 2 for k, v in L.run().items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        doubled = {k: v * 2 for k, v in L.run().items()}  # ordered behind the calls on the same stream
    torch.cuda.current_stream().wait_stream(s)
    same(doubled, want)


@pytest.mark.parametrize("cu", [None, [0, 350, 351, 697]])
def test_two_graphs_replayed_among_eager_calls(cu, monkeypatch):
    # all calls, the scan in segments (with a workspace), captured twice for two inputs; replays of both in turn, with
    # eager calls and synchronisations between them
    monkeypatch.setenv("DR_SCAN_SEG", "64")
    layers = [Layer(seed_of("graph", cu, i), 700, 72, 16, "bf16", cu) for i in range(2)]
    want = [L.rows({k: v.clone() for k, v in L.run().items()}) for L in layers]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for L in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(L.rows(L.run()))
        torch.cuda.synchronize()
        graphs.append(g)
    for r in range(3):
        for i in (0, 1):
            for v in outs[i].values():
                v.zero_()
            graphs[i].replay()
            eager = layers[1 - i].rows(layers[1 - i].run())
            torch.cuda.synchronize()
            same(outs[i], want[i], f"replay {r} of graph {i}")
            same(eager, want[1 - i], f"eager call {r} beside graph {i}")


def test_a_captured_call_without_a_workspace_is_refused():
    L = Layer(91, 100, 64, 16, "bf16")
    m = L.norm
    d = _scan._norm_dims(m["x"], m["w"], None, 1e-5, 0)
    out = [torch.zeros_like(m["x"]), torch.zeros_like(m["w"])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = call_lib("dr_norm_bwd", [m["x"], m["w"], m["dy"], None] + out, d, None, 0)
        out[1].add_(1.0)  # (a graph with no node in it makes torch warn)
    assert st == -5 and b"workspace" in drl.load_library().dr_last_error()


def test_captured_gradients():
    # forward and backward through autograd in one graph, on leaves of their own
    L = Layer(92, 150, 72, 16, "bf16")
    s, c, m = L.scan, L.conv, L.norm
    leaves = [a.detach().clone().requires_grad_() for a in (m["x"], m["w"], c["w"], c["b"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"])]

    def run(v):
        y = drl.rms_norm(v[0], v[1]).view(1, -1, 72)
        x, _ = drl.causal_conv(y, v[2], v[3])
        o, _ = drl.selective_scan(x, v[4][:, :40], v[5], v[6][:, :40], v[7][:, :40], v[8], v[9][:, :40], v[10])
        return torch.autograd.grad(o, v, s["dy"][:, :40])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [a.clone() for a in run(leaves)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(leaves)
    torch.cuda.synchronize()
    for r in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {r}"
        eager = run([a.detach().requires_grad_() for a in leaves])  # eager work between the replays
        assert all(torch.equal(a, b) for a, b in zip(eager, want)), f"eager {r}"


def test_gradients_that_are_parts_of_larger_tensors():
    # what arrives at the nodes is a transposed view, an expanded scalar, and nothing
    L = Layer(93, 30, 72, 16, "f32")
    s, c, m = L.scan, L.conv, L.norm
    wide = torch.randn(1, 72, 30, device="cuda")
    leaves = [s[k].detach().requires_grad_() for k in SCAN_IN]
    (drl.selective_scan(*leaves)[0].transpose(1, 2) * wide).sum().backward()
    g = drl.scan_bwd(*[s[k] for k in SCAN_IN], dy=wide.transpose(1, 2).contiguous())
    for leaf, n in zip(leaves, ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")):
        assert torch.equal(leaf.grad, g[n]), n
    x, w = c["x"].detach().requires_grad_(), c["w"].detach().requires_grad_()
    drl.causal_conv(x, w)[0].sum().backward()
    g = drl.conv_bwd(c["x"], c["w"], dy=torch.ones_like(c["x"]))
    assert torch.equal(x.grad, g["dx"]) and torch.equal(w.grad, g["dweight"])
    x, r, w = (m[k].detach().requires_grad_() for k in ("x", "r", "w"))
    drl.rms_norm(x, w, r)[1].sum().backward()  # only the sum is used
    assert (x.grad == 1).all() and (r.grad == 1).all() and not w.grad.any()
    x.grad.add_(1)
    assert (r.grad == 1).all()  # (gradients of their own)
    # inputs that are one row for every token: their gradient is the sum
    one = torch.randn(1, 1, 1, 16, device="cuda", requires_grad=True)
    drl.selective_scan(s["x"], s["dt"], s["A"], one.expand(1, 30, 1, 16), s["C"])[0].sum().backward()
    g = drl.scan_bwd(s["x"], s["dt"], s["A"], one.detach().expand(1, 30, 1, 16).contiguous(), s["C"], dy=torch.ones_like(s["x"]))
    assert torch.equal(one.grad, g["dB"].sum(1, keepdim=True))


def test_second_derivatives_are_refused():
    L = Layer(94, 20, 64, 16, "f32")
    s, c, m = L.scan, L.conv, L.norm
    for f, ins in ((lambda *a: drl.selective_scan(*a)[0], [s[k] for k in SCAN_IN]), (lambda *a: drl.causal_conv(*a)[0], [c["x"], c["w"]]),
                   (drl.rms_norm, [m["x"], m["w"]])):
        leaves = [a.detach().requires_grad_() for a in ins]
        g, = torch.autograd.grad(f(*leaves).square().sum(), leaves[:1], create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_sequence(value):
    # one such input in the second of three packed sequences: the outputs, states and gradients of the others, and of the other
    # channels (but for the sums over channels), are the same bits
    cu, C, at, ch = [0, 21, 50, 75], 72, 30, 5
    L = Layer(95, 75, C, 16, "f32", cu)
    clean = L.run()
    for t in (L.scan["x"], L.conv["x"]):
        t[0, at, ch] = value
    dirty = L.run()
    others = [c for c in range(C) if c != ch]
    for k in clean:
        if k[:4] == "norm":
            continue
        a, b = clean[k], dirty[k]
        if a.dim() > 1 and a.shape[1] == 75:
            assert torch.equal(a[:, :21], b[:, :21]) and torch.equal(a[:, 50:], b[:, 50:]), k
            if a.shape[-1] == C:
                assert torch.equal(a[..., others], b[..., others]), k
        elif a.shape[0] == 3:  # states
            assert torch.equal(a[[0, 2]], b[[0, 2]]), k
    assert torch.isnan(dirty["scan y"][0, at:50, ch]).all() and not torch.isfinite(dirty["conv y"][0, at, ch])
    assert torch.equal(clean["scan y"][0, 21:at - 1], dirty["scan y"][0, 21:at - 1])


@pytest.mark.parametrize("B,T", [(0, 3), (2, 0)])
def test_no_tokens(B, T):
    # nothing to read: the states pass through, the gradients of parameters are zeros
    N, C = 16, 40
    t = scan_tensors(make_scan(1, 2, 3, C, 1, N, "f32"), "f32")
    v = {k: (t[k] if k in ("A", "D", "bias") else t[k][:B, :T].contiguous()) for k in SCAN_IN}
    S0 = t["S0"][:B].contiguous()
    y, S = drl.scan_fwd(*v.values(), S0=S0)
    assert y.shape == (B, T, C) and torch.equal(S, S0)
    g = drl.scan_bwd(*v.values(), S0=S0, dy=v["x"], dS_T=S0)
    assert torch.equal(g["dS0"], S0) and not any(g[k].any() for k in ("dA", "dD", "ddt_bias"))
    c = {k: dev(a) for k, a in make_conv(2, 2, 3, C, 4, "f32").items()}
    x, e = c["x"][:B, :T].contiguous(), c["state"][:B].contiguous()
    y, last = drl.conv_fwd(x, c["w"], c["b"], e)
    assert y.shape == (B, T, C) and torch.equal(last, e)
    g = drl.conv_bwd(x, c["w"], c["b"], e, dy=x, dstate_T=e)
    assert torch.equal(g["dstate"], e) and not g["dweight"].any() and not g["dbias"].any()
    y, h = drl.norm_fwd(x, c["b"], residual=x)
    assert y.shape == h.shape == x.shape and not drl.norm_bwd(x, c["b"], x)["dweight"].any()
    assert drl.norm_fwd(x, c["b"], fmt="int8")[1].shape == x.shape[:-1]


@pytest.mark.parametrize("C", [66, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_with_slots_outside_the_pool(dtype, C):
    # more sequences than a wave has at a time, every third without a stored state: zeros there, the others as by themselves,
    # and rows that nobody names stay
    S, N = 4099, 16
    t = scan_tensors(make_scan(seed_of("outside", dtype, C), 1, S, C, 1, N, dtype, n=1), dtype)
    one = {k: (t[k] if k in ("A", "D", "bias") else t[k][0]) for k in SCAN_IN}
    idx = np.random.default_rng(6).permutation(S + 5)[:S].astype(np.int32)
    idx[::3] = np.where(np.arange(0, S, 3) % 2, -1, S + 5)
    kept = torch.from_numpy(np.flatnonzero((idx >= 0) & (idx < S + 5))).cuda()
    rows = torch.from_numpy(idx).cuda()[kept].long()
    pool = torch.randn(S + 5, C, N, device="cuda")
    window = torch.randn(S + 5, 3, C, device="cuda").to(t["x"].dtype)
    w, b = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    before, wbefore, own, wown = pool.clone(), window.clone(), pool[rows].clone(), window[rows].clone()
    a = lambda f: [f(one[k]) for k in ("x", "dt")] + [one["A"]] + [f(one[k]) for k in ("B", "C")]  # noqa: E731
    more = lambda f: dict(D=one["D"], z=f(one["z"]), dt_bias=one["bias"])  # noqa: E731
    y = drl.scan_step(*a(lambda v: v), pool, **more(lambda v: v), state_idx=i32(idx))
    u = drl.conv_step(one["x"], w, window, b, state_idx=i32(idx))
    pick = lambda v: v[kept].contiguous()  # noqa: E731
    assert torch.equal(y[kept], drl.scan_step(*a(pick), own, **more(pick))) and torch.equal(u[kept], drl.conv_step(pick(one["x"]), w, wown, b))
    assert not y[::3].any() and not u[::3].any()
    before[rows], wbefore[rows] = own, wown
    assert torch.equal(pool, before) and torch.equal(window, wbefore)


# ------------------------------------------------------------------------------------------------ all of them together
def test_serving_run():
    # Four users: prompts of 1 to 100 tokens packed through norm, projections, convolution and scan into the users' slots,
    # the states parked in 8 bits and taken up again, then token by token. Every operator against its definition over the whole
    # of a user's row, from the inputs that it had (what the operators before it left) and the states that were held.
    D, C, N, W, users, steps = 64, 96, 16, 4, 4, 5
    r = np.random.default_rng(7)
    f = lambda *s: dev(r.standard_normal(s) / np.sqrt(s[-1]), "bf16")  # noqa: E731
    w_in, w_dt, w_bc, w_out = f(2 * C, D), f(C, C), f(2 * N, C), f(D, C)
    x0 = make_scan(8, 1, 4, C, 1, N, "bf16")
    A, skip, bias = dev(x0["A"]), dev(x0["D"]), dev(x0["bias"])
    conv_w, conv_b, norm_w = dev(r.standard_normal((C, W)) / 2), dev(0.1 * r.standard_normal(C)), dev(1 + 0.1 * r.standard_normal(D))
    cu = [0, 30, 31, 131, 150]
    pool, window = torch.full((6, C, N), 9.0, device="cuda"), torch.full((6, W - 1, C), 9.0, device="cuda", dtype=torch.bfloat16)
    slots = [5, 0, 3, 1]
    pool[slots], window[slots] = 0.0, 0.0
    idx = i32(slots)
    seen = {}

    def layer(h, branch, step):
        y, h = drl.norm_fwd(branch, norm_w, residual=h)
        xz = y @ w_in.t()
        x, z = xz[..., :C], xz[..., C:]
        u = drl.conv_step(x, conv_w, window, conv_b, state_idx=idx) if step else drl.conv_fwd(x, conv_w, conv_b, window, i32(cu), state_idx=idx)[0]
        dt, bc = u @ w_dt.t(), (u @ w_bc.t()).unflatten(-1, (2, 1, N))
        B, Cm = bc[..., 0, :, :], bc[..., 1, :, :]
        o = (drl.scan_step(u, dt, A, B, Cm, pool, D=skip, z=z, dt_bias=bias, state_idx=idx) if step else
             drl.scan_fwd(u, dt, A, B, Cm, D=skip, z=z, dt_bias=bias, S0=pool, cu_seqlens=i32(cu), state_idx=idx)[0])
        for k, v in dict(h=h, y=y, x=x, u=u, dt=dt, B=B, C=Cm, z=z, o=o).items():
            seen.setdefault(k, []).append(v.clone())
        return h, o @ w_out.t()

    layer(dev(r.standard_normal((1, 150, D)), "bf16"), dev(r.standard_normal((1, 150, D)), "bf16"), False)
    end = pool.clone()
    codes, scales = drl.state_pack(end[slots].view(users, C // 16, 16, N))
    held = drl.state_unpack(codes, scales).view(users, C, N)
    pool[slots] = held
    h, branch = dev(r.standard_normal((users, D)), "bf16"), dev(r.standard_normal((users, D)), "bf16")
    for _ in range(steps):
        h, branch = layer(h, branch, True)
    assert (pool[[2, 4]] == 9.0).all() and (window[[2, 4]] == 9.0).all()
    np64 = lambda t: t.float().cpu().numpy()  # noqa: E731
    row = lambda k, n: np.concatenate([np64(seen[k][0][0, cu[n]:cu[n + 1]])] + [np64(v[n][None]) for v in seen[k][1:]])  # noqa: E731
    for n in range(users):
        L = cu[n + 1] - cu[n]
        v = {k: row(k, n)[None] for k in seen}
        T = L + steps
        tensor = lambda a: torch.from_numpy(a).to("cuda", torch.bfloat16)  # noqa: E731
        want = oracle.norm(v["h"][0], np64(norm_w))
        close(tensor(v["y"][0]), want, np.abs(want), 32, f"norm {n}")
        a = (v["x"], np64(conv_w), np64(conv_b))
        close(tensor(v["u"]), oracle.conv(*a)[0], oracle.conv(*a, magnitudes=True)[0], CONV_K, f"convolution {n}")
        end_w = np64(window[slots[n]])
        assert np.array_equal(end_w, np.concatenate([np.zeros((W - 1, C)), v["x"][0]])[-(W - 1):])
        par = (np64(A),)
        for part, S0, S1 in ((slice(0, L), np.zeros((1, C, N), np.float32), end[slots[n]]), (slice(L, T), np64(held[n])[None], pool[slots[n]])):
            q = {k: v[k][:, part] for k in ("u", "dt", "B", "C", "z")}
            a = (q["u"], q["dt"], *par, q["B"], q["C"], np64(skip), q["z"], np64(bias), S0)
            (y, S), (my, mS) = oracle.scan(*a), oracle.scan(*a, magnitudes=True)
            slack = scan_slack(dict(x=q["u"], dt=q["dt"], bias=np64(bias), S0=S0, B=q["B"], C=q["C"], z=q["z"]), N, True)
            close(tensor(v["o"][:, part]), y, my, scan_k(T, N), f"scan {n}", slack)
            close(S1[None], S, mS, scan_k(T, N), f"state {n}", slack)


def test_training_step():
    # a layer and its loss through torch autograd; every operator's gradients equal its own backward call at what autograd brought it
    D, C, N, T = 64, 72, 16, 45
    torch.manual_seed(3)
    x0 = scan_tensors(make_scan(9, 2, T, C, 1, N, "f32"), "f32")
    leaf = lambda t: t.detach().clone().requires_grad_()  # noqa: E731
    h0, br = leaf(torch.randn(2, T, D, device="cuda")), leaf(torch.randn(2, T, D, device="cuda"))
    nw, cw, cb, A, skip, bias = map(leaf, (torch.randn(D, device="cuda"), torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda"), x0["A"], x0["D"], x0["bias"]))
    w_in, w_bc = leaf(torch.randn(2 * C, D, device="cuda") / 8), leaf(torch.randn(C + 2 * N, C, device="cuda") / 8)
    y, h = drl.rms_norm(br, nw, h0)
    xz = y @ w_in.t()
    u, _ = drl.causal_conv(xz[..., :C], cw, cb)
    low = u @ w_bc.t()
    B, Cm = low[..., C:C + N].unflatten(-1, (1, N)), low[..., C + N:].unflatten(-1, (1, N))
    o, _ = drl.selective_scan(u, low[..., :C], A, B, Cm, skip, xz[..., C:], bias)
    for t in (y, h, xz, u, low, o):
        t.retain_grad()
    loss = o.square().mean() + h.square().mean()
    loss.backward()
    with torch.no_grad():
        g = drl.scan_bwd(u, low[..., :C], A, B, Cm, skip, xz[..., C:], bias, dy=o.grad)
        assert torch.equal(A.grad, g["dA"]) and torch.equal(skip.grad, g["dD"]) and torch.equal(bias.grad, g["ddt_bias"])
        assert torch.equal(low.grad, torch.cat([g["ddt"], g["dB"][:, :, 0], g["dC"][:, :, 0]], -1))
        du = g["dx"] + low.grad @ w_bc  # autograd's sum of the two, in either order
        assert (u.grad - du).abs().max() <= (C + 2 * N + 2) * 2.0 ** -23 * (g["dx"].abs() + low.grad.abs() @ w_bc.abs()).max()
        gc = drl.conv_bwd(xz[..., :C], cw, cb, dy=u.grad)
        assert torch.equal(cw.grad, gc["dweight"]) and torch.equal(cb.grad, gc["dbias"])
        assert torch.equal(xz.grad, torch.cat([gc["dx"], g["dz"]], -1))
        gn = drl.norm_bwd(h, nw, y.grad, h.grad)
        assert torch.equal(nw.grad, gn["dweight"]) and torch.equal(br.grad, gn["dx"]) and torch.equal(h0.grad, gn["dx"])


# ------------------------------------------------------------------------------------------------ offsets past 32 bits
def test_offsets_past_32_bits(monkeypatch):
    # 2^31 elements lie before what is checked: the last tokens of a long row that is zero up to them, and the last slots of pools
    monkeypatch.setenv("DR_SCAN_BLOCK", "2")
    monkeypatch.setenv("DR_SCAN_SEG", str(1 << 22))  # one segment: the tail's tiles are then the same work in both
    C, N, tail = 4096, 16, 176
    T = (1 << 19) + tail
    t = scan_tensors(make_scan(20, 1, tail, C, 1, N, "bf16"), "bf16")
    small = [t[k] for k in SCAN_IN]
    big = {k: torch.zeros((1, T) + tuple(t[k].shape[2:]), dtype=t[k].dtype, device="cuda") for k in ("x", "dt", "B", "C", "z", "dy")}
    for k, v in big.items():
        v[:, T - tail:] = t[k]
    assert big["x"].numel() - tail * C >= 2 ** 31
    full = [big.get(k, t[k]) for k in SCAN_IN]
    y, S = drl.scan_fwd(*full)
    ys, Ss = drl.scan_fwd(*small)
    assert torch.equal(y[:, T - tail:], ys) and torch.equal(S, Ss)
    del y
    g, part = drl.scan_bwd(*full, dy=big["dy"], need_dS0=False), drl.scan_bwd(*small, dy=t["dy"], need_dS0=False)
    for k in ("dx", "ddt", "dB", "dC", "dz"):
        assert torch.equal(g[k][:, T - tail:], part[k]), k
    del g, full, big["dt"], big["z"]
    w, b = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    y, last = drl.conv_fwd(big["x"], w, b)
    ys, _ = drl.conv_fwd(t["x"], w, b)
    assert torch.equal(y[:, T - tail:], ys) and torch.equal(last, t["x"][:, -3:])
    del y
    g, part = drl.conv_bwd(big["x"], w, b, dy=big["dy"]), drl.conv_bwd(t["x"], w, b, dy=t["dy"])
    assert torch.equal(g["dx"][:, T - tail:], part["dx"])
    del g, part
    rows = 300  # (as many as the same rule takes for the backward pass)
    x, dy = big["x"][0], big["dy"][0]
    w = torch.randn(C, device="cuda")
    y, h = drl.norm_fwd(x, w, residual=dy)
    ys, hs = drl.norm_fwd(x[T - rows:], w, residual=dy[T - rows:])
    assert torch.equal(y[T - rows:], ys) and torch.equal(h[T - rows:], hs)
    codes, scales, _ = drl.norm_fwd(x, w, fmt="e4m3")
    cs, ss, _ = drl.norm_fwd(x[T - rows:], w, fmt="e4m3")
    assert torch.equal(codes[T - rows:].view(torch.uint8), cs.view(torch.uint8)) and torch.equal(scales[T - rows:], ss)
    del y, h, codes
    assert torch.equal(drl.norm_bwd(x, w, dy)["dx"][T - rows:], drl.norm_bwd(x[T - rows:], w, dy[T - rows:])["dx"])
    del x, dy, big
    slots = 4 + 2 ** 31 // (C * N)
    pool = torch.zeros(slots, C, N, device="cuda")
    idx = i32([slots - 1, 0, slots - 2])
    S = torch.randn(3, C, N, device="cuda")
    pool[idx.long()] = S
    one = {k: (t[k] if k in ("A", "D", "bias") else t[k][0, :3]) for k in SCAN_IN}
    a = (one["x"], one["dt"], one["A"], one["B"], one["C"])
    more = dict(D=one["D"], z=one["z"], dt_bias=one["bias"])
    assert torch.equal(drl.scan_step(*a, pool, **more, state_idx=idx), drl.scan_step(*a, S, **more))
    assert torch.equal(pool[idx.long()], S)
    del pool
    slots = 4 + 2 ** 31 // (3 * C)
    pool = torch.zeros(slots, 3, C, device="cuda", dtype=torch.bfloat16)
    idx = i32([slots - 1, 0, slots - 2])
    S = torch.randn(3, 3, C, device="cuda").bfloat16()
    pool[idx.long()] = S
    w, b = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    assert torch.equal(drl.conv_step(one["x"], w, pool, b, state_idx=idx), drl.conv_step(one["x"], w, S, b))
    assert torch.equal(pool[idx.long()], S)
