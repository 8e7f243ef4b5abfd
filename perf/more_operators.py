"""The selective scan, its short convolution and the norm in front of them as they are measured: cases, inputs, plain forms
and definitions.

Selective scan: h_t[c,n] = exp(d_t[c] A[c,n]) h_{t-1}[c,n] + d_t[c] x_t[c] B_t[n], d = softplus(dt + bias),
y_t[c] = (sum_n C_t[n] h_t[c,n] + D[c] x_t[c]) silu(z_t[c]); groups of channels share B and C.
Convolution: y_t[c] = act(bias[c] + sum_j w[c,j] e_{t+j}[c]), e the last inputs of before (the state) and then x.
Norm: h = x + r, y = h w / sqrt(mean h^2 + eps), in the type of x or in 8 bits with a scale for each token.
Activations (x, dt, B, C, z and their gradients) have the case's type, parameters and scan states are fp32.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------------ cases
def _conv(kind, name, B, T, C, W, dtype, act="silu", packed=0, state=True):
    """kind conv_fwd / conv_bwd; packed: number of sequences in one packed row of T tokens (B is then 1), 0 for B rows."""
    c = {"kind": kind, "B": B, "T": T, "C": C, "W": W, "dtype": dtype, "act": act, "packed": packed, "state": state}
    return dict(c, name=name) if name else c


def _scan(kind, name, B, T, C, G, N, dtype, gate=True, packed=0, state=True):
    """kind scan_fwd / scan_bwd; C channels in G groups, N states for each channel."""
    c = {"kind": kind, "B": B, "T": T, "C": C, "G": G, "N": N, "dtype": dtype, "gate": gate, "packed": packed, "state": state}
    return dict(c, name=name) if name else c


def _conv_step(name, S, pool, C, W, dtype):
    c = {"kind": "conv_step", "S": S, "pool": pool, "C": C, "W": W, "dtype": dtype}
    return dict(c, name=name) if name else c


def _scan_step(name, S, pool, C, G, N, dtype):
    c = {"kind": "scan_step", "S": S, "pool": pool, "C": C, "G": G, "N": N, "dtype": dtype}
    return dict(c, name=name) if name else c


def _norm(kind, name, rows, C, dtype, residual=True, fmt=""):
    """kind norm / norm_bwd; fmt: int8 or e4m3, or none for the type of x."""
    c = {"kind": kind, "rows": rows, "C": C, "dtype": dtype, "residual": residual, "fmt": fmt}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the convolution in front of the recurrence at the library's prefill workload (16 heads of 128 channels)
        _conv("conv_fwd", "conv", 4, 4096, 2048, 4, "bf16", state=False),
        # its training step: documents packed in one row, an odd number of channels, fp32
        _conv("conv_bwd", "conv backward, packed, fp32", 1, 7777, 1531, 4, "f32", packed=5),
        # continuous batching: one token for each of 512 sequences out of a pool
        _conv_step("conv step, 512 sequences", 512, 520, 4096, 4, "bf16"),
        # a chat turn of a few tokens appended to a stored state: latency
        _scan("scan_fwd", "scan, one short turn", 1, 37, 2048, 1, 16, "bf16"),
        # the library's prefill workload
        _scan("scan_fwd", "scan", 4, 4096, 2048, 1, 16, "bf16", state=False),
        # packed documents of a small fp32 layer: two groups, an odd number of channels, more states
        _scan("scan_fwd", "scan, packed, fp32, 32 states", 1, 7777, 2 * 333, 2, 32, "f32", gate=False, packed=12),
        # a training step's backward at half the prefill workload
        _scan("scan_bwd", "scan backward", 2, 4096, 2048, 1, 16, "bf16", state=False),
        # one token for each of 512 sequences out of a pool
        _scan_step("scan step, 512 sequences", 512, 520, 4096, 1, 16, "bf16"),
        # one user decoding: the smallest norm, latency
        _norm("norm", "norm, one token", 1, 2048, "bf16"),
        # the prefill workload's tokens, the output in 8 bits for a quantised projection
        _norm("norm", "norm, int8", 16384, 2048, "bf16", fmt="int8"),
        # odd rows in fp32 (e4m3)
        _norm("norm", "norm, fp32, e4m3, odd", 1333, 1531, "f32", fmt="e4m3"),
        # the same tokens' training step
        _norm("norm_bwd", "norm backward", 16384, 2048, "bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "norm", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    C = rng.choice([_logint(rng, 1, 4096), 64 * _logint(rng, 1, 64)])
    if kind in ("norm", "norm_bwd"):
        rows = _logint(rng, 1, 16384 * 2048 // (2 * C if dtype == "f32" else C))
        fmt = rng.choice(["", "", "int8", "e4m3"]) if kind == "norm" else ""
        return _norm(kind, None, min(rows, 65536), C, dtype, rng.random() < 0.7, fmt)
    S = _logint(rng, 1, 512 * 4096 // max(C, 512))
    if kind == "conv_step":
        return _conv_step(None, S, S + rng.randrange(0, 9), C, rng.choice([2, 3, 4, 4]), dtype)
    N, G = rng.choice([16, 16, 32, 64]), rng.choice([1, 1, 2, 3])
    if kind == "scan_step":
        return _scan_step(None, max(1, S * 16 // N), S + rng.randrange(0, 9), G * -(-C // G), G, N, dtype)
    B = rng.choice([1, 1, 2, 3, 4])
    packed = rng.choice([0, 0, 1])
    most = 4 * 4096 * 2048
    if kind.startswith("conv"):
        tokens = _logint(rng, 1, min(65536, most // (2 if kind == "conv_bwd" or dtype == "f32" else 1) // C))
        T = tokens if packed else max(1, tokens // B)
        return _conv(kind, None, 1 if packed else B, T, C, rng.choice([2, 3, 4, 4]), dtype, rng.choice(["silu", "none"]),
                     min(T, rng.randrange(1, 20)) if packed else 0, rng.random() < 0.5)
    C = G * -(-C // G)
    tokens = _logint(rng, 1, min(32768, most * 16 // (2 if kind == "scan_bwd" else 1) // (C * N)))
    T = tokens if packed else max(1, tokens // B)
    return _scan(kind, None, 1 if packed else B, T, C, G, N, dtype, rng.random() < 0.7, min(T, rng.randrange(1, 20)) if packed else 0, rng.random() < 0.5)


def work(case):
    c = case
    b, kind, C = 2 if c["dtype"] == "bf16" else 4, c["kind"], c["C"]
    if kind == "norm":
        n = c["rows"] * C
        out = 1 if c["fmt"] else b  # (the values that 8 bits stand for are formed by whoever asks for them)
        return {"bytes": n * (b * (3 if c["residual"] else 1) + out) + 4 * C, "flops": 5 * n}
    if kind == "norm_bwd":
        n = c["rows"] * C
        return {"bytes": n * b * (4 if c["residual"] else 3) + 8 * C, "flops": 9 * n}
    if kind == "conv_step":
        return {"bytes": c["S"] * C * b * 2 * c["W"] + 4 * C * (c["W"] + 1), "flops": 2 * c["W"] * c["S"] * C}
    if kind == "scan_step":
        return {"bytes": c["S"] * (8 * C * c["N"] + b * (4 * C + 2 * c["G"] * c["N"])) + 4 * C * (c["N"] + 2), "flops": 7 * c["S"] * C * c["N"]}
    tokens, seqs = c["B"] * c["T"], c["packed"] or c["B"]
    if kind.startswith("conv"):
        back = kind == "conv_bwd"
        state = seqs * (c["W"] - 1) * C * b * ((2 if c["state"] else 1) + (1 if back else 0))
        return {"bytes": tokens * C * b * (3 if back else 2) + state + 4 * C * (c["W"] + 1) * (2 if back else 1),
                "flops": tokens * C * 2 * c["W"] * (3 if back else 1)}
    bc, state = 2 * c["G"] * c["N"] * b, seqs * C * c["N"] * 4
    if kind == "scan_fwd":
        return {"bytes": tokens * (C * b * (4 if c["gate"] else 3) + bc) + state * (2 if c["state"] else 1) + 4 * C * (c["N"] + 2), "flops": 7 * tokens * C * c["N"]}
    return {"bytes": tokens * (C * b * (7 if c["gate"] else 5) + 2 * bc) + state * (3 if c["state"] else 2) + 8 * C * (c["N"] + 2), "flops": 18 * tokens * C * c["N"]}


# ------------------------------------------------------------------------------------------------ inputs
def _lengths(T, n, seed):
    """n positive lengths that sum to T, uneven."""
    r = torch.Generator().manual_seed(seed)
    cuts = torch.randperm(T - 1, generator=r)[: n - 1].sort().values + 1 if n > 1 else torch.empty(0, dtype=torch.long)
    return torch.diff(torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), T)]))


def _offsets(s, c, seed):
    s["cu"] = None
    if c["packed"]:
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), _lengths(c["T"], c["packed"], seed).cumsum(0)]).to(torch.int32).cuda()


def prepare(case, seed):
    c, dev, kind, C = case, "cuda", case["kind"], case["C"]
    t = _T[c["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *sh: torch.randn(sh, generator=g, device=dev)  # noqa: E731
    s = {"case": c}
    if kind.startswith("norm"):
        s["x"], s["w"] = rnd(c["rows"], C).to(t), 1 + 0.2 * rnd(C)
        s["r"] = (3 * rnd(c["rows"], C)).to(t) if c["residual"] else None
        if kind == "norm_bwd":  # the forward's sum and the gradients that reach its two outputs
            s["h"] = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(t)
            s["dy"] = rnd(c["rows"], C).to(t)
            s["dh"] = rnd(c["rows"], C).to(t) if c["residual"] else None
        return s
    if kind.startswith("conv"):
        s["w"], s["bias"] = rnd(C, c["W"]) / math.sqrt(c["W"]), 0.1 * rnd(C)
        if kind == "conv_step":
            s["x"] = rnd(c["S"], 2 * C).to(t)[:, :C]  # one half of a fused projection
            s["state"] = rnd(c["pool"], c["W"] - 1, C).to(t)
            s["idx"] = torch.randperm(c["pool"], generator=g, device=dev)[: c["S"]].to(torch.int32)
            return s
        s["x"] = rnd(c["B"], c["T"], 2 * C).to(t)[..., :C]
        _offsets(s, c, seed)
        n = c["packed"] or c["B"]
        s["state"] = rnd(n, c["W"] - 1, C).to(t) if c["state"] else None
        if kind == "conv_bwd":
            s["dy"], s["dstate_T"] = rnd(c["B"], c["T"], C).to(t), rnd(n, c["W"] - 1, C).to(t)
        return s
    N, G = c["N"], c["G"]
    lead = (c["S"],) if kind == "scan_step" else (c["B"], c["T"])
    s["A"] = -torch.exp(torch.log(torch.arange(1.0, N + 1, device=dev)) + 0.1 * rnd(C, N))
    s["D"] = 1 + 0.1 * rnd(C)
    step = torch.exp(torch.rand(C, generator=g, device=dev) * math.log(100.0) + math.log(1e-3))  # 0.001 to 0.1
    s["bias"] = step + torch.log(-torch.expm1(-step))
    s["x"], s["dt"] = rnd(*lead, C).to(t), (0.5 * rnd(*lead, C)).to(t)
    low = rnd(*lead, 64 + 2 * G * N).to(t)  # what the step's projection, B and C are split from
    s["B"], s["C"] = (low[..., a:a + G * N].unflatten(-1, (G, N)) for a in (64, 64 + G * N))
    s["z"] = rnd(*lead, 2 * C).to(t)[..., C:] if kind == "scan_step" or c["gate"] else None
    if kind == "scan_step":
        s["S"] = rnd(c["pool"], C, N)
        s["idx"] = torch.randperm(c["pool"], generator=g, device=dev)[: c["S"]].to(torch.int32)
        return s
    _offsets(s, c, seed)
    n = c["packed"] or c["B"]
    s["S0"] = rnd(n, C, N) if c["state"] else None
    if kind == "scan_bwd":
        s["dy"], s["dS_T"] = rnd(*lead, C).to(t), rnd(n, C, N)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _first(s, c):
    """For each token of a row its sequence [B, T] and the first token of that sequence in the row."""
    if s["cu"] is None:
        return torch.arange(c["B"], device="cuda")[:, None].expand(c["B"], c["T"]), torch.zeros((), dtype=torch.long, device="cuda").expand(c["B"], c["T"])
    n = torch.searchsorted(s["cu"][1:].long(), torch.arange(c["T"], device="cuda"), right=True)[None]
    return n, s["cu"].long()[n]


def _ends(s, c):
    """Row and position of each sequence's last token."""
    if s["cu"] is None:
        return torch.arange(c["B"], device="cuda"), torch.full((c["B"],), c["T"] - 1, device="cuda")
    return torch.zeros(c["packed"], dtype=torch.long, device="cuda"), s["cu"][1:].long() - 1


def _taps(s, c):
    """The W inputs of each output [B, T, W, C] in 32 bits, and where in the row (or, below its start, in the state) they are."""
    W, state = c["W"], s["state"]
    n, first = _first(s, c)
    at = torch.arange(c["T"], device="cuda")[None, :, None] - torch.arange(W - 1, -1, -1, device="cuda")  # [1, T, W]
    before = first[..., None] - at  # > 0: that many tokens before the sequence
    rows = torch.arange(c["B"], device="cuda")[:, None, None].expand(before.shape)
    e = s["x"].float()[rows, at.clamp(min=0).expand(before.shape)]
    old = 0.0 if state is None else state.float()[n[..., None].expand(before.shape), (W - 1 - before).clamp(0, W - 2)]
    return torch.where((before > 0)[..., None], old, e), before


def _conv_last(s, c):
    """Each sequence's last W - 1 inputs, the state's own where it is shorter."""
    W, (row, end) = c["W"], _ends(s, c)
    length = (end + 1 if s["cu"] is None else torch.diff(s["cu"]).long())[:, None]
    back = torch.arange(W - 1, 0, -1, device="cuda")  # tokens from the end
    x = s["x"][row[:, None], (end[:, None] + 1 - back).clamp(min=0)]
    if s["state"] is None:
        return torch.where((back <= length)[..., None], x, torch.zeros_like(x))
    n = torch.arange(len(row), device="cuda")[:, None]
    return torch.where((back <= length)[..., None], x, s["state"][n, (W - 1 - back + length).clamp(max=W - 2)])


def _act(u, act):
    return u * _sigmoid(u) if act == "silu" else u


def _plain_conv(s, c):
    e, _ = _taps(s, c)
    return _act((e * s["w"].T).sum(-2) + s["bias"], c["act"]).to(s["x"].dtype), _conv_last(s, c)


def _plain_conv_bwd(s, c):
    W, t = c["W"], s["x"].dtype
    e, before = _taps(s, c)
    u, du = (e * s["w"].T).sum(-2) + s["bias"], s["dy"].float()
    if c["act"] == "silu":
        sg = _sigmoid(u)
        du = du * sg * (1 + u * (1 - sg))
    de = du[..., None, :] * s["w"].T  # [B, T, W, C]: of each tap
    n, _ = _first(s, c)
    B, T, C = s["x"].shape
    at = torch.arange(T, device="cuda")[None, :, None] - torch.arange(W - 1, -1, -1, device="cuda")
    # taps inside the row add to it, the others to the state
    inside = (before <= 0)[..., None]
    rows = torch.arange(B, device="cuda")[:, None, None] * T + at.clamp(min=0)
    dx = torch.zeros(B * T, C, device="cuda").index_add_(0, rows.flatten(), (de * inside).flatten(0, 2))
    S = s["dstate_T"].shape[0]
    k = n[..., None] * (W - 1) + (W - 1 - before).clamp(0, W - 2)
    ds = torch.zeros(S * (W - 1), C, device="cuda").index_add_(0, k.flatten(), (de * ~inside).flatten(0, 2))
    # what reaches the last inputs directly
    row, end = _ends(s, c)
    length = (end + 1 if s["cu"] is None else torch.diff(s["cu"]).long())[:, None]
    back = torch.arange(W - 1, 0, -1, device="cuda")
    mine, g = (back <= length)[..., None], s["dstate_T"].float()
    dx.index_add_(0, (row[:, None] * T + (end[:, None] + 1 - back).clamp(min=0)).flatten(), (g * mine).flatten(0, 1))
    k = torch.arange(S, device="cuda")[:, None] * (W - 1) + (W - 1 - back + length).clamp(max=W - 2)
    ds.index_add_(0, k.flatten(), (g * ~mine).flatten(0, 1))
    return {"dx": dx.view(B, T, C).to(t), "dweight": torch.stack([(du * e[..., j, :]).sum((0, 1), dtype=torch.float64) for j in range(W)], 1).float(),
            "dbias": du.sum((0, 1), dtype=torch.float64).float(), "dstate": ds.view(S, W - 1, C).to(t) if c["state"] else None}


def _plain_conv_step(s, c):
    i = s["idx"].long()
    e = torch.cat([s["state"][i], s["x"][:, None]], 1)
    s["state"][i] = e[:, 1:]
    return _act((e.float() * s["w"].T).sum(1) + s["bias"], "silu").to(s["x"].dtype), s["state"]


def _running(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, from zero: pairs of tokens first, then the tokens between."""
    T = a.shape[1]
    if T == 1:
        return b
    n, odd = T // 2, a[:, 1::2]
    up = _running(odd * a[:, 0:2 * n:2], torch.addcmul(b[:, 1::2], odd, b[:, 0:2 * n:2]))
    h = torch.empty_like(b)
    h[:, 0], h[:, 1::2] = b[:, 0], up
    h[:, 2::2] = torch.addcmul(b[:, 2::2], a[:, 2::2], up[:, : (T - 1) // 2])
    return h


def _scan_parts(s, c):
    f = lambda x: x.float()  # noqa: E731
    raw = f(s["dt"]) + s["bias"]
    d = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    per = c["C"] // c["G"]
    Bm, Cm = (f(s[m]).repeat_interleave(per, -2) for m in "BC")  # [.., C, N]
    return f(s["x"]), raw, d, Bm, Cm


def _states(s, c, x, d, Bm):
    """Decays and states of every token [B, T, C, N], and the states before the sequences' first tokens, in their places."""
    a = torch.exp(d[..., None] * s["A"])
    b = (d * x)[..., None] * Bm
    n, first = _first(s, c)
    start = torch.arange(c["T"], device="cuda") == first
    before = None
    if s["S0"] is not None:
        before = s["S0"][n[start]]
        b[start] += a[start] * before
    return a, _running(a.masked_fill(start[..., None, None], 0.0), b), start, before


def _plain_scan(s, c):
    x, _, d, Bm, Cm = _scan_parts(s, c)
    _, h, _, _ = _states(s, c, x, d, Bm)
    y = (h * Cm).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(s["x"].dtype), h[_ends(s, c)]


def _plain_scan_bwd(s, c):
    t = s["x"].dtype
    x, raw, d, Bm, Cm = _scan_parts(s, c)
    a, h, start, before = _states(s, c, x, d, Bm)
    dy, out = s["dy"].float(), {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = _sigmoid(z)
        out["dz"] = (dy * ((h * Cm).sum(-1) + s["D"] * x) * sg * (1 + z * (1 - sg))).to(t)
        dy = dy * z * sg
    ends = _ends(s, c)
    g = dy[..., None] * Cm  # what reaches each state: from its output, from the next state, from the sequence's end
    g[ends] += s["dS_T"]
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    after[ends] = 0.0
    g = _running(after.flip(1), g.flip(1)).flip(1)
    group = lambda v: v.unflatten(2, (c["G"], -1)).sum(3, dtype=torch.float64).to(t)  # noqa: E731
    out["dB"], out["dC"] = group(g * (d * x)[..., None]), group(h * dy[..., None])
    into = (g * Bm).sum(-1)
    old = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    old[start] = 0.0 if before is None else before
    old = old.mul_(a).mul_(g)  # gradient of d_t A: g a h_{t-1}
    draw = ((old * s["A"]).sum(-1) + into * x) * _sigmoid(raw)
    out["ddt"], out["ddt_bias"] = draw.to(t), draw.sum((0, 1), dtype=torch.float64).float()
    out["dA"] = old.mul_(d[..., None]).sum((0, 1), dtype=torch.float64).float()
    out["dx"], out["dD"] = (into * d + s["D"] * dy).to(t), (dy * x).sum((0, 1), dtype=torch.float64).float()
    if s["S0"] is not None:
        out["dS0"] = (a * g)[start]
    return out


def _plain_scan_step(s, c):
    x, _, d, Bm, Cm = _scan_parts(s, c)
    i = s["idx"].long()
    h = s["S"][i] * torch.exp(d[..., None] * s["A"]) + (d * x)[..., None] * Bm
    s["S"][i] = h
    z = s["z"].float()
    return (((h * Cm).sum(-1) + s["D"] * x) * z * _sigmoid(z)).to(s["x"].dtype), s["S"]


def _e4m3(x):
    """x rounded to the nearest value of 4 exponent and 3 fraction bits, ties to even (|x| <= 448)."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4
    return torch.ldexp(torch.round(torch.ldexp(x, -e)), e)


EPS = 1e-5


def _plain_norm(s, c):
    t = s["x"].dtype
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(t)
    f = h.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    p = f * s["w"]
    if not c["fmt"]:
        y = (p * r).to(t)
        return y if s["r"] is None else (y, h)
    top = p.abs().amax(-1, keepdim=True)
    if c["fmt"] == "int8":
        scale = (top * (1 / 127)).clamp(min=2.0 ** -126)
        held = torch.round(p.double() / scale.double()).float()  # 64 bits: quotients next to a half
    else:
        m, e = torch.frexp(top)
        scale = torch.ldexp(torch.ones_like(top), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
        held = _e4m3(p / scale)
    scale = scale * r
    values = held.to(_CODE[c["fmt"]]).float() * scale
    return (values, scale[:, 0]) if s["r"] is None else (values, scale[:, 0], h)


def _plain_norm_bwd(s, c):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    wd = s["w"] * dy
    dx = r * (wd - h * (r * r * (wd * h).mean(-1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * h * r).sum(0, dtype=torch.float64).float()}


_PLAIN = {"conv_fwd": _plain_conv, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step, "scan_fwd": _plain_scan, "scan_bwd": _plain_scan_bwd,
          "scan_step": _plain_scan_step, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


def _run_own(s, c):
    import delta_rule_linear_chunked_amd as drl

    kind = c["kind"]
    if kind == "conv_fwd":
        return drl.conv_fwd(s["x"], s["w"], s["bias"], state=s["state"], cu_seqlens=s["cu"], activation=c["act"])
    if kind == "conv_bwd":
        return drl.conv_bwd(s["x"], s["w"], s["bias"], state=s["state"], cu_seqlens=s["cu"], activation=c["act"], dy=s["dy"], dstate_T=s["dstate_T"])
    if kind == "conv_step":
        return drl.conv_step(s["x"], s["w"], s["state"], s["bias"], state_idx=s["idx"]), s["state"]
    if kind == "scan_step":
        return drl.scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["S"], D=s["D"], z=s["z"], dt_bias=s["bias"], state_idx=s["idx"]), s["S"]
    if kind == "scan_fwd":
        return drl.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["bias"], S0=s["S0"], cu_seqlens=s["cu"])
    if kind == "scan_bwd":
        g = drl.scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["bias"], S0=s["S0"], cu_seqlens=s["cu"],
                         dy=s["dy"], dS_T=s["dS_T"], need_dS0=s["S0"] is not None)
        return {k: v for k, v in g.items() if v is not None}
    if kind == "norm_bwd":
        return drl.norm_bwd(s["h"], s["w"], s["dy"], dh=s["dh"], eps=EPS)
    out = drl.norm_fwd(s["x"], s["w"], residual=s["r"], eps=EPS, fmt=c["fmt"] or None)
    if not c["fmt"]:
        return out[0] if s["r"] is None else out
    codes, scale, h = out
    values = codes * scale[:, None] if c["fmt"] == "int8" else codes.float() * scale[:, None]
    return (values, scale) if s["r"] is None else (values, scale, h)


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return _PLAIN[c["kind"]](state, c)


# ------------------------------------------------------------------------------------------------ definitions in 64 bits
def _spans(s, c):
    """(batch row, first token, past the last) of each sequence."""
    if s["cu"] is None:
        return [(b, 0, c["T"]) for b in range(c["B"])]
    cu = s["cu"].tolist()
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def _zeros(*sh):
    return torch.zeros(sh, dtype=torch.float64, device="cuda")


def _silu64(u):
    return u * torch.sigmoid(u)


def _dsilu64(u):
    return torch.sigmoid(u) + u * torch.sigmoid(u) * torch.sigmoid(-u)


def _exact_conv(s, c):
    W, C, w, bias = c["W"], c["C"], s["w"].double(), s["bias"].double()
    B, T = c["B"], c["T"]
    spans = _spans(s, c)
    y, last = _zeros(B, T, C), _zeros(len(spans), W - 1, C)
    dx, dw, db, ds = _zeros(B, T, C), _zeros(C, W), _zeros(C), _zeros(len(spans), W - 1, C)
    for n, (b, t0, t1) in enumerate(spans):
        L = t1 - t0
        e = torch.cat([_zeros(W - 1, C) if s["state"] is None else s["state"][n].double(), s["x"][b, t0:t1].double()])
        u = bias + sum(w[:, j] * e[j:j + L] for j in range(W))
        y[b, t0:t1], last[n] = _silu64(u) if c["act"] == "silu" else u, e[L:]
        if c["kind"] == "conv_bwd":
            du = s["dy"][b, t0:t1].double() * (_dsilu64(u) if c["act"] == "silu" else 1.0)
            de = _zeros(L + W - 1, C)
            for j in range(W):
                de[j:j + L] += w[:, j] * du
                dw[:, j] += (du * e[j:j + L]).sum(0)
            de[L:] += s["dstate_T"][n].double()
            db += du.sum(0)
            ds[n], dx[b, t0:t1] = de[:W - 1], de[W - 1:]
    if c["kind"] == "conv_fwd":
        return y, last
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds if c["state"] else None}


def _rows64(s, c, b, t):
    """delta, x, B and C (by channel) of the tokens t of batch row b (a step: of the sequences t) in 64 bits."""
    at = (t,) if b is None else (b, t)
    g = torch.arange(c["C"], device="cuda") // (c["C"] // c["G"])
    raw = s["dt"][at].double() + s["bias"].double()
    d = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    return raw, d, s["x"][at].double(), s["B"][at].double()[..., g, :], s["C"][at].double()[..., g, :]


def _exact_scan(s, c):
    B, T, C, N, G = (c[k] for k in ("B", "T", "C", "N", "G"))
    A, D = s["A"].double(), s["D"].double()
    spans = _spans(s, c)
    y, S_T = _zeros(B, T, C), _zeros(len(spans), C, N)
    o = {"dx": _zeros(B, T, C), "ddt": _zeros(B, T, C), "dB": _zeros(B, T, G, N), "dC": _zeros(B, T, G, N), "dA": _zeros(C, N), "dD": _zeros(C),
         "ddt_bias": _zeros(C), "dz": _zeros(B, T, C), "dS0": _zeros(len(spans), C, N)}
    back = c["kind"] == "scan_bwd"
    for n, (b, t0, t1) in enumerate(spans):  # one sequence after the other, one token after the other
        for c0 in range(t0, t1, 512):
            raw, d, x, Bm, Cm = _rows64(s, c, b, slice(c0, min(t1, c0 + 512)))
            if c0 == t0:
                h = _zeros(C, N) if s["S0"] is None else s["S0"][n].double()
                kept = [h]
            bx = (d * x)[..., None] * Bm
            for k in range(d.shape[0]):
                h = torch.exp(d[k][:, None] * A) * h + bx[k]
                y[b, c0 + k] = (h * Cm[k]).sum(-1)
                if back:
                    kept.append(h)
            y[b, c0:c0 + d.shape[0]] += D * x
        S_T[n] = h
        if not back:
            continue
        raw, d, x, Bm, Cm = _rows64(s, c, b, slice(t0, t1))
        dy = s["dy"][b, t0:t1].double()
        if s["z"] is not None:
            z = s["z"][b, t0:t1].double()
            o["dz"][b, t0:t1] = dy * y[b, t0:t1] * _dsilu64(z)
            dy = dy * _silu64(z)
        g = s["dS_T"][n].double()
        for k in range(t1 - t0 - 1, -1, -1):
            t = t0 + k
            g = g + dy[k][:, None] * Cm[k]
            o["dC"][b, t] = (kept[k + 1] * dy[k][:, None]).view(G, -1, N).sum(1)
            o["dB"][b, t] = (g * (d[k] * x[k])[:, None]).view(G, -1, N).sum(1)
            u, a = (g * Bm[k]).sum(-1), torch.exp(d[k][:, None] * A)
            g = g * a  # reaches the state before, and by the exponent's product with it the decay
            w = g * kept[k]
            o["dA"] += w * d[k][:, None]
            o["dx"][b, t] = u * d[k] + D * dy[k]
            o["ddt"][b, t] = ((w * A).sum(-1) + u * x[k]) * torch.sigmoid(raw[k])
        o["dS0"][n] = g
        o["dD"] += (dy * x).sum(0)
        o["ddt_bias"] += o["ddt"][b, t0:t1].sum(0)
    if back:
        return {k: v for k, v in o.items() if (k != "dz" or s["z"] is not None) and (k != "dS0" or s["S0"] is not None)}
    return (y if s["z"] is None else y * _silu64(s["z"].double())), S_T


def _exact_norm(s, c):
    if c["kind"] == "norm_bwd":
        h, dy, w = s["h"].double(), s["dy"].double(), s["w"].double()
        ms = (h * h).sum(-1, keepdim=True) / c["C"] + EPS
        n = h / ms.sqrt()
        dn = dy * w
        dx = (dn - n * (dn * n).sum(-1, keepdim=True) / c["C"]) / ms.sqrt()
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dweight": (dy * n).sum(0)}
    t = s["x"].dtype
    h = s["x"].double() if s["r"] is None else (s["x"].double() + s["r"].double()).to(t).double()  # the sum is held in the type of x
    rms = ((h * h).sum(-1, keepdim=True) / c["C"] + EPS).sqrt()
    if not c["fmt"]:
        y = h * s["w"].double() / rms
        return y if s["r"] is None else (y, h)
    p = (h * s["w"].double()).float().double()  # a row to be held in 8 bits is a row of 32-bit numbers
    top = p.abs().amax(-1, keepdim=True)
    if c["fmt"] == "int8":
        # a scale is a 32-bit number: the largest magnitude times the 32-bit number next to 1 / 127
        sc = (top * torch.tensor(1 / 127, device="cuda").double()).float().double().clamp(min=2.0 ** -126)
        held = torch.round(p / sc)
    else:  # all the values that the format has, in order
        bits = torch.arange(127, device="cuda")
        e, m = bits // 8, (bits % 8).double()
        grid = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
        sc = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-126))
        q = (p / sc).abs().contiguous()
        up = torch.searchsorted(grid, q).clamp(max=126)
        lo, hi = grid[(up - 1).clamp(min=0)], grid[up]
        even = torch.where(up % 2 == 0, hi, lo)  # of two neighbours the one with an even fraction
        near = torch.where(q - lo < hi - q, lo, torch.where(q - lo > hi - q, hi, even))
        held = torch.where(q == hi, hi, near) * torch.sign(p)
    values, scale = held * sc / rms, (sc / rms)[:, 0]
    return (values, scale) if s["r"] is None else (values, scale, h)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["kind"] == "conv_step":
        out, pool, w, bias = [], s["state"].double(), s["w"].double(), s["bias"].double()
        for n, i in enumerate(s["idx"].tolist()):  # one sequence after another
            e = torch.cat([pool[i], s["x"][n].double()[None]])
            out.append(_silu64((e.T * w).sum(1) + bias))
            pool[i] = e[1:]
        return torch.stack(out), pool
    if c["kind"] == "scan_step":
        out, pool = [], s["S"].double()
        for n, i in enumerate(s["idx"].tolist()):
            _, d, x, Bm, Cm = _rows64(s, c, None, n)
            pool[i] = torch.exp(d[:, None] * s["A"].double()) * pool[i] + (d * x)[:, None] * Bm
            out.append(((pool[i] * Cm).sum(-1) + s["D"].double() * x) * _silu64(s["z"][n].double()))
        return torch.stack(out), pool
    if c["kind"].startswith("conv"):
        return _exact_conv(s, c)
    return _exact_norm(s, c) if c["kind"].startswith("norm") else _exact_scan(s, c)
