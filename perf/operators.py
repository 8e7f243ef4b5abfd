"""The decayed linear attention and the 8-bit state cache as they are measured: cases, inputs, plain forms and definitions.

Decayed linear attention: S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t, with a scalar decay a for each token and head (or one
for each head) and query/key heads that groups of value heads may share; its prefill, its single-token step and its gradients.
State cache: fp32 states written in 8 bits with a scale for each key channel, and read back.
"""
import math

import torch
import torch.nn.functional as F

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def _seq(kind, name, B, T, H, Hk, dk, dv, dtype, decay, packed=0, s0=True):
    """kind fwd / bwd; packed: number of sequences in one packed row of T tokens (B is then 1), 0 for B rows of T tokens."""
    c = {"kind": kind, "B": B, "T": T, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype, "decay": decay, "packed": packed, "s0": s0}
    return dict(c, name=name) if name else c


def _step(name, N, pool, H, Hk, dk, dv, dtype, decay):
    c = {"kind": "step", "N": N, "pool": pool, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype, "decay": decay}
    return dict(c, name=name) if name else c


def _cache(name, N, slots, H, dk, dv, fmt):
    c = {"kind": "cache", "N": N, "slots": slots, "H": H, "dk": dk, "dv": dv, "fmt": fmt}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a chat turn of a few tokens appended to a stored state: latency
        _seq("fwd", "prefill, one short turn", 1, 37, 16, 16, 128, 128, "bf16", "token"),
        # the library's own prefill workload
        _seq("fwd", "prefill", 4, 4096, 16, 16, 128, 128, "bf16", "token", s0=False),
        # the library's packed workload: twelve documents in one row; queries and keys shared by four value heads
        _seq("fwd", "prefill, packed, shared heads", 1, 32768, 16, 4, 128, 128, "bf16", "token", packed=12),
        # long context, few heads' worth of parallel work, signed decays
        _seq("fwd", "prefill, long, signed", 2, 16384, 16, 16, 128, 128, "bf16", "signed", s0=False),
        # fp32 evaluation of a small layer with a fixed decay for each head, odd lengths
        _seq("fwd", "prefill, fp32, decay per head", 3, 1333, 6, 2, 64, 32, "f32", "head"),
        # one user decoding: latency
        _step("step, one sequence", 1, 1, 16, 16, 128, 128, "bf16", "token"),
        # continuous batching out of a pool of slots
        _step("step, 512 sequences", 512, 520, 32, 32, 128, 128, "bf16", "token"),
        # a training step's backward at the prefill workload
        _seq("bwd", "backward", 4, 4096, 16, 16, 128, 128, "bf16", "token", s0=False),
        # packed documents, shared heads, a state head of another width than the value head
        _seq("bwd", "backward, packed, shared heads", 1, 7777, 12, 3, 64, 128, "bf16", "token", packed=5),
        # fp32 training of a small layer with a learned decay for each head
        _seq("bwd", "backward, fp32, decay per head", 2, 515, 4, 4, 64, 64, "f32", "head"),
        # the states of a full decode batch parked in the cache and resumed
        _cache("cache, 256 states, int8", 256, 300, 32, 128, 128, "int8"),
        # one prefix of a small layer parked and resumed
        _cache("cache, 3 states, e4m3", 3, 8, 16, 64, 128, "e4m3"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "fwd", "step", "step", "bwd", "bwd", "cache"])
    dk, dv = rng.choice([16, 32, 64, 128, 128]), rng.choice([16, 32, 64, 128, 128])
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 4])
    if kind == "cache":
        N = _logint(rng, 1, max(2, min(4096, 256 * 32 * 16384 // (H * dk * dv))))
        return _cache(None, N, N + rng.randrange(0, 9), H, dk, dv, rng.choice(["int8", "e4m3"]))
    if kind == "step":
        N = _logint(rng, 1, max(2, min(4096, 512 * 32 * 16384 // (H * dk * dv))))
        return _step(None, N, N + rng.randrange(0, 9), H, Hk, dk, dv, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["token", "signed", "head"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    room = (131072 if kind == "fwd" else 65536) // (4 if dtype == "f32" else 1)  # tokens of 16 heads in all
    tokens = _logint(rng, 1, max(2, room * 16 // max(H, 16)))
    packed = rng.choice([0, 0, 1])
    if packed:
        T = min(tokens, 32768)
        return _seq(kind, None, 1, T, H, Hk, dk, dv, dtype, rng.choice(["token", "signed", "head"]), packed=min(T, rng.randrange(1, 20)), s0=rng.random() < 0.7)
    B = min(rng.choice([1, 1, 2, 3, 4, 8]), tokens)
    return _seq(kind, None, B, max(1, min(tokens // B, 16384)), H, Hk, dk, dv, dtype, rng.choice(["token", "signed", "head"]), s0=rng.random() < 0.5)


def work(case):
    c = case
    dd = c["H"] * c["dk"] * c["dv"]
    if c["kind"] == "cache":
        return {"bytes": c["N"] * (dd * 10 + c["H"] * c["dk"] * 8), "flops": c["N"] * dd * 4}
    b = 2 if c["dtype"] == "bf16" else 4
    token = b * (2 * c["Hk"] * c["dk"] + c["H"] * c["dv"]) + (0 if c["decay"] == "head" else 4 * c["H"])
    if c["kind"] == "step":
        return {"bytes": c["N"] * (8 * dd + token + 4 * c["H"] * c["dv"]), "flops": 5 * c["N"] * dd}
    tokens, seqs = c["B"] * c["T"], c["packed"] or c["B"]
    if c["kind"] == "fwd":
        return {"bytes": tokens * (token + 4 * c["H"] * c["dv"]) + seqs * dd * 4 * (1 + c["s0"]), "flops": 4 * tokens * dd}
    grads = 4 * (2 * c["Hk"] * c["dk"] + c["H"] * c["dv"]) + (0 if c["decay"] == "head" else 4 * c["H"])
    return {"bytes": tokens * (token + 4 * c["H"] * c["dv"] + grads) + seqs * dd * 4 * (2 + c["s0"]), "flops": 10 * tokens * dd}


# ------------------------------------------------------------------------------------------------ inputs
def _decay(decay, shape, H, g):
    dev = "cuda"
    if decay == "head":  # the fixed decays of retention, 1 - 2^-(5 + h), spread over the heads
        return (1 - torch.exp2(-5 - 4 * torch.rand(H, generator=g, device=dev))).contiguous()
    z = torch.randn(shape, generator=g, device=dev)
    if decay == "signed":  # tanh gates in [-1, 1], a tenth of them +-1
        a = torch.tanh(1.5 * z)
        return torch.where(torch.rand(shape, generator=g, device=dev) < 0.1, torch.sign(z), a).contiguous()
    return torch.exp(-0.1 * F.softplus(z)).contiguous()


def _lengths(T, n, seed):
    """n positive lengths that sum to T, uneven."""
    r = torch.Generator().manual_seed(seed)
    cuts = torch.randperm(T - 1, generator=r)[: n - 1].sort().values + 1 if n > 1 else torch.empty(0, dtype=torch.long)
    return torch.diff(torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), T)]))


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    H, dk, dv = c["H"], c["dk"], c["dv"]
    s = {"case": c}
    if c["kind"] == "cache":
        s["S"] = rnd(c["N"], H, dk, dv) * torch.exp(rnd(c["N"], H, dk, 1))  # key channels of different size
        s["back"] = torch.zeros_like(s["S"])
        s["slots"] = torch.randperm(c["slots"], generator=g, device=dev)[: c["N"]].to(torch.int32)
        code = torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn
        s["codes"] = torch.zeros(c["slots"], H, dk, dv, device=dev, dtype=torch.int8).view(code)
        s["scales"] = torch.zeros(c["slots"], H, dk, device=dev)
        return s
    t = _T[c["dtype"]]
    unit = lambda *sh: F.normalize(rnd(*sh), dim=-1).to(t)  # noqa: E731
    if c["kind"] == "step":
        N = c["N"]
        s["q"], s["k"], s["v"] = unit(N, c["Hk"], dk), unit(N, c["Hk"], dk), rnd(N, H, dv).to(t)
        s["alpha"] = _decay(c["decay"], (N, H), H, g)
        s["S"] = rnd(c["pool"], H, dk, dv) / math.sqrt(dk)
        s["idx"] = torch.randperm(c["pool"], generator=g, device=dev)[:N].to(torch.int32)
        return s
    B, T = c["B"], c["T"]
    s["q"], s["k"], s["v"] = unit(B, T, c["Hk"], dk), unit(B, T, c["Hk"], dk), rnd(B, T, H, dv).to(t)
    s["alpha"] = _decay(c["decay"], (B, T, H), H, g)
    n = c["packed"] or B
    s["cu"], s["longest"] = None, T
    if c["packed"]:
        lens = _lengths(T, n, seed)
        s["longest"] = int(lens.max())
        s["cu"] = F.pad(lens.cumsum(0), (1, 0)).to(torch.int32).to(dev)
    s["S0"] = rnd(n, H, dk, dv) / math.sqrt(dk) if c["s0"] else None
    if c["kind"] == "bwd":
        s["dO"], s["dS_T"] = rnd(B, T, H, dv), rnd(n, H, dk, dv)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
C = 64  # tokens of a chunk


def _rows(s, x):
    """[B, T, ...] as [sequences, longest, ...]: packed tokens by sequence, zeros behind each."""
    if s["cu"] is None:
        return x
    at = s["cu"][:-1, None].long() + torch.arange(s["longest"], device=x.device)
    inside = at < s["cu"][1:, None]
    return x[0][at.clamp(max=x.shape[1] - 1)] * inside.view(inside.shape + (1,) * (x.dim() - 2))


def _packed(s, x, B, T):
    """_rows undone."""
    if s["cu"] is None:
        return x
    t = torch.arange(T, device=x.device)
    n = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return x[n, t - s["cu"][n].long()][None]


def _chunked(s, x, heads=1):
    """[B, T, H, d] as [sequences, H, chunks, C, d] in 32 bits, shared heads repeated, zeros behind the end."""
    x = _rows(s, x).float().repeat_interleave(heads, dim=2)
    x = F.pad(x, (0, 0, 0, 0, 0, -x.shape[1] % C))
    return x.view(x.shape[0], -1, C, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4).contiguous()


def _flat(s, x, B, T):
    """_chunked undone (heads as they are)."""
    x = x.permute(0, 2, 3, 1, 4)
    x = x.reshape(x.shape[0], -1, x.shape[3], x.shape[4])
    return _packed(s, x[:, : s["longest"]], B, T).contiguous()


def _products(a):
    """Of the decays a [..., C]: ratio(r, s) = a_{s+1} ... a_r for s <= r else 0, as [..., C, C], and the running product of
    the first r + 1 of them; exact zeros and signs kept apart from the logarithms, which are summed in 64 bits."""
    none, sign = (a == 0).cumsum(-1), torch.where(a < 0, -1.0, 1.0).cumprod(-1)
    c = torch.where(a == 0, 0.0, a.double().abs().log()).cumsum(-1)
    low = torch.ones(a.shape[-1], a.shape[-1], dtype=torch.bool, device=a.device).tril()
    on = low & (none[..., :, None] == none[..., None, :])
    ratio = (c[..., :, None] - c[..., None, :]).masked_fill(~on, -math.inf).exp().float()
    ratio = ratio * sign[..., :, None] * sign[..., None, :]
    return ratio, (c.masked_fill(none > 0, -math.inf).exp().float() * sign)


def _decays(s, B, T, H):
    a = s["alpha"]
    a = a.expand(B, T, H) if a.dim() == 1 else a
    if s["cu"] is not None:  # ones behind each sequence
        inside = (torch.arange(s["longest"], device=a.device) < torch.diff(s["cu"])[:, None])[..., None]
        a = torch.where(inside, _rows(s, a), 1.0)
    a = F.pad(a, (0, 0, 0, -a.shape[1] % C), value=1.0)
    a = a.view(a.shape[0], -1, C, H).permute(0, 3, 1, 2).contiguous()  # [sequences, H, chunks, C]
    ratio, gamma = _products(a)
    return a, ratio, gamma


def _between(gamma_end, local, first):
    """States at each chunk's start (and behind the last) from the chunks' own contributions [.., chunks, dk, dv] and the state before the first."""
    ratio, run = _products(gamma_end)  # over chunks
    n = gamma_end.shape[-1]
    ends = (ratio @ local.flatten(-2)).view_as(local)
    if first is not None:
        ends = ends + run[..., None, None] * first[:, :, None]
    before = torch.zeros_like(ends[:, :, :1]) if first is None else first[:, :, None]
    return torch.cat([before, ends[:, :, : n - 1]], 2), ends[:, :, n - 1]


def _plain_fwd(s):
    c = s["case"]
    g = c["H"] // c["Hk"]
    q, k, v = _chunked(s, s["q"], g), _chunked(s, s["k"], g), _chunked(s, s["v"])
    _, ratio, gamma = _decays(s, c["B"], c["T"], c["H"])
    local = k.transpose(-1, -2) @ (ratio[..., -1, :, None] * v)
    S0, S_T = _between(gamma[..., -1].contiguous(), local, s["S0"])
    o = ((q @ k.transpose(-1, -2)) * ratio) @ v + gamma[..., None] * (q @ S0)
    return _flat(s, o, c["B"], c["T"]), S_T.contiguous()


def _plain_bwd(s):
    c = s["case"]
    g = c["H"] // c["Hk"]
    q, k, v, dO = _chunked(s, s["q"], g), _chunked(s, s["k"], g), _chunked(s, s["v"]), _chunked(s, s["dO"])
    _, ratio, gamma = _decays(s, c["B"], c["T"], c["H"])
    end, tail = gamma[..., -1].contiguous(), ratio[..., -1, :]
    S0, _ = _between(end, k.transpose(-1, -2) @ (tail[..., None] * v), s["S0"])
    back, dS0 = _between(end.flip(-1), (q.transpose(-1, -2) @ (gamma[..., None] * dO)).flip(2), s["dS_T"])
    dS = back.flip(2)
    qk, ov = q @ k.transpose(-1, -2), dO @ v.transpose(-1, -2)
    P, E = qk * ratio, ov * ratio
    inq, ink = dO @ S0.transpose(-1, -2), v @ dS.transpose(-1, -2)
    dq = E @ k + gamma[..., None] * inq
    dk = E.transpose(-1, -2) @ q + tail[..., None] * ink
    dv = P.transpose(-1, -2) @ dO + tail[..., None] * (k @ dS)
    # da_t: what reaches rows r >= t from tokens s < t and from the start state, and what reaches the chunk's end
    upto = F.pad(ratio, (0, 0, 1, 0))[..., :-1, :]  # ratio(t - 1, s)
    start = F.pad(gamma, (1, 0), value=1.0)[..., :-1]  # the product before t
    X, Y, Z = (q * inq).sum(-1), (k * ink).sum(-1), (S0 * dS).sum((-1, -2))
    rows = (qk * ov) @ upto.transpose(-1, -2) + X[..., :, None] * start[..., None, :]
    da = (ratio * rows).sum(-2) + tail * ((upto @ Y[..., None])[..., 0] + start * Z[..., None])
    da = _flat(s, da[..., None], c["B"], c["T"])[..., 0]
    if c["decay"] == "head":
        da = da.sum((0, 1), dtype=torch.float64).float()
    shared = lambda x: _flat(s, x, c["B"], c["T"]).unflatten(2, (c["Hk"], g)).sum(3)  # noqa: E731
    return {"dq": shared(dq), "dk": shared(dk), "dv": _flat(s, dv, c["B"], c["T"]), "dalpha": da, "dS0": dS0.contiguous()}


def _plain_step(s):
    c = s["case"]
    g = c["H"] // c["Hk"]
    q, k, v = (s[x].float() for x in "qkv")
    q, k = q.repeat_interleave(g, 1), k.repeat_interleave(g, 1)
    a = s["alpha"] if c["decay"] != "head" else s["alpha"].expand(c["N"], c["H"])
    i = s["idx"].long()
    S = s["S"][i] * a[..., None, None] + k[..., :, None] * v[..., None, :]
    s["S"][i] = S
    return (S * q[..., None]).sum(-2), s["S"]


def _e4m3(x):
    """x rounded to the nearest value of 4 exponent and 3 fraction bits, ties to even (|x| <= 448)."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4
    return torch.ldexp(torch.round(torch.ldexp(x, -e)), e)


def _plain_cache(s):
    c = s["case"]
    x = s["S"]
    top = x.abs().amax(-1)
    if c["fmt"] == "int8":
        scale = (top / 127).clamp(min=2.0 ** -126)
        held = torch.round(x.double() / scale.double()[..., None]).float()  # 64 bits: quotients next to a half
    else:
        m, e = torch.frexp(top)
        scale = torch.ldexp(torch.ones_like(top), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
        scale = torch.where(top == 0, 2.0 ** -126, scale)
        held = _e4m3(x / scale[..., None])
    i = s["slots"].long()
    s["codes"][i] = held.to(s["codes"].dtype)
    s["scales"][i] = scale
    s["back"].copy_(s["codes"][i].float() * s["scales"][i][..., None])
    return s["back"], s["scales"]


def run(state):
    s = state
    kind = s["case"]["kind"]
    if own:
        import delta_rule_linear_chunked_amd as drl

        if kind == "fwd":
            return drl.decay_fwd(s["q"], s["k"], s["v"], s["alpha"], S0=s["S0"], cu_seqlens=s["cu"])
        if kind == "bwd":
            return drl.decay_bwd(s["q"], s["k"], s["v"], s["alpha"], S0=s["S0"], cu_seqlens=s["cu"], dO=s["dO"], dS_T=s["dS_T"])
        if kind == "step":
            return drl.decay_step(s["q"], s["k"], s["v"], s["alpha"], s["S"], state_idx=s["idx"]), s["S"]
        drl.dr_state_pack(s["S"], s["codes"], s["scales"], slot_idx=s["slots"])
        drl.dr_state_unpack(s["codes"], s["scales"], s["back"], slot_idx=s["slots"])
        return s["back"], s["scales"]
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "cache": _plain_cache}[kind](s)


# ------------------------------------------------------------------------------------------------ definitions in 64 bits
def _pairs(s):
    """(batch row, first token, tokens, sequence) of each sequence."""
    if s["cu"] is None:
        return [(n, 0, s["case"]["T"], n) for n in range(s["case"]["B"])]
    cu = s["cu"].tolist()
    return [(0, a, b - a, n) for n, (a, b) in enumerate(zip(cu, cu[1:]))]


def _weights(a):
    """w[r, s] = a_{s+1} ... a_r over a whole sequence (s <= r), and the products from its start; a has no zeros."""
    c, sg = a.abs().log().cumsum(0), torch.where(a < 0, -1.0, 1.0).double().cumprod(0)
    w = (c[:, None] - c[None, :]).masked_fill_(~torch.ones(len(a), len(a), dtype=torch.bool, device=a.device).tril(), -math.inf).exp_()
    return w.mul_(sg[:, None]).mul_(sg[None, :]), c.exp() * sg


def _exact_seq(s):
    """Every pair of tokens of a sequence at once, head by head."""
    c = s["case"]
    B, T, H, Hk, dk, dv = (c[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    f = lambda *sh: torch.zeros(sh, dtype=torch.float64, device="cuda")  # noqa: E731
    n = c["packed"] or B
    o, S_T = f(B, T, H, dv), f(n, H, dk, dv)
    dq, dk_, dv_, da, dS0 = f(B, T, Hk, dk), f(B, T, Hk, dk), f(B, T, H, dv), f(B, T, H), f(n, H, dk, dv)
    for b, t0, L, j in _pairs(s):
        for h in range(H):
            hk, t = h // (H // Hk), slice(t0, t0 + L)
            q, k, v = s["q"][b, t, hk].double(), s["k"][b, t, hk].double(), s["v"][b, t, h].double()
            a = s["alpha"][b, t, h].double() if s["alpha"].dim() == 3 else s["alpha"][h].double().expand(L)
            S0 = f(dk, dv) if s["S0"] is None else s["S0"][j, h].double()
            w, run_ = _weights(a)
            qk = q @ k.T
            if c["kind"] == "fwd":
                o[b, t, h] = (w * qk) @ v + run_[:, None] * (q @ S0)
                S_T[j, h] = run_[-1] * S0 + (w[-1][:, None] * k).T @ v
                continue
            dO, dS = s["dO"][b, t, h].double(), s["dS_T"][j, h].double()
            E = (dO @ v.T) * w
            dq[b, t, hk] += E @ k + run_[:, None] * (dO @ S0.T)
            dk_[b, t, hk] += E.T @ q + w[-1][:, None] * (v @ dS.T)
            dv_[b, t, h] = (w * qk).T @ dO + w[-1][:, None] * (k @ dS)
            dS0[j, h] = run_[-1] * dS + (run_[:, None] * q).T @ dO
            # every path from s (or the start) to r (or the end) that passes token t carries a_t once
            W = E * qk
            into = W.sum(1) + run_ * (q * (dO @ S0.T)).sum(1)
            out = W.sum(0) + w[-1] * (k * (v @ dS.T)).sum(1)
            end = (dS * (run_[-1] * S0 + (w[-1][:, None] * k).T @ v)).sum()
            da[b, t, h] = (end + (into - out).flip(0).cumsum(0).flip(0)) / a
    if c["kind"] == "fwd":
        return o, S_T
    return {"dq": dq, "dk": dk_, "dv": dv_, "dalpha": da.sum((0, 1)) if c["decay"] == "head" else da, "dS0": dS0}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] in ("fwd", "bwd"):
        return _exact_seq(s)
    if c["kind"] == "step":
        r = torch.arange(c["H"], device="cuda") // (c["H"] // c["Hk"])
        pool, o = s["S"].double(), []
        for n, i in enumerate(s["idx"].tolist()):  # one sequence after another
            a = (s["alpha"][n] if s["alpha"].dim() == 2 else s["alpha"]).double()
            pool[i] = a[:, None, None] * pool[i] + torch.einsum("hk,hv->hkv", s["k"][n, r].double(), s["v"][n].double())
            o.append(torch.einsum("hkv,hk->hv", pool[i], s["q"][n, r].double()))
        return torch.stack(o), pool
    back, scales = torch.empty(s["S"].shape, dtype=torch.float64, device="cuda"), s["scales"].double()
    grid = None
    if c["fmt"] == "e4m3":  # all the values that the format has, in order
        bits = torch.arange(127, device="cuda")
        e, m = bits // 8, (bits % 8).double()
        grid = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    for n, i in enumerate(s["slots"].tolist()):
        x = s["S"][n].double()
        top = x.abs().amax(-1)
        if c["fmt"] == "int8":
            sc = (top / 127).float().double().clamp(min=2.0 ** -126)  # a scale is a 32-bit number
            held = torch.round(x / sc[..., None])
        else:
            sc = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-126))
            y = (x / sc[..., None]).abs().contiguous()
            up = torch.searchsorted(grid, y).clamp(max=126)
            lo, hi = grid[(up - 1).clamp(min=0)], grid[up]
            even = torch.where(up % 2 == 0, hi, lo)  # of two neighbours the one with an even fraction
            near = torch.where(y - lo < hi - y, lo, torch.where(y - lo > hi - y, hi, even))
            held = torch.where(y == hi, hi, near) * torch.sign(x)
        back[n], scales[i] = held * sc[..., None], sc
    return back, scales
