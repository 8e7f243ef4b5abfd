"""The largest numbers of (sequence, head) pairs that a call takes, with small heads of one token: the first, the last and
some sequences between against float64."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from decay_util import close, oracle
from gpu_util import seed_of
from oracle.decay import pack

pytestmark = pytest.mark.gpu
H, D = 16, 16


def inputs(N, name):
    """bf16 q, k, v of N sequences of one token, fp32 decays, and the sequences that are looked at."""
    g = torch.Generator(device="cuda").manual_seed(seed_of("largest", name))
    r = lambda h: (torch.randn(N, 1, h, D, generator=g, device="cuda", dtype=torch.float32) / 4).bfloat16()  # noqa: E731
    q, k, v = r(1), r(1), r(H)
    a = torch.rand(N, 1, H, generator=g, device="cuda")
    look = torch.tensor([0, 1, N // 3, N // 2, N - 2, N - 1], device="cuda")
    return q, k, v, a, look


def picked(look, *ts):
    return [t[look].float().cpu().numpy() for t in ts]


def test_prefill():
    N = 349520  # 5592320 workgroups of 768 threads
    q, k, v, a, look = inputs(N, "fwd")
    o, S = drl.decay_fwd(q, k, v, a)
    args = picked(look, q, k, v, a)
    want, mag = oracle.forward(*args), oracle.forward(*args, magnitudes=True)
    close(o[look], want[0], mag[0], 1, "o")
    close(S[look], want[1], mag[1], 1, "S_T")


def test_gradients():
    N = 524287  # 8388592 workgroups of 512 threads
    q, k, v, a, look = inputs(N, "bwd")
    dO = torch.randn(N, 1, H, D, device="cuda")
    dS = torch.randn(N, H, D, D, device="cuda")
    g = drl.decay_bwd(q, k, v, a, dO=dO, dS_T=dS)
    args = picked(look, q, k, v, a, dO, dS)
    want, mag = oracle.backward(*args), oracle.backward(*args, magnitudes=True)
    for n in ("dq", "dk", "dv", "dalpha", "dS0"):
        # (a term's sums: 16 channels twice, 16 heads, and the roundings of one token's chunk)
        close(g[n][look], want[n], mag[n], 1, n, 48)


def test_step():
    N = (1 << 22) - 1  # 67108848 workgroups of 64 threads
    q, k, v, a, look = inputs(N, "step")
    one = [t[:, 0].contiguous() for t in (q, k, v, a)]
    S = torch.full((N, H, D, D), 0.5, device="cuda")
    o = drl.decay_step(*one, S)
    args = picked(look, *one)
    S0 = np.full((len(look), H, D, D), 0.5, np.float32)
    (wS, wo), (mS, mo) = oracle.step(S0, *args), oracle.step(S0, *args, magnitudes=True)
    close(S[look], wS, mS, 1, "S")
    close(o[look], wo, mo, 1, "o")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_cache(fmt):
    N = (1 << 20) - 1  # 16777200 workgroups of 256 threads
    S = torch.randn(N, H, D, D, device="cuda")
    codes, scales = drl.state_pack(S, fmt)
    back = drl.state_unpack(codes, scales)
    look = torch.tensor([0, N // 2, N - 1], device="cuda")
    held, sc = pack(S[look].cpu().numpy(), fmt)
    assert np.array_equal(scales[look].cpu().double().numpy(), sc)
    assert np.array_equal(back[look].cpu().numpy(), held.astype(np.float32))
