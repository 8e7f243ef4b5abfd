"""The selective scan over packed rows of many sequences on the GPU: results against the definition in float64, with the
segments that the library chooses, and in workspaces of the stated size."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from delta_rule_linear_chunked_amd import _scan
from layer_util import SCAN_IN, i32, make_scan, scan_tensors
from test_gpu_layer_use import GRADS, call_lib, need
from test_gpu_scan import NAMES, check, check_grad

pytestmark = pytest.mark.gpu


def documents(n, mean, long, seed):
    """Offsets of n documents of uneven lengths (some of them empty), the middle one `long` tokens."""
    r = np.random.default_rng(seed)
    lens = r.geometric(1 / mean, n) - 1
    lens[n // 2] = long
    return [0, *(int(a) for a in np.cumsum(lens))]


@pytest.mark.parametrize("dtype,C,G,N", [("bf16", 72, 1, 16), ("f32", 66, 2, 32), ("bf16", 33, 1, 64)])
def test_many_documents(dtype, C, G, N):
    cu = documents(300, 6, 400, 1)
    T = cu[-1] + 5
    x = make_scan(31 + N, 1, T, C, G, N, dtype, n=300)
    check(x, dtype, cu)
    t = scan_tensors(x, dtype)
    g = {n: torch.full_like(t[GRADS[n]], 7.0) for n in NAMES}
    drl.dr_scan_bwd(*[t[k] for k in SCAN_IN], t["S0"], i32(cu), t["dy"], t["dS"], *[g[n] for n in NAMES])
    check_grad(x, dtype, cu, got=g)
    for n in ("dx", "ddt", "dB", "dC", "dz"):
        assert (g[n][:, cu[-1]:] == 7.0).all(), n


@pytest.mark.parametrize("seg", [0, 8, 16, 56])
@pytest.mark.parametrize("cu", [documents(300, 6, 400, 1), [0, 7, 15, 23, 31, 32, 33, 41, 57], [0, 1, 9, 9, 9, 17, 18, 82, 90]])
def test_a_workspace_of_the_stated_size_is_enough(cu, seg, monkeypatch):
    # between guard bands, filled with NaN bits before the call; with segments of one length the same bits as each sequence by itself
    if seg:
        monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    n, T = len(cu) - 1, cu[-1]
    t = scan_tensors(make_scan(3, 1, T, 40, 1, 16, "bf16", n=n), "bf16")
    d = _scan._scan_inputs(*[t[k] for k in SCAN_IN], True, 2)
    d.num_seqs = n
    size = need("dr_scan_workspace", d, 1, 1)
    g = {k: torch.full_like(t[v], float("nan")) for k, v in GRADS.items()}
    buf = torch.full((size + (2 << 20),), 255, dtype=torch.uint8, device="cuda")
    args = [t[k] for k in SCAN_IN] + [t["S0"], i32(cu), t["dy"], t["dS"], *g.values()]
    assert call_lib("dr_scan_bwd", args, d, buf.data_ptr() + (1 << 20), size) == 0
    torch.cuda.synchronize()
    assert (buf[:1 << 20] == 255).all() and (buf[(1 << 20) + size:] == 255).all()
    assert not any(a.isnan().any() for a in g.values())
    for i in range(n if seg and n <= 8 else 0):
        if cu[i] == cu[i + 1]:
            assert torch.equal(g["dS0"][i], t["dS"][i])
            continue
        one = {k: (t[k] if k in ("A", "D", "bias") else t[k][:, cu[i]:cu[i + 1]]) for k in SCAN_IN}
        w = drl.scan_bwd(*one.values(), S0=t["S0"][i:i + 1], dy=t["dy"][:, cu[i]:cu[i + 1]].contiguous(), dS_T=t["dS"][i:i + 1])
        for k in ("dx", "ddt", "dB", "dC", "dz"):
            assert torch.equal(g[k][:, cu[i]:cu[i + 1]], w[k]), (i, k)
        assert torch.equal(g["dS0"][i], w["dS0"][0]), i
