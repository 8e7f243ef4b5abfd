"""The selective scan's step d = softplus(dt + bias): to a few units in the last place over its range, and at infinities."""
import numpy as np
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from layer_util import dev, oracle

pytestmark = pytest.mark.gpu

# In units of 2^-23 of d. What is left of the exponent's rounding (LN2 in float32, 2.7e-9 of |v|) 0.4 at 16, exp2 1, the product that puts it
# back 1/2, 2 + e 1/2, rcp 1, e / (2 + e) 1/2, its square's errors through the polynomial's slope (at most a third of it) 1, the fit 0.1, the
# polynomial's last sum 1/2, d 1/2.
ULPS = 6
V = np.concatenate([np.linspace(-16, 16, 4001), -np.exp(np.linspace(-20, np.log(16), 500)), np.exp(np.linspace(-20, 4, 500)), [0.0]]).astype(np.float32)


def one_token(v, N=16):
    """Inputs of one token with A = 0, x = B = 1 and no state in front of it: the new state is d."""
    C = len(v)
    return dict(x=torch.ones(1, 1, C, device="cuda"), dt=dev(v).view(1, 1, C), A=torch.zeros(C, N, device="cuda"),
                B=torch.ones(1, 1, 1, N, device="cuda"), C=torch.ones(1, 1, 1, N, device="cuda"))


def check(d, v):
    want = oracle.softplus(v.astype(np.float64))
    err = np.abs(d.double().cpu().numpy() - want) / (want * 2.0 ** -23)
    assert err.max() <= ULPS, f"{err.max():.2f} units at {v[err.argmax()]}"


@pytest.mark.parametrize("block", ["1", "2"])
@pytest.mark.parametrize("N", [16, 32, 64])
def test_step_sizes(N, block, monkeypatch):
    monkeypatch.setenv("DR_SCAN_BLOCK", block)
    a = one_token(V, N)
    S = drl.scan_fwd(**a)[1][0]
    assert (S == S[:, :1]).all()
    check(S[:, 0], V)


def test_step_sizes_of_single_tokens():
    a, S = one_token(V), torch.zeros(1, len(V), 16, device="cuda")
    drl.scan_step(*[a[k] if k == "A" else a[k][0] for k in ("x", "dt", "A", "B", "C")], S)
    check(S[0, :, 3], V)


def test_step_sizes_of_gradients():
    # with a gradient of 1 at one state: dx is d
    a, dS = one_token(V), torch.zeros(1, len(V), 16, device="cuda")
    dS[..., 2] = 1.0
    check(drl.scan_bwd(**a, dy=torch.zeros_like(a["x"]), dS_T=dS)["dx"][0, 0], V)


@pytest.mark.parametrize("softplus", [True, False])
def test_steps_given_and_infinite(softplus, monkeypatch):
    # steps that are used as they are come through bit for bit; softplus of -infinity, and of what exp takes to zero, is zero and leaves the state
    v = V if not softplus else np.array([-np.inf, -3.3e38, -1e5, -200.0], np.float32)
    a = one_token(v)
    start = torch.randn(1, len(v), 16, device="cuda") * float(softplus)
    want = start if softplus else dev(v).view(1, -1, 1).expand(1, -1, 16)
    for block in ("1", "2"):
        monkeypatch.setenv("DR_SCAN_BLOCK", block)
        assert (drl.scan_fwd(**a, S0=start, softplus=softplus)[1] == want).all()
    S = start.clone()
    drl.scan_step(*[a[k] if k == "A" else a[k][0] for k in ("x", "dt", "A", "B", "C")], S, softplus=softplus)
    assert (S == want).all()
    top = drl.scan_fwd(**one_token(np.array([np.inf, np.nan], np.float32)), softplus=softplus)[1]
    assert not torch.isfinite(top).any()
