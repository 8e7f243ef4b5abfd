"""The selective scan cut into segments, with every number of states and with groups, against its definition in float64; and the
convolution's autograd node with one output unused."""
import pytest

import delta_rule_linear_chunked_amd as drl
from gpu_util import seed_of
from layer_util import dev, make_conv, make_scan
from test_gpu_conv import check_bwd
from test_gpu_scan import check, check_grad

pytestmark = pytest.mark.gpu
CU = [0, 0, 1, 3, 3, 40, 41, 90, 90]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [8, 16, 40])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("cu", [None, CU, [0, 64, 72, 72, 75]])
def test_segments(cu, N, seg, dtype, monkeypatch):
    monkeypatch.setenv("DR_SCAN_SEG", str(seg))
    B = 2 if cu is None else 1
    x = make_scan(seed_of("states", cu, N, seg, dtype), B, 97, 99, 3, N, dtype, n=B if cu is None else len(cu) - 1)
    check(x, dtype, cu)
    check_grad(x, dtype, cu)


@pytest.mark.parametrize("used", [0, 1])
def test_a_convolution_with_one_output_unused(used):
    x = make_conv(3, 2, 30, 40, 4, "f32")
    x["dy" if used else "dl"][:] = 0
    leaves = [dev(x[k]).requires_grad_() for k in ("x", "w", "b", "state")]
    (drl.causal_conv(*leaves)[used] * dev(x["dl" if used else "dy"])).sum().backward()
    check_bwd(x, "f32", None, "silu", got=dict(zip(("dx", "dweight", "dbias", "dstate"), (t.grad for t in leaves))))
    # and without bias and state
    a, w = dev(x["x"]).requires_grad_(), dev(x["w"]).requires_grad_()
    (drl.causal_conv(a, w)[used] * dev(x["dl" if used else "dy"])).sum().backward()
    check_bwd(x, "f32", None, "silu", state=False, bias=False, got=dict(dx=a.grad, dweight=w.grad, dbias=None, dstate=None))
