"""Gradients that autograd hands over as parts of a larger tensor: dense, but not 16-byte aligned."""
import pytest
import torch

import delta_rule_linear_chunked_amd as drl
from decay_util import make, tensors

NAMES = ("q", "k", "v", "alpha")


def test_a_part_of_a_tensor_is_copied_only_where_it_has_to_be():
    x = torch.arange(64.0)
    assert drl._dense(None) is None
    assert drl._dense(x) is x and drl._dense(x[4:]).data_ptr() == x[4:].data_ptr()
    for part in (x[1:], x[2:10].view(2, 4), x.view(8, 8).t()):
        y = drl._dense(part)
        assert torch.equal(y, part) and y.is_contiguous() and y.data_ptr() % 16 == 0


@pytest.mark.gpu
@pytest.mark.parametrize("node", ["decay", "delta rule"])
def test_outputs_joined_with_other_values(node):
    # the loss joins both outputs behind one number: their gradients start 4 bytes into the joined gradient
    x = make(81, 2, 70, 2, 2, 32, 32, "f32", "token")
    base = list(tensors(x, "f32").values())
    if node == "delta rule":
        base[3] = base[3][..., None].expand(2, 70, 2, 32).contiguous()

    def run(leaves):
        if node == "decay":
            return drl.decay_attention(*leaves)
        return drl.delta_rule(*leaves[:4], torch.full((2, 70, 2), 0.5, device="cuda"), variant="kda", S0=leaves[4])

    r = torch.Generator(device="cuda").manual_seed(1)
    leaves = [a.clone().requires_grad_() for a in base]
    o, S = run(leaves)
    w = torch.randn(1 + o.numel() + S.numel() + 1, generator=r, device="cuda")
    joined = torch.cat([torch.ones(1, device="cuda"), o.reshape(-1), torch.ones(1, device="cuda"), S.reshape(-1)])
    got = torch.autograd.grad((joined * w).sum(), leaves)
    leaves = [a.clone().requires_grad_() for a in base]
    o, S = run(leaves)
    n = o.numel()
    want = torch.autograd.grad((o, S), leaves, (w[1:1 + n].view(o.shape).clone(), w[n + 2:].view(S.shape).clone()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
