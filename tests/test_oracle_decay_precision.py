"""The norm bound of the decayed linear attention's tests tells the evaluation that the kernels use from those that lose
bits: two bf16 terms of an operand instead of three, and products of decays rounded one after another."""
import pytest

from decay_norm import LIMIT, exact, model, norm_error
from decay_util import make


@pytest.mark.parametrize("decay", ["token", "head"])
def test_two_terms_are_not_enough(decay):
    x = make(91, 1, 300, 2, 1, 64, 64, "f32", decay)
    want = exact(x)
    for got, w in zip(model(x), want):
        assert norm_error(got, w) <= LIMIT / 4
    for got, w in zip(model(x, n=2), want):
        assert norm_error(got, w) > LIMIT


def test_products_of_decays_in_fp32_are_not_enough():
    x = make(92, 1, 1333, 6, 2, 32, 32, "f32", "head")
    # one decay for each head, close to 1: every chunk leaves the same roundings
    x["alpha"][:] = 1 - 2.0 ** -9 * (1 + 0.1 * x["alpha"])
    want = exact(x)
    for got, w in zip(model(x), want):
        assert norm_error(got, w) <= LIMIT / 4
    o, S = model(x, wide=False)
    assert norm_error(S, want[1]) > LIMIT
