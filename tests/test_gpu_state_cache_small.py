"""int8 codes of the state cache where half a scale is not a float32 number: scales between 2^-126 and 2^-125, whose
last place is the smallest subnormal."""
import numpy as np
import pytest

import delta_rule_linear_chunked_amd as drl
from decay_util import dev
from oracle import decay as oracle

pytestmark = pytest.mark.gpu


def rows():
    """Rows of halves of the scale and of their neighbours on both sides, all scales odd multiples of 2^-149."""
    r = np.random.default_rng(11)
    tiny, out = 2.0 ** -149, []
    while len(out) < 64:
        top = np.float32(127 * r.integers(1 << 23, 1 << 24) * tiny)
        scale = oracle.pack(top[None, None], "int8")[1][0]
        units = int(round(scale / tiny))
        if units % 2 == 0 or not 1 << 23 <= units < 1 << 24:
            continue
        k = np.arange(-62, 63)
        half = (2 * k + 1) * units / 2.0 * tiny  # float64: exact
        pick = r.integers(-1, 2, k.size)
        x = half.astype(np.float32)
        x = np.where(pick < 0, np.nextafter(x, np.float32(-1)), np.where(pick > 0, np.nextafter(x, np.float32(1)), x))
        out.append(np.concatenate([[top], x, np.zeros(2)]).astype(np.float32))
    return np.stack(out)


def test_codes_are_those_of_the_exact_quotient():
    S = rows().reshape(4, 1, 16, 128)
    codes, scales = drl.state_pack(dev(S), "int8")
    held, sc = oracle.pack(S, "int8")
    assert np.array_equal(scales.cpu().double().numpy(), sc)
    got = codes.cpu().numpy()
    want = np.rint(S.astype(np.float64) / sc[..., None])
    assert np.array_equal(got, want), f"{np.sum(got != want)} of {got.size} codes differ"
