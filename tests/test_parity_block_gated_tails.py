"""The gated activations far out, where act(gate) is tiny and its error grows with the exponent:
down to the least scale, 2^-100.  The room is test_parity_block_quant's: of SiLU and the
tanh GELU 10 + 4 |z| units of 2^-23, z the logistic function's argument, of the erf GELU 10 + g^2.

The reference has no 1 + tanh or 1 + erf: in float64 those are off by 2^-54, which is more
than all of the value from z = -37 on.  g exp(z) / (1 + exp(z)) and g erfc(-g / sqrt 2) / 2 keep
2^-52 (2 + |z|) of it."""
import math

import numpy as np
import pytest

from oracle.formats import bf16_decode, bf16_encode
from test_parity_block_quant import ACTS, U, bits, check_codes, gbf, run_gated        # noqa: F401

pytestmark = pytest.mark.gpu

GATES = {"silu": (-8, -20, -40, -60, -71), "gelu_tanh": (-5.5, -6.5, -7.5, -8.5, -9.3), "gelu_erf": (-6, -8, -10, -11, -11.9)}


def tail_ref(x, act):
    v = bf16_decode(x)
    g, up = v[:, :v.shape[1] // 2], v[:, v.shape[1] // 2:]
    if act == "gelu_erf":
        a, ulps = g * 0.5 * np.vectorize(math.erfc)(-g / math.sqrt(2)), 10 + g * g
    else:
        z = g if act == "silu" else 2 * 0.7978845608 * (g + 0.044715 * g ** 3)
        a, ulps = g * np.exp(z) / (1 + np.exp(z)), 10 + 4 * np.abs(z)
    return a * up, np.abs(a * up) * ulps * 2 * U + np.abs(up) * 2.0 ** -125


@pytest.mark.parametrize("act", list(ACTS))
def test_far_tails(gbf, act):                                                         # noqa: F811
    rng = np.random.default_rng(21)
    x = bits(rng, 10, 512)
    for r, at in enumerate(GATES[act]):
        x[r, :256] = bf16_encode(at + 0.5 * rng.random(256))
        x[5 + r, :256] = bf16_encode(at * (1 + 0.02 * rng.standard_normal(256)))
        x[r, 256:] = bf16_encode(np.exp2(rng.integers(-3, 20, 256)) * rng.choice([-1, 1], 256))
    codes, scales = run_gated(gbf, x, act)
    check_codes(codes, scales, *tail_ref(x, act))
    assert ((codes & 0x7F) != 0).any(1)[:4].all()          # the rows are no zeros
