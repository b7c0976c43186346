"""The activations of the block-scaled Linear's epilogue alone, at every bf16 argument: codes of
zero leave the bias as the sum, exactly.  Room: the errors that the header gives them, the
float32 products' 2^-21 and one rounding to bf16."""
import numpy as np
import pytest
import torch

from oracle import ops
from oracle.formats import bf16_decode
from parity import from_bits, to_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    return g


@pytest.mark.parametrize("m", [1, 40, 100, 1024])
@pytest.mark.parametrize("act", [1, 2, 3])
def test_activation_of_every_bf16(gbf, m, act):
    n = 65536
    assert m != 1024 or gbf.linear_fp8_block_plan(m, n, 128)[0] == 256
    z = np.arange(n, dtype=np.uint16)
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gbf.linear_fp8_block(torch.zeros(m, 128, dtype=torch.uint8, device="cuda"), torch.ones(m, 1, device="cuda"),
                         torch.zeros(n, 128, dtype=torch.uint8, device="cuda"), torch.ones(n // 128, 1, device="cuda"),
                         from_bits(z), y, act=act)
    torch.cuda.synchronize()
    assert (y == y[:1]).all(0).logical_or(y.isnan().all(0)).all()
    got, a = bf16_decode(to_bits(y[m - 1])), bf16_decode(z)
    finite = np.isfinite(a)
    with np.errstate(all="ignore"):
        ref = ops.activation(a, act)
        if act == 3:
            # the fast exponential's 2 + 1.2 |z| ulp, the fast division's 2, which is 0 for divisors above 2^126
            room = np.abs(ref) * (8 + 2 * np.abs(a)) * 2.0 ** -23 + np.abs(a) * 2.0 ** -126
        else:
            # half of |z| times the tanh's 2^-10.9, or the erf's 1.5e-7 and some five roundings of values up to 1
            room = np.abs(a) * (2.0 ** -11.9 if act == 1 else 2.0 ** -21) + np.abs(ref) * 2.0 ** -21
        room = room + (np.abs(ref) + room) * 2.0 ** -8 + 2.0 ** -133
        bad = finite & ~(np.abs(got - ref) <= room)
    assert not bad.any(), (bad.sum(), a[bad][:4], got[bad][:4], ref[bad][:4], room[bad][:4])
    assert np.isnan(got[np.isnan(a)]).all() and got[a == np.inf].tolist() == [np.inf]
