"""The block-scaled oracle against worked examples, closed forms and brute force."""
import numpy as np

from oracle import block, ops
from oracle.formats import e4m3_decode, e4m3_encode_sat


def test_scales_worked():
    y = np.zeros((2, 200), np.float32)
    y[0, 3], y[0, 127], y[0, 128] = -448.0, 56.0, 7.0
    codes, s = block.quantize(y)
    assert s.shape == (2, 2) and s[0, 0] == 1.0 and (s[1] == np.float32(2.0 ** -100)).all()
    assert np.isclose(s[0, 1], 7 / 448, rtol=2 ** -23)
    v = e4m3_decode(codes)
    assert v[0, 3] == -448 and v[0, 127] == 56 and v[0, 128] == 448 and not v[1].any()


def test_scale_of_a_tile():
    y = np.zeros((130, 130), np.float32)
    y[0, 0], y[127, 127], y[128, 0], y[129, 129] = 1, -3, 5, 7
    _, s = block.quantize(y, 128)
    assert np.allclose(s * 448, [[3, 2.0 ** -100 * 448], [5, 7]], rtol=2 ** -22)


def test_special_values():
    y = np.ones((3, 16), np.float32)
    y[0, 2], y[1, 5], y[2, 7] = np.nan, np.inf, -np.inf
    codes, s = block.quantize(y)
    assert np.isnan(s[0, 0]) and (codes[0] == 0x7F).all()
    for r, c in ((1, 5), (2, 7)):
        assert s[r, 0] == np.inf and codes[r, c] == 0x7F and (np.delete(codes[r], c) == 0).all()


def test_a_power_of_two_scales_everything():
    y = np.random.default_rng(0).standard_normal((4, 300)).astype(np.float32)
    codes, s = block.quantize(y)
    more, t = block.quantize(y * np.float32(64))
    assert (codes == more).all() and (t == 64 * s).all()


def test_dequantised_is_within_half_a_step():
    y = np.random.default_rng(1).standard_normal((8, 512)).astype(np.float32)
    codes, s = block.quantize(y)
    s = block.spread(s, *y.shape)
    # half a step of three fraction bits, or of the subnormals' 2^-9; two roundings of the quotient
    assert (np.abs(e4m3_decode(codes) * s - y) <= np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20)).all()


def test_linear_by_loops():
    rng = np.random.default_rng(2)
    m, n, k = 3, 130, 140
    xq, wq = (e4m3_encode_sat(rng.standard_normal((r, k)) * 30) for r in (m, n))
    sx, sw = rng.random((m, 2)), rng.random((2, 2))
    bias = rng.standard_normal(n)
    a, size = block.linear(xq, sx, wq, sw, bias)
    for i, j in ((0, 0), (2, 127), (1, 128), (2, 129)):
        t = [e4m3_decode(xq[i, c]) * e4m3_decode(wq[j, c]) * sx[i, c // 128] * sw[j // 128, c // 128] for c in range(k)]
        assert np.isclose(a[i, j], sum(t) + bias[j]) and np.isclose(size[i, j], sum(map(abs, t)) + abs(bias[j]))


def test_linear_with_equal_scales_is_the_per_tensor_one():
    rng = np.random.default_rng(3)
    xq, wq = (e4m3_encode_sat(rng.standard_normal((r, 256)) * 30) for r in (5, 16))
    a, _ = block.linear(xq, np.full((5, 2), 0.25), wq, np.full((1, 2), 0.5))
    assert np.allclose(a, ops.linear_dequant(e4m3_decode(xq), 0.25, e4m3_decode(wq), np.full(16, 0.5)))


def test_norm_terms():
    rng = np.random.default_rng(4)
    x, res = rng.standard_normal((2, 64)), rng.standard_normal((2, 64))
    r, y, size = block.norm(x, res, 0.0, ada_scale=np.full(64, -1.0), ada_shift=np.full(64, 3.0))
    assert (y == 3).all() and (size == 3).all()
    r, y, size = block.norm(x, res, 0.0)
    assert np.allclose((y * y).mean(1), 1) and (size == np.abs(y)).all()
