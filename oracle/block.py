"""The block-scaled 8-bit operators: scales of 128 columns (or 128 x 128), and
the Linear on such codes.  Plain, in float64 but for the quantiser, whose steps
are binary32 by definition.  Values in, values out; codes are uint8.
"""
import numpy as np

from . import ops
from .formats import bf16_round, e4m3_decode, e4m3_encode_sat

BLOCK = 128
F32 = np.float32


def block_count(n):
    return -(-n // BLOCK)


def amax(y, block_rows=1):
    """The largest magnitude of each block [row blocks, column blocks]; NaN if it holds one."""
    y = np.abs(np.asarray(y))
    rows, d = y.shape
    out = np.zeros((-(-rows // block_rows), block_count(d)), y.dtype)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.max(y[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK])
    return out


def scales_of(largest):
    """scale = max(RN(amax * RN(1/448)), 2^-100), binary32."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.maximum(np.asarray(largest, F32) * (F32(1) / F32(448)), F32(2.0 ** -100))


def spread(scales, rows, d, block_rows=1):
    """Each element's scale [rows, d]."""
    return scales[np.arange(rows)[:, None] // block_rows, np.arange(d)[None, :] // BLOCK]


def quantize(y, block_rows=1):
    """(codes, scales) of binary32 y: code = e4m3(RN(y * RN(1 / scale)))."""
    y = np.asarray(y, F32)
    s = scales_of(amax(y, block_rows))
    with np.errstate(all="ignore"):
        codes = e4m3_encode_sat(y * (F32(1) / spread(s, *y.shape, block_rows)))
    return codes, s


def norm(x, res, eps, weight=None, gate=None, ada_scale=None, ada_shift=None):
    """(res_out, y, size) of the residual add and the norm in front of the quantiser, from
    values: y in float64, `size` the sum of the magnitudes of y's terms."""
    r = ops.residual_add(x, res) if gate is None else ops.gated_residual_add(x, res, gate)
    r = bf16_round(r)
    if ada_scale is not None:
        n = ops.rmsnorm(r, eps)
        y = ops.ada_modulate(n, ada_scale, ada_shift)
        return r, y, np.abs(n * (1 + ada_scale)) + np.abs(ada_shift)
    y = ops.rmsnorm(r, eps, weight) if weight is not None else ops.rmsnorm(r, eps)
    return r, y, np.abs(y)


def linear(xq, x_scales, wq, w_scales, bias=None):
    """(a, size): X W^T + bias of block-scaled codes, and the sum of its terms' magnitudes."""
    m, k = xq.shape
    n = wq.shape[0]
    x = e4m3_decode(xq) * spread(np.asarray(x_scales, np.float64), m, k)
    w = e4m3_decode(wq) * spread(np.asarray(w_scales, np.float64), n, k, BLOCK)
    b = 0.0 if bias is None else np.asarray(bias, np.float64)[None, :]
    return x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)
