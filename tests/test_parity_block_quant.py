"""The writers of block-scaled E4M3 codes against the oracle: the quantiser bit for
bit; the norm and the gated activation within the roundings of their float32 steps.

How far codes and scales may be off, given |y - y_ref| <= err element by element
(y the kernel's float32 value): a block's largest |y| is then off by at most its
largest err, and the scale by that over 448 and two roundings; code * scale is off
from y by half a step of E4M3 (2^-4 of the value, or half of the subnormals' 2^-9
times the scale), the roundings of 1 / scale and of the quotient adding 2^-22.
"""
import numpy as np
import pytest
import torch

from oracle import block, ops
from oracle.formats import bf16_decode, bf16_encode, e4m3_decode
from parity import from_bits, to_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # float32's unit roundoff


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    return g


def bits(rng, *shape, std=1.0):
    return bf16_encode(rng.standard_normal(shape) * std)


class Guarded:
    """An output with a border of a known byte before and behind it."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.raw[256:256 + n].view(dtype).view(*shape)

    def check(self):
        assert (self.raw[:256] == 0xA5).all() and (self.raw[-256:] == 0xA5).all(), "written outside"


def check_codes(codes, scales, y, err, block_rows=1):
    rows, d = y.shape
    worst = block.amax(err, block_rows)
    ref = np.maximum(block.amax(np.abs(y), block_rows) / 448, 2.0 ** -100)
    assert (np.abs(scales - ref) <= worst / 448 + 4 * U * ref).all(), "scales"
    s = block.spread(scales.astype(np.float64), rows, d, block_rows)
    off = np.abs(e4m3_decode(codes) * s - y)
    size = np.abs(y) + err
    room = err + np.maximum(size * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20) + size * 2.0 ** -20
    bad = off > room
    assert not bad.any(), f"{bad.sum()} codes, first at {np.argwhere(bad)[0]}: off {off[bad][0]:.3e}, room {room[bad][0]:.3e}"


# ------------------------------------------------------------- the quantiser

def run_quantize(gbf, x, block_rows=1, stream=None):
    rows, d = x.shape
    q = Guarded((rows, d), torch.uint8)
    s = Guarded((-(-rows // block_rows), block.block_count(d)), torch.float32)
    gbf.quantize_fp8_block(from_bits(x), q.t, s.t, block_rows=block_rows, stream=stream)
    torch.cuda.synchronize()
    q.check()
    s.check()
    return q.t.cpu().numpy(), s.t.cpu().numpy()


def same_bits(got, ref):
    assert np.array_equal(got[0], ref[0]), f"{(got[0] != ref[0]).sum()} codes"
    assert np.array_equal(got[1].view(np.uint32)[~np.isnan(ref[1])], ref[1].view(np.uint32)[~np.isnan(ref[1])])
    assert np.array_equal(np.isnan(got[1]), np.isnan(ref[1]))


@pytest.mark.parametrize("rows,d", [(1, 16), (1, 128), (3, 112), (7, 144), (5, 1040), (130, 256), (257, 2736), (1, 32768),
                                    (4099, 48), (64, 11008)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_bits(gbf, rows, d, block_rows):
    rng = np.random.default_rng(rows * 7 + d)
    x = bf16_encode(rng.standard_normal((rows, d)) * np.exp2(rng.integers(-20, 20, (rows, 1))))
    same_bits(run_quantize(gbf, x, block_rows), block.quantize(bf16_decode(x), block_rows))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_every_bf16(gbf, block_rows):
    """All 65,536 patterns, in blocks of one sign and exponent (NaN and infinity apart, and among finite ones)."""
    x = np.arange(65536, dtype=np.uint16).reshape(512, 128)
    same_bits(run_quantize(gbf, x, block_rows), block.quantize(bf16_decode(x), block_rows))
    mixed = np.ascontiguousarray(x.T).reshape(512, 128)
    same_bits(run_quantize(gbf, mixed, block_rows), block.quantize(bf16_decode(mixed), block_rows))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(gbf, block_rows):
    x = bits(np.random.default_rng(5), 300, 400)
    for i, v in enumerate((np.inf, -np.inf, np.nan, 0.0)):
        x[i, 130 + i] = bf16_encode(v)
    x[140, :] = 0
    x[150:, 128:256] = 0x8000                   # -0
    x[200, 399] = 0xFFC0                        # a NaN with its sign set
    x[210, 5] = 0x0001                          # the smallest subnormal alone
    x[210, :5] = x[210, 6:128] = 0
    same_bits(run_quantize(gbf, x, block_rows), block.quantize(bf16_decode(x), block_rows))


def test_quantize_rows_past_a_grid_stride(gbf):
    """More blocks than one pass of the grid takes, a width that no stride divides."""
    x = bits(np.random.default_rng(6), 20011, 400)
    same_bits(run_quantize(gbf, x), block.quantize(bf16_decode(x)))


# --------------------------------------------------------------- gated activation

ACTS = {"gelu_tanh": 1, "gelu_erf": 2, "silu": 3}


def gated_ref(x, d, act):
    """y and how far float32 may be from it: the exponential's 2 + 1.2 |z| ulp (CUDA's bound
    for the fast form) and the roundings of z, or erfcf's 4 ulp and its argument's rounding,
    which the function amplifies by at most g^2; products, sum and quotient add a few ulp."""
    v = bf16_decode(x)
    g, up = v[:, :d], v[:, d:]
    y = ops.gated_activation(g, up, ACTS[act])
    if act == "gelu_erf":
        ulps = 10 + g * g
    else:
        z = np.abs(g) if act == "silu" else 2 * 0.7978845608 * np.abs(g + 0.044715 * g ** 3)
        ulps = 10 + 4 * z
    return y, np.abs(y) * ulps * 2 * U + np.abs(up) * 2.0 ** -125


def run_gated(gbf, x, act):
    rows, d = x.shape[0], x.shape[1] // 2
    q, s = Guarded((rows, d), torch.uint8), Guarded((rows, block.block_count(d)), torch.float32)
    gbf.gated_act_fp8_block(from_bits(x), q.t, s.t, act=ACTS[act])
    torch.cuda.synchronize()
    q.check()
    s.check()
    return q.t.cpu().numpy(), s.t.cpu().numpy()


@pytest.mark.parametrize("rows,d", [(1, 16), (2, 128), (3, 240), (33, 1040), (32, 11008), (1000, 144)])
@pytest.mark.parametrize("act", list(ACTS))
def test_gated_parity(gbf, rows, d, act):
    x = bits(np.random.default_rng(rows + d), rows, 2 * d, std=2.0)
    codes, scales = run_gated(gbf, x, act)
    check_codes(codes, scales, *gated_ref(x, d, act))


@pytest.mark.parametrize("act", list(ACTS))
def test_gated_tails(gbf, act):
    """Whole blocks of strongly negative gates, where act(gate) is small but not zero, beside zeros and large ones."""
    rng = np.random.default_rng(9)
    x = bits(rng, 6, 512, std=1.0)
    for r, lo in enumerate((-2.0, -4.0, -5.0, 3.0, 20.0)):
        x[r, :256] = bf16_encode(lo + 0.5 * rng.random(256))
    x[5, :256] = 0
    codes, scales = run_gated(gbf, x, act)
    check_codes(codes, scales, *gated_ref(x, 256, act))
    assert (scales[5] == np.float32(2.0 ** -100)).all() and not (codes[5] & 0x7F).any()


@pytest.mark.parametrize("act", list(ACTS))
def test_gated_special_values(gbf, act):
    x = bits(np.random.default_rng(10), 4, 512)
    x[0, 3] = bf16_encode(np.nan)
    x[1, 130] = bf16_encode(np.inf)
    x[1, 256 + 130] = bf16_encode(1.0)
    x[2, 256 + 7] = bf16_encode(np.nan)
    x[3, 5] = bf16_encode(-np.inf)               # infinity times the activation's 0
    codes, scales = run_gated(gbf, x, act)
    for row in (0, 2, 3):
        assert np.isnan(scales[row, 0]) and (codes[row, :128] == 0x7F).all() and np.isfinite(scales[row, 1])
    assert scales[1, 1] == np.inf and codes[1, 130] == 0x7F
    assert not (np.delete(codes[1, 128:], 2) & 0x7F).any() and np.isfinite(scales[1, 0])


# ------------------------------------------------------------------- the norm

def norm_case(rows, hidden, mode, gated, seed):
    rng = np.random.default_rng(seed)
    c = dict(x=bits(rng, rows, hidden), res=bits(rng, rows, hidden, std=2.0))
    c["x"][:, ::97] = bf16_encode(bf16_decode(c["x"][:, ::97]) * 20)        # outlier columns
    if mode == 0:
        c["weight"] = bf16_encode(1 + 0.1 * rng.standard_normal(hidden))
    if mode == 2:
        c["ada_scale"], c["ada_shift"] = bits(rng, hidden, std=0.2), bits(rng, hidden, std=0.2)
    if gated:
        c["gate"] = bits(rng, hidden, std=0.2)
    return c


def run_norm(gbf, c, mode, eps=1e-6, in_place=False):
    rows, hidden = c["x"].shape
    q, s = Guarded((rows, hidden), torch.uint8), Guarded((rows, block.block_count(hidden)), torch.float32)
    res = from_bits(c["res"])
    out = Guarded((rows, hidden), torch.bfloat16)
    if in_place:
        out.t.copy_(res)
        res = out.t
    extra = {k: from_bits(c[k]) for k in ("weight", "gate", "ada_scale", "ada_shift") if k in c}
    gbf.add_rmsnorm_fp8_block(from_bits(c["x"]), res, out.t, q.t, s.t, mode, eps=eps, **extra)
    torch.cuda.synchronize()
    for g in (q, s, out):
        g.check()
    return to_bits(out.t), q.t.cpu().numpy(), s.t.cpu().numpy()


def check_norm(got, c, eps=1e-6):
    extra = {k: bf16_decode(c[k]) for k in ("weight", "gate", "ada_scale", "ada_shift") if k in c}
    r, y, size = block.norm(bf16_decode(c["x"]), bf16_decode(c["res"]), eps, **extra)
    out, codes, scales = got
    assert np.array_equal(out, bf16_encode(r))
    # the mean square: at most 64 additions in a thread, 16 over warps and 5 in a shuffle, halved by the
    # square root; its quotient, root and reciprocal, and three steps from the value to y
    check_codes(codes, scales, y, size * (0.5 * 85 + 10) * U)


# every width class: under one block, one, a cut last block, one warp a row, several, two and four blocks a lane group
WIDTHS = [16, 64, 128, 144, 512, 656, 1024, 1040, 2736, 4096, 4112, 8192, 12288, 16384, 16400, 32768]


@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("mode,gated", [(0, False), (1, True), (2, False), (2, True)])
def test_norm_parity(gbf, hidden, mode, gated):
    c = norm_case(5, hidden, mode, gated, hidden + mode)
    check_norm(run_norm(gbf, c, mode), c)


@pytest.mark.parametrize("rows", [1, 2, 31, 777, 3001])
@pytest.mark.parametrize("hidden", [64, 400, 1024, 4096])
def test_norm_rows(gbf, rows, hidden):
    """One row, rows that share a warp or a CTA with none, more rows than the grid holds."""
    c = norm_case(rows, hidden, 0, True, rows)
    check_norm(run_norm(gbf, c, 0, in_place=rows % 2 == 1), c)


def test_norm_special_rows(gbf):
    c = norm_case(6, 400, 2, False, 3)
    c["x"][1], c["res"][1] = 0, 0                                # a row of zeros: y is the shift alone
    c["x"][2, 7] = bf16_encode(np.nan)
    c["res"][3, 9] = bf16_encode(np.inf)
    c["res"][4], c["x"][4] = c["x"][4], c["x"][4] ^ 0x8000       # cancels
    out, codes, scales = run_norm(gbf, c, 2)
    ok = [0, 1, 4, 5]
    check_norm((out[ok], codes[ok], scales[ok]), {k: v[ok] if v.ndim == 2 else v for k, v in c.items()})
    assert np.isnan(scales[2]).all() and (codes[2] == 0x7F).all()
    # an infinity makes the row's factor 0: its own block is NaN (inf * 0), the others hold the shift
    assert np.isnan(scales[3, 0]) and (codes[3, :128] == 0x7F).all() and np.isfinite(scales[3, 1:]).all()


def test_norm_zero_rows_have_the_least_scale(gbf):
    c = norm_case(3, 256, 1, False, 4)
    c["x"][:], c["res"][:] = 0, 0
    _, codes, scales = run_norm(gbf, c, 1)
    assert (scales == np.float32(2.0 ** -100)).all() and not codes.any()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_inputs_on_sixteen_bytes_only(gbf, block_rows):
    """A tensor that begins 16 bytes into a 32-byte line is read as well."""
    rng = np.random.default_rng(11)
    x = bits(rng, 37, 272)
    for act in (None, *ACTS):
        d = 272 if act is None else 136 - 8
        v = x if act is None else np.ascontiguousarray(x[:, :2 * d])
        raw = torch.empty(v.size + 8, dtype=torch.bfloat16, device="cuda")
        t = raw[8:].view(*v.shape)
        t.copy_(from_bits(v))
        assert t.data_ptr() % 32 == 16
        br = block_rows if act is None else 1
        q = torch.empty(37, d, dtype=torch.uint8, device="cuda")
        s = torch.empty(-(-37 // br), block.block_count(d), device="cuda")
        if act is None:
            gbf.quantize_fp8_block(t, q, s, block_rows=br)
            same_bits((q.cpu().numpy(), s.cpu().numpy()), block.quantize(bf16_decode(v), br))
        else:
            gbf.gated_act_fp8_block(t, q, s, act=ACTS[act])
            check_codes(q.cpu().numpy(), s.cpu().numpy(), *gated_ref(v, d, act))


def test_offsets_past_32_bits(gbf):
    """The last rows of tensors of more than 2^31 elements."""
    rows, d = (1 << 31) // 8192 + 300, 8192
    rng = np.random.default_rng(12)
    last = {k: bits(rng, 3, d) for k in ("x", "res")}
    x, res = (torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-3:], res[-3:] = from_bits(last["x"]), from_bits(last["res"])
    q = torch.empty(rows, d, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, d // 128, device="cuda")
    gbf.quantize_fp8_block(x, q, s)
    same_bits((q[-3:].cpu().numpy(), s[-3:].cpu().numpy()), block.quantize(bf16_decode(last["x"])))
    tiles = torch.empty(-(-rows // 128), d // 128, device="cuda")
    gbf.quantize_fp8_block(x, q, tiles, block_rows=128)
    tail = np.zeros((rows % 128, d), np.uint16)
    tail[-3:] = last["x"]
    ref = block.quantize(bf16_decode(tail), 128)
    same_bits((q[-3:].cpu().numpy(), tiles[-1:].cpu().numpy()), (ref[0][-3:], ref[1]))
    gbf.add_rmsnorm_fp8_block(x, res, res, q, s, gbf.NORM_NOWEIGHT)
    check_norm((to_bits(res[-3:]), q[-3:].cpu().numpy(), s[-3:].cpu().numpy()), last)
    gbf.gated_act_fp8_block(x.view(rows // 2, 2 * d), q[:rows // 2], s[:rows // 2], act=ACTS["silu"])
    v = np.zeros((1, 2 * d), np.uint16)
    v[0, :d], v[0, d:] = last["x"][1], last["x"][2]
    check_codes(q[rows // 2 - 1:rows // 2].cpu().numpy(), s[rows // 2 - 1:rows // 2].cpu().numpy(), *gated_ref(v, d, "silu"))


def test_streams_and_graph(gbf):
    """Captured on another stream and replayed on new inputs; two calls at once on two streams."""
    a, b = (norm_case(64, 1040, 0, False, s) for s in (1, 2))
    x, res, w = (from_bits(a[k]) for k in ("x", "res", "weight"))
    mk = lambda: (torch.empty_like(x), torch.empty(64, 1040, dtype=torch.uint8, device="cuda"),      # noqa: E731
                  torch.empty(64, 9, device="cuda"))
    out, q, s = mk()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gbf.add_rmsnorm_fp8_block(x, res, out, q, s, 0, weight=w)
    x.copy_(from_bits(b["x"]))
    res.copy_(from_bits(b["res"]))
    w.copy_(from_bits(b["weight"]))
    g.replay()
    torch.cuda.synchronize()
    check_norm((to_bits(out), q.cpu().numpy(), s.cpu().numpy()), b)
    outs, streams = [mk(), mk()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (o, cq, cs), st in zip(outs, streams):
        gbf.add_rmsnorm_fp8_block(x, res, o, cq, cs, 0, weight=w, stream=st)
    torch.cuda.synchronize()
    for o, cq, cs in outs:
        assert torch.equal(o, out) and torch.equal(cq, q) and torch.equal(cs, s)
