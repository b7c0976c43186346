"""gbfb_linear_fp8 against the float64 oracle.

Room: a is the sum of K terms in float32 (a block's on the tensor core, then one
product and one addition a block): each of the K / 32 + K / 128 additions and the
scale's product may lose 2^-23 of the sum of the terms' magnitudes (twice the
rounding to nearest, in case the tensor core cuts off).  The activations' slope
is below 1.13; the hardware tanh is off by 2^-10.9, so the tanh GELU by
|a| 2^-11.9, and the other forms by 2^-20 of |a|.  Then one bf16 rounding.
"""
import threading

import numpy as np
import pytest
import torch

from oracle import block, ops
from oracle.formats import bf16_decode, bf16_encode, e4m3_encode_sat
from parity import from_bits, to_bits
from test_parity_block_quant import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    return g


def case(m, n, k, seed, bias=True):
    """Codes over the whole E4M3 range, scales over four orders of magnitude, some of them zero or negative."""
    rng = np.random.default_rng(seed)
    kb = block.block_count(k)
    scales = lambda r: (np.exp(rng.uniform(-5, 4, (r, kb))) * rng.choice([1, 1, 1, -1], (r, kb))).astype(np.float32)  # noqa: E731
    c = dict(xq=e4m3_encode_sat(rng.standard_normal((m, k)) * 60), x_scales=scales(m),
             wq=e4m3_encode_sat(rng.standard_normal((n, k)) * 60), w_scales=scales(block.block_count(n)) * np.float32(1e-4),
             bias=bf16_encode(rng.standard_normal(n)) if bias else None)
    c["x_scales"][0, -1] = 0
    return c


def tensors(c):
    t = {k: torch.from_numpy(np.ascontiguousarray(c[k])).cuda() for k in ("xq", "x_scales", "wq", "w_scales")}
    return dict(t, bias=None if c["bias"] is None else from_bits(c["bias"]))


def run(gbf, c, act=0, stream=None):
    y = Guarded((c["xq"].shape[0], c["wq"].shape[0]), torch.bfloat16)
    gbf.linear_fp8_block(**tensors(c), y=y.t, act=act, stream=stream)
    torch.cuda.synchronize()
    y.check()
    assert gbf.device_status()[0] == 0
    return bf16_decode(to_bits(y.t))


def check(got, c, act=0):
    k = c["xq"].shape[1]
    a, size = block.linear(c["xq"], c["x_scales"], c["wq"], c["w_scales"], None if c["bias"] is None else bf16_decode(c["bias"]))
    ref = ops.activation(a, act) if act else a
    room = 1.13 * size * (k / 32 + 2 * k / 128 + 4) * 2.0 ** -23
    room += np.abs(a) * (2.0 ** -11.9 if act == 1 else 2.0 ** -20 if act else 0)
    room += (np.abs(ref) + room) * 2.0 ** -8 + 2.0 ** -133
    off = np.abs(got - ref)
    bad = off > room
    assert not bad.any(), (f"{bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {ref[bad][0]}, "
                           f"room {room[bad][0]:.3e}")


# rows: every tile width and its edges; N: one block, cut ones, several; K: under one block, cut, many
@pytest.mark.parametrize("m", [1, 15, 16, 17, 32, 33, 64, 65, 128, 129, 200, 257, 511])
@pytest.mark.parametrize("n,k", [(8, 16), (128, 128), (136, 144), (384, 1040)])
def test_small(gbf, m, n, k):
    c = case(m, n, k, m + n, bias=m % 2 == 0)
    check(run(gbf, c), c)


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("m", [3, 50, 130, 300])
def test_activations(gbf, act, m):
    c = case(m, 264, 512, act, bias=True)
    c["w_scales"] *= np.float32(0.01)          # sums of a few units, where the activations bend
    check(run(gbf, c, act), c, act)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (32, 1024, 16384), (7, 256, 32768), (96, 2048, 1536),
                                   (333, 1000, 2736), (640, 2304, 1024), (1030, 520, 656), (2048, 4104, 256),
                                   (1024, 8192, 2304), (1040, 8200, 4224), (768, 12288, 2048)])
def test_sizes(gbf, m, n, k):
    """K cut over clusters, long and short K, more tiles than the GPU holds at once (with one, two and three
    fillings of the scales' place to a tile, so that a tile's bias has to outlast them)."""
    c = case(m, n, k, m + n + k)
    check(run(gbf, c), c)


@pytest.mark.parametrize("m", [4, 40, 100, 300, 700])
def test_special_values(gbf, m):
    """NaN codes and scales reach their own row or columns alone; a scale of infinity gives one."""
    c = case(m, 256, 384, 7, bias=False)
    clean = run(gbf, c)
    c["xq"][1, 5] = 0x7F
    c["x_scales"][2, 1] = np.nan
    c["wq"][9, 300] = 0xFF
    got = run(gbf, c)
    assert np.isnan(got[1:3]).all() and np.isnan(got[:, 9]).all()
    keep = np.ones(got.shape, bool)
    keep[1:3] = keep[:, 9] = False
    assert np.array_equal(got[keep], clean[keep])
    c = case(m, 256, 384, 7, bias=False)
    c["x_scales"][3, 0] = np.inf
    got = run(gbf, c)
    assert not np.isfinite(got[3]).any() and np.array_equal(got[:3], clean[:3])


@pytest.mark.parametrize("m", [5, 24, 80, 400, 600])
def test_same_bits_again_and_in_another_batch(gbf, m):
    """A row's bits do not depend on the call before it, nor on what the other rows hold."""
    c = case(m, 640, 2048, 11)
    first = run(gbf, c)
    assert np.array_equal(first, run(gbf, c))
    other = case(m, 640, 2048, 12)
    mixed = dict(c, xq=other["xq"].copy(), x_scales=other["x_scales"].copy())
    mixed["xq"][m // 2], mixed["x_scales"][m // 2] = c["xq"][m // 2], c["x_scales"][m // 2]
    assert np.array_equal(run(gbf, mixed)[m // 2], first[m // 2])


@pytest.mark.parametrize("m", [8, 48, 320])
def test_streams_and_graph(gbf, m):
    c, d = case(m, 512, 1024, 1), case(m, 512, 1024, 2)
    t, y = tensors(c), torch.empty(m, 512, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gbf.linear_fp8_block(**t, y=y, act=0)
    for name, v in tensors(d).items():
        t[name].copy_(v)
    g.replay()
    torch.cuda.synchronize()
    check(bf16_decode(to_bits(y)), d)
    outs, streams = [torch.empty_like(y) for _ in range(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, st in zip(outs, streams):
            gbf.linear_fp8_block(**t, y=o, act=0, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, y)
    assert gbf.device_status()[0] == 0


def test_calls_of_all_widths_at_once(gbf):
    """Two threads with two streams each, every kernel and cluster size among them and the static
    Linears between: tensor memory and shared memory are shared, the results are those of calls alone."""
    sizes = [(8, 512, 4096), (16, 4096, 1024), (30, 1024, 2048), (32, 8192, 512), (60, 1024, 4096), (120, 512, 2048),
             (300, 1024, 4096), (700, 2048, 1024)]
    cases = [(tensors(case(m, n, k, 20 + i)), torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))
             for i, (m, n, k) in enumerate(sizes)]

    def block_call(i, y, stream=None):
        gbf.linear_fp8_block(**cases[i][0], y=y, act=2, stream=stream)

    def static_call(i, y, stream=None):
        t = cases[i][0]
        gbf.linear_fp8_act(t["xq"], 1e-3, t["wq"], ones[:y.shape[1]], t["bias"], y, act=0, stream=stream)

    ones = torch.ones(8192, device="cuda")
    calls = [(f, i) for i in range(len(sizes)) for f in (block_call, static_call)]
    alone = [torch.empty_like(cases[i][1]) for _, i in calls]
    for (f, i), y in zip(calls, alone):
        f(i, y)
    torch.cuda.synchronize()
    wrong = []

    def worker(seed):
        try:
            streams = [torch.cuda.Stream(), torch.cuda.Stream()]
            ys = [[torch.zeros_like(y) for y in alone] for _ in streams]
            torch.cuda.synchronize()
            rng = np.random.default_rng(seed)
            for _ in range(10):
                for st, out in zip(streams, ys):
                    for j in rng.permutation(len(calls)):
                        f, i = calls[j]
                        f(i, out[j], st)
            for st in streams:
                st.synchronize()
            wrong.extend((seed, calls[j][0].__name__, sizes[calls[j][1]]) for out in ys for j in range(len(calls))
                         if not torch.equal(out[j], alone[j]))
        except Exception as e:  # noqa: BLE001 - the main thread reports it
            wrong.append((seed, repr(e)))

    threads = [threading.Thread(target=worker, args=(s,)) for s in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert gbf.device_status()[0] == 0


def test_leading_dimensions_and_empty_batch(gbf):
    c = case(12, 256, 256, 3)
    t, y = tensors(c), torch.empty(3, 4, 256, dtype=torch.bfloat16, device="cuda")
    gbf.linear_fp8_block(t["xq"].view(3, 4, 256), t["x_scales"].view(3, 4, 2), t["wq"], t["w_scales"], t["bias"], y, act=0)
    check(bf16_decode(to_bits(y)).reshape(12, 256), c)
    e = torch.empty(0, 256, dtype=torch.uint8, device="cuda")
    gbf.linear_fp8_block(e, torch.empty(0, 2, device="cuda"), t["wq"], t["w_scales"], t["bias"],
                         torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), act=0)


@pytest.mark.parametrize("m,n,k", [((1 << 31) // 8192 + 300, 8192, 128), ((1 << 31) // 4096 + 300, 16, 4096)])
def test_offsets_past_32_bits(gbf, m, n, k):
    """The last rows of outputs, or inputs, of more than 2^31 elements."""
    c = case(3, n, k, 5)
    c["x_scales"][0, -1] = 1
    t = tensors(c)
    xq = torch.zeros(m, k, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(m, block.block_count(k), device="cuda")
    xq[-3:], xs[-3:] = t["xq"], t["x_scales"]
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gbf.linear_fp8_block(xq, xs, t["wq"], t["w_scales"], t["bias"], y, act=0)
    torch.cuda.synchronize()
    check(bf16_decode(to_bits(y[-3:])), c)
    assert torch.equal(y[0], t["bias"]) and torch.equal(y[m // 2], t["bias"])
