"""gbfb_linear_fp8 where CTA pairs take the call, K whole and cut in two, three and four,
against the float64 oracle.  What a size launches is asked of the library, so that a
size that goes elsewhere fails and does not pass for it.  The room is
test_parity_block_linear's."""
import threading

import numpy as np
import pytest
import torch

from oracle.formats import bf16_decode, bf16_encode
from parity import from_bits, to_bits
from test_parity_block_linear import case, check, run, tensors
from test_parity_block_quant import bits, check_codes, check_norm, gated_ref

pytestmark = pytest.mark.gpu

SPLITS = [1, 2, 3, 4]


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    return g


def pair_sizes(gbf, split, odd=False):
    """Sizes that pairs take with K cut in `split`; odd: rows, channels and K that fill no tile or block."""
    even = [(1024, 4096, 4096), (333, 4096, 11008), (256, 5120, 8192), (256, 4608, 8192), (256, 4096, 14336),
            (256, 3584, 14336), (256, 2560, 14336)]
    cut = [(m, n, k) for n in (4104, 5000, 3592, 3080) for m in (1030, 300, 511, 201) for k in (2736, 8176, 10992, 14352, 16400)]
    found = [s for s in (cut if odd else even) if gbf.linear_fp8_block_plan(*s) == (256, split)]
    assert found, f"no size here is taken by pairs with K cut in {split}"
    return found[0]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("split", SPLITS)
def test_sizes(gbf, split, odd):
    m, n, k = pair_sizes(gbf, split, odd)
    c = case(m, n, k, m + n + k)
    check(run(gbf, c), c)


@pytest.mark.parametrize("act", [1, 2, 3])
@pytest.mark.parametrize("split", SPLITS)
def test_activations(gbf, split, act):
    m, n, k = pair_sizes(gbf, split, odd=act == 2)
    c = case(m, n, k, act, bias=True)
    c["w_scales"] *= np.float32(0.01 * (512 / k) ** 0.5)   # sums of a few units, where the activations bend
    check(run(gbf, c, act), c, act)


@pytest.mark.parametrize("act", [0, 1, 2, 3])
def test_more_tiles_than_the_gpu_holds(gbf, act):
    """A CTA's second and third tile, each with its own bias, in columns of tiles that are walked together."""
    m, n, k = (1500, 8200, 784) if act % 2 else (2048, 9000, 2304)
    assert gbf.linear_fp8_block_plan(m, n, k)[0] == 256
    c = case(m, n, k, 30 + act)
    c["w_scales"] *= np.float32(0.01)
    check(run(gbf, c, act), c, act)


@pytest.mark.parametrize("split", SPLITS)
def test_special_values(gbf, split):
    """NaN codes and scales reach their own row or columns alone; a scale of infinity gives one."""
    m, n, k = pair_sizes(gbf, split, odd=True)
    c = case(m, n, k, 7, bias=False)
    clean = run(gbf, c)
    c["xq"][1, 5] = 0x7F
    c["xq"][130, k - 1] = 0x7F
    c["x_scales"][m - 1, 1] = np.nan
    c["wq"][9, 300] = 0xFF
    c["wq"][n - 3, k - 1] = 0xFF
    c["w_scales"][3, -1] = np.nan                          # channels 384 to 511
    got = run(gbf, c)
    rows, cols = [1, 130, m - 1], [9, n - 3, *range(384, 512)]
    assert np.isnan(got[rows]).all() and np.isnan(got[:, cols]).all()
    keep = np.ones(got.shape, bool)
    keep[rows] = keep[:, cols] = False
    assert np.array_equal(got[keep], clean[keep])
    c = case(m, n, k, 7, bias=False)
    c["x_scales"][3, -1] = np.inf
    got = run(gbf, c)
    assert not np.isfinite(got[3]).any() and np.array_equal(np.delete(got, 3, 0), np.delete(clean, 3, 0))


@pytest.mark.parametrize("split", SPLITS)
def test_same_bits_again_and_in_another_batch(gbf, split):
    """A row's bits depend neither on the call before it, nor on its place among the calls, nor on
    what the other rows hold."""
    m, n, k = pair_sizes(gbf, split, odd=True)
    c = case(m, n, k, 11)
    first = run(gbf, c)
    t, ys = tensors(c), [torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(40)]
    for y in ys:
        gbf.linear_fp8_block(**t, y=y, act=0)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_decode(to_bits(ys[0])), first)
    assert all(torch.equal(y, ys[0]) for y in ys)
    other = case(m, n, k, 12)
    mixed = dict(c, xq=other["xq"].copy(), x_scales=other["x_scales"].copy())
    for row in (m // 2, m - 1):
        mixed["xq"][row], mixed["x_scales"][row] = c["xq"][row], c["x_scales"][row]
    got = run(gbf, mixed)
    assert np.array_equal(got[[m // 2, m - 1]], first[[m // 2, m - 1]])


@pytest.mark.parametrize("split", SPLITS)
def test_streams_and_graph(gbf, split):
    m, n, k = pair_sizes(gbf, split)
    c, d = case(m, n, k, 1), case(m, n, k, 2)
    t, y = tensors(c), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
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
    assert all(torch.equal(o, y) for o in outs)
    assert gbf.device_status()[0] == 0


def test_calls_of_all_kernels_at_once(gbf):
    """Two threads with two streams each, pairs with every cut of K and single CTAs with every tile among
    them and the static Linears between: the results are those of calls alone."""
    sizes = [pair_sizes(gbf, s) for s in SPLITS] + [(8, 512, 4096), (30, 4096, 2048), (60, 1024, 4096), (512, 4096, 1024)]
    plans = [gbf.linear_fp8_block_plan(*s) for s in sizes]
    assert plans[:4] == [(256, s) for s in SPLITS] and {p[0] for p in plans[4:]} == {16, 32, 64, 128}, plans
    cases = [tensors(case(m, n, k, 20 + i)) for i, (m, n, k) in enumerate(sizes)]
    ones = torch.ones(16384, device="cuda")

    def block_call(i, y, stream=None):
        gbf.linear_fp8_block(**cases[i], y=y, act=2, stream=stream)

    def static_call(i, y, stream=None):
        t = cases[i]
        gbf.linear_fp8_act(t["xq"], 1e-3, t["wq"], ones[:y.shape[1]], t["bias"], y, act=0, stream=stream)

    calls = [(f, i) for i in range(len(sizes)) for f in (block_call, static_call)]
    alone = [torch.empty(sizes[i][0], sizes[i][1], dtype=torch.bfloat16, device="cuda") for _, i in calls]
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


def test_a_prompts_feed_forward(gbf):
    """Norm, up projection, gated activation and down projection of a thousand tokens, where pairs take the up
    projection: eager, each call against the oracle on what it was given, and as a graph on other tokens."""
    t, h, ffn = 1000, 2048, 4096
    assert gbf.linear_fp8_block_plan(t, 2 * ffn, h)[0] == 256
    rng = np.random.default_rng(4)
    dev = lambda dtype, *s: torch.zeros(*s, dtype=dtype, device="cuda")                  # noqa: E731
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    weights = {}
    for name, (n, k) in dict(up=(2 * ffn, h), down=(h, ffn)).items():
        weights[name] = dev(u8, n, k), dev(f32, n // 128, k // 128)
        gbf.quantize_fp8_block(from_bits(bits(rng, n, k, std=k ** -0.5)), *weights[name], block_rows=128)
    w = from_bits(bf16_encode(1 + 0.1 * rng.standard_normal(h)))
    x, res, res_out = dev(bf, t, h), dev(bf, t, h), dev(bf, t, h)
    c1, c2 = (dev(u8, t, h), dev(f32, t, h // 128)), (dev(u8, t, ffn), dev(f32, t, ffn // 128))
    up, y = dev(bf, t, 2 * ffn), dev(bf, t, h)

    def step():
        gbf.add_rmsnorm_fp8_block(x, res, res_out, *c1, gbf.NORM_WEIGHT, weight=w)
        gbf.linear_fp8_block(*c1, *weights["up"], None, up, act=gbf.ACT_NONE)
        gbf.gated_act_fp8_block(up, *c2, act=gbf.ACT_SILU)
        gbf.linear_fp8_block(*c2, *weights["down"], None, y, act=gbf.ACT_NONE)

    def fill(seed):
        r = np.random.default_rng(seed)
        x.copy_(from_bits(bits(r, t, h)))
        res.copy_(from_bits(bits(r, t, h, std=2.0)))

    n = lambda v: v.cpu().numpy()                                                        # noqa: E731
    lin = lambda c, name, out: check(bf16_decode(to_bits(out)), dict(                    # noqa: E731
        xq=n(c[0]), x_scales=n(c[1]), wq=n(weights[name][0]), w_scales=n(weights[name][1]), bias=None))
    fill(1)
    step()
    torch.cuda.synchronize()
    check_norm((to_bits(res_out), n(c1[0]), n(c1[1])), dict(x=to_bits(x), res=to_bits(res), weight=to_bits(w)))
    lin(c1, "up", up)
    check_codes(n(c2[0]), n(c2[1]), *gated_ref(to_bits(up), ffn, "silu"))
    lin(c2, "down", y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (2, 3):
        fill(seed)
        step()
        torch.cuda.synchronize()
        eager = [v.clone() for v in (res_out, *c1, up, *c2, y)]
        for v in (res_out, *c1, up, *c2, y):
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, (res_out, *c1, up, *c2, y)))
    assert gbf.device_status()[0] == 0
