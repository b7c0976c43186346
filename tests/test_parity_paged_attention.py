"""gbfd_paged_attention against the float64 oracle.

Bound per output, from the roundings the kernel makes (u = 2^-24, binary32 half
step; e = 2^-8, bf16 half step):
  * a score is a sum of head_dim exact products in binary32 and one product
    with the scale: |ds| <= (head_dim + 2) u reach, reach = scale sum|q k|; the
    exponent's argument is rounded too, by u (|s| + max|s|) log2(e) <= 3 u reach;
  * each weight takes two further relative errors of 2^-21 (the hardware
    exponential, documented at 2^-22 plus the rounding of its argument's
    difference) and 2^-16 (its bf16 pair), and sums of n weights
    n u each at worst: in all w = 2 ((head_dim + 5) u reach + 2^-16 + 2^-20 + n u)
    for numerator and denominator together;
  * the output is off by at most w sum|p v| before it is rounded to bf16 (half
    a step of 2^-8) or to E4M3 (2^-4, and half the smallest subnormal, 2^-10).
"""
import numpy as np
import pytest
import torch

from oracle import decode, formats
from parity import from_bits, to_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    assert g.device_status()[0] == g.OK
    return g


def bits(rng, *shape, std=1.0):
    t = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def case(lens, hq, hkv, d, block, seed=0, spare=2, width=None):
    """Scattered blocks; every cache row that no position refers to is NaN."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    have = -(-lens // block)
    blocks = int(have.sum()) + spare
    order = rng.permutation(blocks).astype(np.int32)
    width = max(1, int(have.max())) if width is None else width
    table = np.full((lens.size, width), -1, np.int32)
    rows, at = np.zeros(blocks * block, bool), 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
        j = np.arange(lens[b])
        rows[table[b, j // block] * block + j % block] = True
    k, v = bits(rng, blocks * block, hkv, d), bits(rng, blocks * block, hkv, d)
    k[~rows], v[~rows] = 0x7FC0, 0x7FC0
    return dict(q=bits(rng, lens.size, hq, d, std=1.5), k=k, v=v, table=table, lens=lens, block=block, hq=hq, hkv=hkv,
                d=d, scale=d ** -0.5)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def workspace(gbf, c):
    # what an earlier user left there must not matter
    return torch.full((gbf.paged_attention_workspace(c["hq"], c["hkv"], c["d"]),), 0xFF, dtype=torch.uint8,
                      device="cuda")


def run(gbf, c, window=0, out_scale=None, lse=True):
    q = from_bits(c["q"])
    out = torch.full(q.shape, 0x7F, dtype=torch.uint8, device="cuda") if out_scale else torch.full_like(q, float("nan"))
    l = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
    gbf.paged_attention(q, from_bits(c["k"]), from_bits(c["v"]), dev(c["table"]), dev(c["lens"]), c["block"], out,
                        workspace(gbf, c), window=window, lse=l, out_scale=out_scale)
    torch.cuda.synchronize()
    return to_bits(out), None if l is None else l.cpu().numpy()


def check(c, got, got_lse, window=0, out_scale=None, lens=None, table=None):
    k, v = (np.nan_to_num(formats.bf16_decode(c[n])) for n in "kv")
    out, lse, size, reach = decode.paged_attention(formats.bf16_decode(c["q"]), k, v,
                                                   c["table"] if table is None else table,
                                                   c["lens"] if lens is None else lens, c["block"], c["scale"], window)
    n = max(1, int(np.max(c["lens"])))
    w = 2 * ((c["d"] + 5) * U * reach + 2.0 ** -16 + 2.0 ** -20 + n * U)[..., None]
    if out_scale is None:
        y, tol = formats.bf16_decode(got), w * size + 2.0 ** -8 * (np.abs(out) + w * size)
        ref = out
    else:
        y, s = formats.e4m3_decode(got), float(np.float32(out_scale))
        ref = np.clip(out / s, -448, 448)
        tol = w * size / s * (1 + 2.0 ** -4) + 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2 * U * np.abs(ref)
    assert np.isfinite(y).all()
    bad = np.abs(y - ref) > tol
    assert not bad.any(), f"{bad.sum()} outputs off, worst {np.abs(y - ref)[bad].max():.3e} against {tol[bad].min():.3e}"
    if got_lse is not None:
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse))
        on = np.isfinite(lse)
        # the sum's relative error, the score's, the logarithm and the products with ln 2 (3 roundings of |lse| + reach)
        tol = (w[..., 0] + 6 * U * (np.abs(lse) + reach + 1))[on]
        assert (np.abs(got_lse[on] - lse[on]) <= tol).all()


RAGGED = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 5]


@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 176, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (5, 5), (12, 1), (24, 2)])
def test_heads_and_widths(gbf, d, hq, hkv):
    c = case(RAGGED, hq, hkv, d, 16, seed=d + hq)
    check(c, *run(gbf, c))


@pytest.mark.parametrize("block", [1, 3, 8, 16, 24, 64, 256])
def test_block_sizes(gbf, block):
    c = case(RAGGED, 8, 2, 128, block, seed=block)
    check(c, *run(gbf, c))


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 15, 16, 17, 33, 64])
def test_groups(gbf, group):
    c = case([3, 40, 0, 129], 2 * group, 2, 64, 16, seed=group)
    check(c, *run(gbf, c))


@pytest.mark.parametrize("lens", [[1], [0], [5000], [4097, 1, 1, 1], [0, 0, 2049, 0], [16] * 70, [1000] * 9])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 1, 256)])
def test_splits(gbf, lens, hq, hkv, d):
    """One request over the whole GPU, ranges that end on tile, head and request
    borders, empty requests at either end."""
    c = case(lens, hq, hkv, d, 16, seed=sum(lens))
    check(c, *run(gbf, c))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1000, 1 << 40])
def test_windows(gbf, window):
    c = case(RAGGED + [1500], 8, 4, 128, 16, seed=3)
    check(c, *run(gbf, c, window=window), window=window if window < 1 << 31 else 0)


@pytest.mark.parametrize("out_scale", [0.01, 1.0, 0.0005])
@pytest.mark.parametrize("d,hq", [(64, 8), (128, 32), (256, 8)])
def test_codes(gbf, out_scale, d, hq):
    c = case(RAGGED, hq, 2, d, 16, seed=d)
    check(c, *run(gbf, c, out_scale=out_scale, lse=False), out_scale=out_scale)


def test_table_column_range_and_wide_rows(gbf):
    """A column range of a wider table (rows apart), wider than any request."""
    c = case(RAGGED, 8, 2, 128, 16, seed=4, width=40)
    wide = torch.full((len(RAGGED), 64), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, 7:47] = dev(c["table"])
    q = from_bits(c["q"])
    out = torch.empty_like(q)
    gbf.paged_attention(q, from_bits(c["k"]), from_bits(c["v"]), wide[:, 7:47], dev(c["lens"]), 16, out,
                        workspace(gbf, c))
    torch.cuda.synchronize()
    check(c, to_bits(out), None)
    assert gbf.device_status()[0] == gbf.OK


def test_shared_blocks(gbf):
    """Requests with a common prefix point to the same blocks."""
    c = case([200, 200], 8, 2, 128, 16, seed=6)
    c["table"][1, :6] = c["table"][0, :6]
    check(c, *run(gbf, c))


def test_large_scores_and_shifts(gbf):
    """Scores of +-10^3 with the largest at either end: the running maximum moves
    in every tile or in none, and most weights underflow to zero."""
    for ascending in (True, False):
        c = case([300, 37], 8, 2, 64, 16, seed=7)
        k = formats.bf16_decode(c["k"])
        for b in range(2):
            j = np.arange(c["lens"][b])
            ramp = (j if ascending else j[::-1]) / 10.0
            k[c["table"][b, j // 16] * 16 + j % 16] = ramp[:, None, None]
        c["k"] = formats.bf16_encode(k)
        c["q"] = formats.bf16_encode(np.abs(formats.bf16_decode(c["q"])) * 8)
        check(c, *run(gbf, c))


def test_cache_beyond_32_bits(gbf):
    """A cache of more than 2^32 bytes and 2^31 elements per tensor, the request's
    blocks at its far end."""
    hq, hkv, d, block = 8, 8, 128, 16
    c = case([333, 1, 50], hq, hkv, d, block, seed=8, spare=0)
    blocks = (1 << 31) // (hkv * d * block) + 64
    kc = torch.empty(blocks * block, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    n = c["k"].shape[0]
    kc[-n:], vc[-n:] = from_bits(c["k"]), from_bits(c["v"])
    q = from_bits(c["q"])
    out = torch.empty_like(q)
    table = np.where(c["table"] >= 0, c["table"] + blocks - n // block, -1)
    gbf.paged_attention(q, kc, vc, dev(table), dev(c["lens"]), block, out, workspace(gbf, c))
    torch.cuda.synchronize()
    check(c, to_bits(out), None)


def test_bad_ids_and_lengths_are_reported_and_left_out(gbf):
    c = case([40, 64, 30], 8, 2, 128, 16, seed=9)
    good = c["table"].copy()
    c["table"][0, 1] = 1 << 20            # positions 16..31 of request 0
    c["table"][1, 3] = -5                 # positions 48..63 of request 1
    got, lse = run(gbf, c)
    s, msg = gbf.device_status()
    assert s == gbf.EDEVICE and "block id" in msg
    # what is left: request 0 keeps 0..15 and 32..39, request 1 keeps 0..47
    first = c.copy()
    first["lens"] = np.array([24, 48, 30], np.int32)
    first["table"] = good.copy()
    first["table"][0, 1] = good[0, 2]
    check(first, got, lse)
    c["table"] = good
    c["lens"] = np.array([-3, 9999, 30], np.int32)
    width = good.shape[1] * 16
    c["table"] = np.where(good < 0, good[1, 0], good).astype(np.int32)      # every entry of row 1 is a block: clamped
    c["k"], c["v"] = np.where(c["k"] == 0x7FC0, 0, c["k"]), np.where(c["v"] == 0x7FC0, 0, c["v"])
    got, lse = run(gbf, c)
    assert gbf.device_status()[0] == gbf.EDEVICE
    c["lens"] = np.array([0, width, 30], np.int32)
    check(c, got, lse)


def test_repeats_bit_for_bit_graph_and_streams(gbf):
    """The same bits from a second call, from a replayed graph, and from two calls
    at once on two streams with a workspace each."""
    c = case([3000, 0, 17, 900], 16, 2, 128, 16, seed=10)
    q, k, v, t, n = from_bits(c["q"]), from_bits(c["k"]), from_bits(c["v"]), dev(c["table"]), dev(c["lens"])
    outs = [torch.empty_like(q) for _ in range(4)]
    ws = [workspace(gbf, c) for _ in range(2)]
    gbf.paged_attention(q, k, v, t, n, 16, outs[0], ws[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                gbf.paged_attention(q, k, v, t, n, 16, outs[1 + i], ws[i])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gbf.paged_attention(q, k, v, t, n, 16, outs[3], ws[0])
        gbf.paged_attention(q, k, v, t, n, 16, outs[3], ws[0])
    outs[3].zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    # the lengths are read on the device: a replayed graph follows them
    short = np.array([100, 0, 3, 16], np.int32)
    n.copy_(dev(short))
    g.replay()
    torch.cuda.synchronize()
    check({**c, "lens": short}, to_bits(outs[3]), None)
    assert gbf.device_status()[0] == gbf.OK


def test_empty_batch(gbf):
    z = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(16, 2, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    gbf.paged_attention(z, kc, kc.clone(), i.view(0, 4), i, 16, torch.empty_like(z),
                        torch.empty(1 << 23, dtype=torch.uint8, device="cuda"))
    assert gbf.device_status()[0] == gbf.OK


# Which of the two splits a call takes depends on the block table's width and on how many items there are: the cases above
# have tables as narrow as their lengths; these have room for more tokens than clusters take, or more items.

WIDE = 600      # blocks of 16: 9600 tokens


@pytest.mark.parametrize("d", [16, 64, 80, 128, 176, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (5, 5), (12, 1), (24, 2)])
def test_wide_tables(gbf, d, hq, hkv):
    c = case(RAGGED, hq, hkv, d, 16, seed=d + hq, width=WIDE)
    check(c, *run(gbf, c))


@pytest.mark.parametrize("group", [1, 7, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("out_scale", [None, 0.01])
def test_wide_tables_groups_and_codes(gbf, group, out_scale):
    c = case([3, 40, 0, 129, 700], 2 * group, 2, 64, 16, seed=group, width=WIDE)
    check(c, *run(gbf, c, out_scale=out_scale), out_scale=out_scale)


@pytest.mark.parametrize("lens", [[1], [0], [5000], [4097, 1, 1, 1], [0, 0, 2049, 0], [16] * 70, [1000] * 9])
@pytest.mark.parametrize("window", [0, 4500])
def test_wide_tables_splits(gbf, lens, window):
    c = case(lens, 8, 2, 128, 16, seed=sum(lens), width=WIDE)
    check(c, *run(gbf, c, window=window), window=window)


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 2), (128, 24, 2), (256, 16, 2)])
@pytest.mark.parametrize("batch,longest", [(1, 50), (1, 300), (3, 4000), (8, 500), (16, 900), (30, 130), (60, 260), (150, 60),
                                           (170, 60), (200, 250), (300, 5)])
def test_few_items_by_their_number_and_length(gbf, d, hq, hkv, batch, longest):
    """Clusters of 1 to 8 CTAs, items of one warp each, and more items than find room as such."""
    rng = np.random.default_rng(batch * longest)
    lens = rng.integers(0, longest + 1, batch)
    lens[0] = longest
    c = case(lens, hq, hkv, d, 16, seed=batch)
    check(c, *run(gbf, c))


@pytest.mark.parametrize("width", [4, WIDE])
def test_bad_ids_and_lengths_in_either_split(gbf, width):
    """The GPU skips what it cannot look up, reports it, and the other requests come out as ever."""
    c = case([40, 33, 64, 20], 8, 2, 128, 16, seed=9, width=width)
    table, lens = c["table"].copy(), c["lens"].copy()
    bad = dict(c, table=table, lens=lens)
    bad["table"] = table.copy()
    bad["table"][1, 1] = 1 << 20                       # tokens 16..31 of request 1 lie nowhere
    bad["lens"] = lens.copy()
    bad["lens"][3] = -5                                # request 3 has no length
    out, lse = run(gbf, bad)
    s, msg = gbf.device_status()
    assert s == gbf.EDEVICE and "block id or length" in msg
    good, good_lse = run(gbf, c)
    assert gbf.device_status()[0] == gbf.OK
    for b in (0, 2):
        assert np.array_equal(out[b], good[b]) and np.array_equal(lse[b], good_lse[b])
    y = formats.bf16_decode(out)
    assert np.isfinite(y).all() and (y[3] == 0).all() and np.isneginf(lse[3]).all() and np.isfinite(lse[1]).all()


# A score that is not a number shows in its head's output however the call is split; scores of -inf alone are no tokens.

@pytest.mark.parametrize("lens,width", [([40, 5, 9], None), ([300, 900, 77], None), ([3000, 2500], None), ([60] * 200, None),
                                        ([40, 5, 200, 700, 5000], WIDE), ([5000], WIDE)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 24, 2), (256, 5, 1), (128, 40, 1)])
@pytest.mark.parametrize("out_scale", [None, 0.01])
def test_a_query_that_is_nan(gbf, lens, width, d, hq, hkv, out_scale):
    c = case(lens, hq, hkv, d, 16, seed=len(lens), width=width)
    good, good_lse = run(gbf, c, out_scale=out_scale)
    gone = np.zeros((len(lens), hq), bool)
    gone[::2, hq // 2], gone[-1, 0] = True, True
    q = c["q"].copy()
    q[gone, d // 3] = 0x7FC0
    out, lse = run(gbf, dict(c, q=q), out_scale=out_scale)
    assert (out[gone] & 0x7F == 0x7F).all() if out_scale else np.isnan(formats.bf16_decode(out[gone])).all()
    assert np.isnan(lse[gone]).all()
    assert np.array_equal(out[~gone], good[~gone]) and np.array_equal(lse[~gone], good_lse[~gone])
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("lens,width", [([40, 5, 9], None), ([300, 900, 77], None), ([60] * 200, None),
                                        ([40, 5, 200, 700, 5000], WIDE), ([5000, 3], WIDE)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 24, 2), (256, 5, 1)])
def test_keys_that_are_not_finite(gbf, lens, width, d, hq, hkv):
    c = case(lens, hq, hkv, d, 16, seed=len(lens), width=width)
    c["q"] &= 0x7FFF                                       # all above 0: a key of -inf gives a score of -inf
    good, good_lse = run(gbf, c)
    rows = lambda b, j: c["table"][b, j // 16] * 16 + j % 16                # noqa: E731
    k, group = c["k"].copy(), hq // hkv
    for b, n in enumerate(lens):
        k[rows(b, np.arange(n)), 0, 1] = 0xFF80            # -inf throughout, in KV head 0
    out, lse = run(gbf, dict(c, k=k))
    y = formats.bf16_decode(out)
    assert (y[:, :group] == 0).all() and np.isneginf(lse[:, :group]).all()
    assert np.array_equal(out[:, group:], good[:, group:]) and np.array_equal(lse[:, group:], good_lse[:, group:])
    k = c["k"].copy()
    for b, n in enumerate(lens):
        k[rows(b, np.array([n // 2])), hkv - 1, 1] = 0x7FC0                 # one NaN key, in the last KV head
    out, lse = run(gbf, dict(c, k=k))
    assert np.isnan(formats.bf16_decode(out[:, -group:])).all() and np.isnan(lse[:, -group:]).all()
    assert np.array_equal(out[:, :-group], good[:, :-group]) and np.array_equal(lse[:, :-group], good_lse[:, :-group])
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("batch,new", [(40, 1), (40, 150), (600, 3)])
def test_lengths_written_by_the_call_before(gbf, batch, new):
    """Step after step without a pause, lengths growing in place: the kernel, and the join behind it, see those of
    their own step, whatever an SM held of the last one."""
    steps, block = 12, 16
    c = case([steps * new + 40] * batch, 8, 2, 128, block, seed=batch, width=WIDE)
    start = torch.from_numpy(np.random.default_rng(new).integers(1, 40, batch).astype(np.int32)).cuda()
    q, k, v, table = from_bits(c["q"]), from_bits(c["k"]), from_bits(c["v"]), dev(c["table"])
    add = torch.full((batch,), new, dtype=torch.int32, device="cuda")
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")      # noqa: E731
    lens, slots, pos, ws = start.clone(), i32(batch * new), i32(batch * new), workspace(gbf, c)
    # the table has every block already: what paged_slots would enter goes to one of its own
    spare, free, ring = i32(batch, WIDE), torch.arange(40000, dtype=torch.int32, device="cuda"), dev(np.array([0, 40000], np.int32))
    outs = torch.zeros(steps, *q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(steps, *q.shape[:2], device="cuda")
    torch.cuda.synchronize()
    for i in range(steps):
        gbf.paged_slots(lens, add, spare, free, ring, block, lens, ring, slots, pos)
        gbf.paged_attention(q, k, v, table, lens, block, outs[i], ws, lse=lse[i])
    torch.cuda.synchronize()
    assert torch.equal(lens, start + steps * new)
    out, l = torch.empty_like(q), torch.empty_like(lse[0])
    for i in range(steps):
        at = start + (i + 1) * new
        torch.cuda.synchronize()
        gbf.paged_attention(q, k, v, table, at, block, out, ws, lse=l)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), outs[i].view(torch.int16)) and torch.equal(l, lse[i]), i
    assert gbf.device_status()[0] == gbf.OK
