"""gbfd_sample_tokens against the float64 oracle: the same token, always, and
its log-probability.

The kernel's weights are within 2^-37 of their value or half a unit of 2^-43 of
the largest, and its sums are exact, so a running mass is within
d = 2^-37 + vocab 2^-44 / total of itself (total: the kept mass, the largest weight
as 1): a row whose smallest margin (distance of a running mass from a bound it is
compared with) is below 4 d may fall either way and is left out.  A bound that
is uniform over the mass comes that near one of vocab sums with a chance of
8 d vocab at most, below 1 in 100 for 151936 and total >= 4; one row in eight may be.
logprob = (l - top) / T - ln(mass): two float32 terms, each off by at most a few
half steps 2^-24 of its size."""
import numpy as np
import pytest
import torch

from oracle import decode, formats
from parity import from_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    assert g.device_status()[0] == g.OK
    return g


def logits(rng, batch, vocab, f32, std=2.5):
    l = (rng.standard_normal((batch, vocab)) * std).astype(np.float32)
    strong = rng.integers(0, vocab, (batch, 8))
    np.put_along_axis(l, strong, (rng.random((batch, 8)) * 8 + 2).astype(np.float32), 1)
    if f32:
        return l
    return torch.from_numpy(l).to(torch.bfloat16).float().numpy()


def run(gbf, l, u, f32, temperature=None, top_k=None, top_p=None, min_p=None, stride=None, logprob=True):
    batch, vocab = l.shape
    t = torch.from_numpy(np.ascontiguousarray(l, np.float32)).cuda()
    t = t if f32 else t.to(torch.bfloat16)
    if stride:
        wide = torch.full((batch, stride), float("inf"), dtype=t.dtype, device="cuda")    # beside the rows: never read as theirs
        wide[:, :vocab] = t
        t = wide[:, :vocab]
    f = lambda a, ty: None if a is None else torch.from_numpy(np.asarray(a, ty)).cuda()            # noqa: E731
    tokens = torch.full((batch,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((batch,), 9.0, device="cuda") if logprob else None
    gbf.sample_tokens(t, f(u, np.float32), tokens, temperature=f(temperature, np.float32), top_k=f(top_k, np.int32),
                      top_p=f(top_p, np.float32), min_p=f(min_p, np.float32), logprob=lp)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), None if lp is None else lp.cpu().numpy()


def check(l, u, got, temperature=None, top_k=None, top_p=None, min_p=None, skip=0):
    tokens, lps = got
    batch, vocab = l.shape
    at = lambda a, b, other, ty: other if a is None else ty(np.asarray(a, ty)[b])                 # noqa: E731
    skipped = 0
    for b in range(batch):
        t = at(temperature, b, 1.0, np.float32)
        token, lp, margin, total = decode.sample_row(l[b], np.float32(u[b]), float(t), int(at(top_k, b, 0, np.int32)),
                                                     float(at(top_p, b, 1.0, np.float32)),
                                                     float(at(min_p, b, 0.0, np.float32)))
        near = 4 * (2.0 ** -37 + vocab * 2.0 ** -44 / max(total, 1.0))
        if margin < near:
            skipped += 1
            continue
        assert tokens[b] == token, f"row {b}: {tokens[b]}, the oracle says {token} (margin {margin:.1e})"
        if lps is not None:
            if np.isnan(lp):
                assert np.isnan(lps[b])
            else:
                assert abs(lps[b] - lp) <= 8 * 2.0 ** -24 * (abs(lp) + 1e-3) + near, (b, lps[b], lp)
    assert skipped <= max(skip, batch // 8), f"{skipped} rows with margins too small to compare"


def params(rng, batch):
    kind = np.arange(batch) % 8
    return dict(temperature=np.where(kind == 1, 0, 0.4 + rng.random(batch)).astype(np.float32),
                top_k=np.where((kind >= 2) & (kind <= 4), rng.integers(1, 100, batch), 0).astype(np.int32),
                top_p=np.where((kind == 3) | (kind == 5) | (kind == 7), 0.3 + 0.69 * rng.random(batch), 1).astype(np.float32),
                min_p=np.where((kind == 4) | (kind == 6) | (kind == 7), 0.3 * rng.random(batch), 0).astype(np.float32))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("batch,vocab", [(1, 1), (3, 2), (9, 7), (16, 8), (16, 63), (24, 1000), (40, 4099), (16, 32000),
                                         (16, 50257), (16, 151936)])
def test_mixed_parameters(gbf, batch, vocab, f32):
    rng = np.random.default_rng(batch * vocab + f32)
    l, u, p = logits(rng, batch, vocab, f32), rng.random(batch).astype(np.float32), params(rng, batch)
    check(l, u, run(gbf, l, u, f32, **p), **p)


@pytest.mark.parametrize("f32", [False, True])
def test_defaults_and_no_logprob(gbf, f32):
    rng = np.random.default_rng(5)
    l, u = logits(rng, 12, 5001, f32), rng.random(12).astype(np.float32)
    check(l, u, run(gbf, l, u, f32))
    check(l, u, run(gbf, l, u, f32, logprob=False))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("vocab,stride", [(1000, 1001), (1001, 1003), (1001, 4096), (17, 18)])
def test_row_strides(gbf, vocab, stride, f32):
    """Rows that begin at any element offset; what lies between them is +inf."""
    rng = np.random.default_rng(stride)
    l, u, p = logits(rng, 19, vocab, f32), rng.random(19).astype(np.float32), params(rng, 19)
    check(l, u, run(gbf, l, u, f32, stride=stride, **p), **p)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["equal", "two", "few", "ramp"])
def test_ties(gbf, kind, f32):
    """Logits with very few values: the borders of top-k and top-p fall inside runs
    of thousands of equals and are drawn by index."""
    rng = np.random.default_rng(11)
    batch, vocab = 16, 20011
    l = {"equal": np.full((batch, vocab), 1.5), "two": rng.integers(0, 2, (batch, vocab)) * 3.0,
         "few": rng.integers(0, 5, (batch, vocab)) * 0.5, "ramp": np.tile(np.arange(vocab) // 64 / 64.0, (batch, 1))}[kind]
    l = l.astype(np.float32)
    if not f32:
        l = torch.from_numpy(l).to(torch.bfloat16).float().numpy()
    u = rng.random(batch).astype(np.float32)
    k = rng.integers(1, vocab, batch).astype(np.int32)
    p = (0.05 + 0.9 * rng.random(batch)).astype(np.float32)
    for q in (dict(top_k=k), dict(top_p=p), dict(top_k=k, top_p=p), dict(top_k=np.ones(batch)),
              dict(top_k=np.full(batch, vocab)), dict(top_k=np.full(batch, vocab - 1)), dict(min_p=np.ones(batch))):
        check(l, u, run(gbf, l, u, f32, **q), **q)


@pytest.mark.parametrize("f32", [False, True])
def test_masked_infinite_and_nan_logits(gbf, f32):
    rng = np.random.default_rng(12)
    l = logits(rng, 10, 3001, f32)
    l[0, 100:] = -np.inf
    l[1] = -np.inf
    l[1, 1234] = -50.0
    l[2] = -np.inf                         # nothing to draw
    l[3, ::3] = np.nan
    l[4] = np.nan
    l[5, [7, 2000, 2999]] = np.inf         # the only weights
    l[6] = np.finfo(np.float32).min if f32 else -3.3895313892515355e38
    l[7] = -np.inf
    l[7, -1] = 3.0
    l[8] = 0.0
    l[8, ::2] = -0.0                       # equal to +0
    u = rng.random(10).astype(np.float32)
    for q in (dict(), dict(top_k=np.full(10, 2)), dict(top_p=np.full(10, 0.7)), dict(min_p=np.full(10, 0.5)),
              dict(temperature=np.zeros(10)), dict(top_k=np.full(10, 500), top_p=np.full(10, 0.5))):
        got = run(gbf, l, u, f32, **q)
        check(l, u, got, **q)
        assert got[0][2] == -1 and got[0][4] == -1 and np.isnan(got[1][[2, 4]]).all()
        s, msg = gbf.device_status()
        assert s == gbf.EDEVICE and "candidate" in msg
    assert gbf.device_status()[0] == gbf.OK


def test_extreme_parameters(gbf):
    rng = np.random.default_rng(13)
    l, u = logits(rng, 8, 2000, True), np.array([0, 2.0 ** -30, 0.5, 1 - 2.0 ** -24, 0, 1 - 2.0 ** -24, 0.3, 0.6], np.float32)
    for q in (dict(temperature=np.full(8, 1e-30)), dict(temperature=np.full(8, 1e-45)), dict(temperature=np.full(8, 1e30)),
              dict(top_p=np.zeros(8)), dict(top_p=np.full(8, -1.0)), dict(top_p=np.full(8, 1e-30)),
              dict(top_p=np.full(8, 1 - 2.0 ** -24)), dict(top_k=np.full(8, -5)), dict(top_k=np.full(8, 2 ** 31 - 1)),
              dict(min_p=np.full(8, 1e-30)), dict(min_p=np.full(8, -1.0)), dict(top_p=np.full(8, np.inf))):
        check(l, u, run(gbf, l, u, True, **q), **q, skip=8 if "temperature" in q and q["temperature"][0] > 1 else 4)
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("scale,shift", [(1e30, 0.0), (1e9, 1e12), (1e-30, 0.0), (3e37, -3e38), (1e-3, 1e6), (1e-38, 0.0)])
def test_logits_of_any_size(gbf, scale, shift):
    """Logits whose differences are far larger or smaller than 1, or lost in their size."""
    rng = np.random.default_rng(17)
    with np.errstate(over="ignore"):                          # some become infinite
        l = (rng.standard_normal((8, 20000)) * scale + shift).astype(np.float32)
    l[3, 5:] = l[3, 4]
    u = rng.random(8).astype(np.float32)
    for t in (1.0, float(np.float32(min(scale, 1e20)))):
        t = np.full(8, max(t, 1e-29), np.float32)
        for q in (dict(), dict(top_p=np.full(8, 0.7)), dict(top_k=np.full(8, 40)), dict(min_p=np.full(8, 0.1))):
            check(l, u, run(gbf, l, u, True, temperature=t, **q), temperature=t, **q, skip=4)
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("f32,batch", [(True, 3), (False, 3), (True, 160), (False, 160)])
def test_long_runs_of_equals(gbf, f32, batch):
    """Tens of thousands of equal logits in one CTA's slice, one CTA or several per
    row: a bin overflows its counter, the lists overflow, the border is found by
    logit and index."""
    rng = np.random.default_rng(18)
    vocab = 70001
    row = np.full(vocab, 2.0, np.float32)
    row[::7] = 1.0
    row[::11] = -np.inf
    l, u = np.tile(row, (batch, 1)), rng.random(batch).astype(np.float32)
    k, p = rng.integers(1, vocab, batch), (0.05 + 0.9 * rng.random(batch)).astype(np.float32)
    some = np.r_[0:2, batch - 1]
    for q in (dict(top_k=k), dict(top_p=p), dict(top_k=k, top_p=p), dict()):
        tokens, lps = run(gbf, l, u, f32, **q)
        check(l[some], u[some], (tokens[some], lps[some]), **{n: v[some] for n, v in q.items()}, skip=3)


def test_parameters_out_of_range_are_reported(gbf):
    rng = np.random.default_rng(14)
    l, u = logits(rng, 4, 500, False), np.full(4, 0.5, np.float32)
    nan, inf = np.nan, np.inf
    for q in (dict(temperature=[-1.0, 1, 1, 1]), dict(temperature=[nan, 1, 1, 1]), dict(temperature=[inf, 1, 1, 1]),
              dict(top_p=[nan, 1, 1, 1]), dict(min_p=[nan, 0, 0, 0]), dict(min_p=[1.5, 0, 0, 0])):
        got = run(gbf, l, u, False, **q)
        assert got[0][0] == -1 and np.isnan(got[1][0])
        check(l, u, got, **q)
        assert gbf.device_status()[0] == gbf.EDEVICE
    for x in (1.0, -0.1, nan):
        u[1] = x
        got = run(gbf, l, u, False)
        assert got[0][1] == -1 and (got[0][[0, 2, 3]] >= 0).all()
        assert gbf.device_status()[0] == gbf.EDEVICE


def test_frequencies(gbf):
    """An even grid of uniforms draws each kept token in proportion to its weight."""
    rng = np.random.default_rng(15)
    n = 4096
    row = rng.standard_normal(300).astype(np.float32) * 2
    l = np.tile(row, (n, 1))
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tokens, _ = run(gbf, l, u, True, temperature=np.full(n, 0.8), top_k=np.full(n, 40))
    w = np.exp(row.astype(np.float64) / np.float32(0.8))
    w[np.argsort(-row, kind="stable")[40:]] = 0
    got = np.bincount(tokens, minlength=300)
    assert np.abs(got - n * w / w.sum()).max() <= 1.0 + 1e-3      # an interval of length x holds x n or one more or less


@pytest.mark.parametrize("f32,vocab", [(True, 262144), (False, 262147), (True, 1 << 20), (False, 1 << 20)])
def test_large_vocabularies(gbf, f32, vocab):
    """Up to the largest vocabulary: slices that do not fit in shared memory."""
    rng = np.random.default_rng(vocab)
    l, u, p = logits(rng, 8, vocab, f32), rng.random(8).astype(np.float32), params(rng, 8)
    check(l, u, run(gbf, l, u, f32, **p), **p)


def test_repeats_graph_and_streams(gbf):
    rng = np.random.default_rng(16)
    l = torch.from_numpy(logits(rng, 64, 30011, False)).cuda().bfloat16()
    u = torch.from_numpy(rng.random(64).astype(np.float32)).cuda()
    p = torch.full((64,), 0.9, device="cuda")
    outs = [torch.full((64,), -9, dtype=torch.int32, device="cuda") for _ in range(4)]
    gbf.sample_tokens(l, u, outs[0], top_p=p)
    torch.cuda.synchronize()
    for i in (1, 2):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(4):
                gbf.sample_tokens(l, u, outs[i], top_p=p)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gbf.sample_tokens(l, u, outs[3], top_p=p)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    u.copy_(torch.rand(64, device="cuda"))                    # new numbers: the graph reads them
    g.replay()
    gbf.sample_tokens(l, u, outs[0], top_p=p)
    torch.cuda.synchronize()
    assert torch.equal(outs[3], outs[0])


def test_min_p_of_one_keeps_the_largest_alone(gbf):
    """Logits one float32 step below the largest, hot enough that their weights round to the same float32 number."""
    rng = np.random.default_rng(12)
    batch, vocab = 4, 70000
    top = np.float32(10.0)
    l = np.full((batch, vocab), np.nextafter(top, np.float32(0)), np.float32)
    u = np.array([0.0, 0.25, 0.6, 1 - 2.0 ** -24], np.float32)
    tops = [np.sort(rng.choice(vocab, 1000, replace=False)) for _ in range(batch)]
    for b in range(batch):
        l[b, tops[b]] = top
    tokens, lps = run(gbf, l, u, True, temperature=np.full(batch, 100.0), min_p=np.ones(batch))
    want = [tops[b][int(np.float64(u[b]) * 1000)] for b in range(batch)]
    assert tokens.tolist() == want
    # log(1 / 1000): a float32 logarithm (2 ulp) of a sum that is right to 2^-23
    assert np.all(np.abs(lps + np.log(1000.0)) <= 3 * 2.0 ** -23 * np.log(1000.0))


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("batch,vocab", [(2, 60000), (30, 60001), (60, 50000), (160, 40000), (4, 300000)])
def test_borders_that_fall_on_an_element(gbf, batch, vocab, f32):
    """n equal logits and nothing else of weight: a top_p of 1 / 2 ends exactly at an element, and so does a u of 1 / 2
    or 0 (or a u with no top_p).  The float32 pass may not decide those; all sums are exact, and logprob = -log(kept)
    is a float32 logarithm (2 ulp) of a ratio that is right to half of one."""
    rng = np.random.default_rng(batch)
    counts = np.array([64, 4, 16, 2])[np.arange(batch) % 4]
    l = np.full((batch, vocab), -200.0, np.float32)
    at = [np.sort(rng.choice(vocab, n, replace=False)) for n in counts]
    for b in range(batch):
        l[b, at[b]] = 1.5
    u = np.where(np.arange(batch) % 3 == 0, 0.0, 0.5).astype(np.float32)
    for top_p in (np.full(batch, 0.5), np.where(np.arange(batch) % 2, 0.5, 0.25), None):
        tokens, lps = run(gbf, l, u, f32, top_p=top_p)
        kept = counts if top_p is None else (counts * np.maximum(top_p, 1.0 / counts)).astype(int)
        assert tokens.tolist() == [at[b][int(kept[b] * u[b])] for b in range(batch)]
        assert np.all(np.abs(lps + np.log(kept)) <= 3 * 2.0 ** -23 * np.log(kept))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("batch", [1, 5, 18, 40])
def test_short_rows_on_clusters(gbf, batch, f32):
    """Rows shorter than a vector per CTA, whose CTAs have next to nothing to do before they first write to one
    another, in long runs of calls behind one another and beside a kernel that keeps part of the SMs busy."""
    rng = np.random.default_rng(batch)
    busy = torch.zeros(64 << 20, device="cuda")
    other = torch.cuda.Stream()
    for vocab in (1, 2, 7, 9, 63):
        l, u = logits(rng, batch, vocab, f32), rng.random(batch).astype(np.float32)
        p = params(rng, batch)
        t = torch.from_numpy(l).cuda() if f32 else torch.from_numpy(l).to(torch.bfloat16).cuda()
        args = {k: torch.from_numpy(v).cuda() for k, v in p.items()}
        uniform = torch.from_numpy(u).cuda()
        tokens = torch.full((60, batch), -7, dtype=torch.int32, device="cuda")
        lp = torch.full((60, batch), 9.0, device="cuda")
        torch.cuda.synchronize()
        for i in range(60):
            if i % 10 == 0:
                with torch.cuda.stream(other):
                    busy.add_(1.0)
            gbf.sample_tokens(t, uniform, tokens[i], logprob=lp[i], **args)
        torch.cuda.synchronize()
        tokens, lp = tokens.cpu().numpy(), lp.cpu().numpy()
        check(l, u, (tokens[0], lp[0]), **p)
        assert (tokens == tokens[0]).all() and (lp.view(np.int32) == lp[0].view(np.int32)).all()
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("batch", [1, 20, 44, 120])
@pytest.mark.parametrize("k,vocab", [(3, 801), (75, 801), (300, 801), (700, 801), (900, 2001), (1500, 2001)])
def test_top_k_keeps_candidates_of_next_to_no_weight(gbf, k, vocab, batch, f32):
    """One strong candidate, the others 2^-32 of it and less, beyond the last bin with a lower end: top-k keeps as many
    of them as it says, and a uniform next to 1 draws one of them.  As many as fit one list, and more."""
    rng = np.random.default_rng(k + batch)
    l = -22.2 - 3.0 * rng.random((batch, vocab)) ** 2
    l[:, 0] = 0.0
    l = l.astype(np.float32) if f32 else torch.from_numpy(l).to(torch.bfloat16).float().numpy()
    u, top_k = np.full(batch, np.float32(1 - 2.0 ** -24)), np.full(batch, k, np.int32)
    u[::3] = 0.5
    kept = np.minimum(np.exp(np.sort(l.astype(np.float64), axis=1)[:, ::-1]), 1)[:, 1:k].sum(1)
    tokens, lp = run(gbf, l, u, f32, top_k=top_k)
    # the kept mass beside the first candidate's: weights to 2^-36 or half a unit of 2^-43, the logarithm to float32
    first = tokens == 0
    assert first[::3].all()
    assert (np.abs(lp + np.log1p(kept))[first] <= 2.0 ** -22 * kept[first] + k * 2.0 ** -44).all()
    behind = (1 - 2.0 ** -24) * (1 + kept) - 1             # how far u times the kept mass lies behind the first candidate's
    sure = (np.arange(batch) % 3 != 0) & (np.abs(behind) > 1e-9)
    assert np.array_equal(first[sure], behind[sure] < 0)
    rank = (l > np.take_along_axis(l, tokens[:, None], 1)).sum(1)
    assert (rank < k).all() and (k < 700 or not first[sure].any())
