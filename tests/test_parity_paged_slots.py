"""gbfd_paged_slots against the oracle's request-by-request allocation: every
output equal, entries it has no business with unchanged."""
import numpy as np
import pytest
import torch

from oracle import decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    assert g.device_status()[0] == g.OK
    return g


def case(rng, batch, block, longest, prompts=0, ended=0, spare=5, head=None, extra_width=2):
    """A pool in use: scattered blocks in the table, the rest free in a ring that has gone round."""
    ctx = rng.integers(0, longest + 1, batch)
    new = np.where(rng.random(batch) < 0.1, 0, 1)
    who = rng.permutation(batch)
    new[who[:prompts]] = rng.integers(1, 3 * longest + 2, min(prompts, batch))
    new[who[prompts:prompts + ended]] = -1 - rng.integers(0, 3, len(who[prompts:prompts + ended]))
    have = -(-ctx // block)
    need = -(-(ctx + np.maximum(new, 0)) // block) - have
    blocks = max(1, int(have.sum() + need.sum()) + spare)
    order = rng.permutation(blocks)
    width = int((-(-(ctx + np.maximum(new, 0)) // block)).max()) + extra_width
    table = np.full((batch, width), -3, np.int32)
    at = 0
    for b in range(batch):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    head = int(rng.integers(0, blocks)) if head is None else head
    free = np.full(blocks, -4, np.int32)
    free[(head + np.arange(blocks - at)) % blocks] = order[at:]
    return dict(ctx=ctx.astype(np.int32), new=new.astype(np.int32), table=table, free=free,
                ring=np.array([head, blocks - at], np.int32), block=block,
                tokens=int(np.maximum(new, 0).sum()))


def run(gbf, c, pad=3, in_place=False, start=True, apart=0, tokens=None):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()      # noqa: E731
    n, batch = (c["tokens"] if tokens is None else tokens) + pad, c["ctx"].size
    wide = torch.full((batch, c["table"].shape[1] + apart), -8, dtype=torch.int32, device="cuda")
    table = wide[:, apart // 2:apart // 2 + c["table"].shape[1]]
    table.copy_(d(c["table"]))
    ctx, new, free, ring = d(c["ctx"]), d(c["new"]), d(c["free"]), d(c["ring"])
    full = lambda m: torch.full((m,), -9, dtype=torch.int32, device="cuda")           # noqa: E731
    seq, ring_out = (ctx, ring) if in_place else (full(batch), full(2))
    slots, pos, st = full(n), full(n), full(batch + 1) if start else None
    gbf.paged_slots(ctx, new, table, free, ring, c["block"], seq, ring_out, slots, pos, st)
    torch.cuda.synchronize()
    out = dict(table=table, free=free, ring=ring_out, seq=seq, slots=slots, pos=pos, start=st, wide=wide)
    return {k: None if v is None else v.cpu().numpy() for k, v in out.items()}


def check(c, got, pad=3, apart=0):
    p, seq, slots, pos, start, refused = decode.paged_slots(c["ctx"], c["new"], c["table"], c["free"], c["ring"],
                                                            c["block"])
    assert np.array_equal(got["table"], p.table)
    assert np.array_equal(got["free"], p.free_ring) and got["ring"].tolist() == [p.head, p.count]
    assert np.array_equal(got["seq"], seq)
    n = got["slots"].size - pad
    assert np.array_equal(got["slots"][:n], slots[:n]) and np.array_equal(got["pos"][:n], pos[:n])
    assert (got["slots"][n:] == -9).all() and (got["pos"][n:] == -9).all()
    if got["start"] is not None:
        assert np.array_equal(got["start"], start)
    if apart:
        assert (got["wide"][:, :apart // 2] == -8).all() and (got["wide"][:, apart // 2 + c["table"].shape[1]:] == -8).all()
    return refused


@pytest.mark.parametrize("block", [1, 7, 16, 64])
@pytest.mark.parametrize("batch,longest,prompts,ended", [(1, 0, 1, 0), (1, 100, 0, 1), (5, 40, 2, 1), (33, 300, 5, 4),
                                                         (257, 90, 40, 30), (1500, 60, 20, 100), (8192, 20, 10, 50)])
def test_steps(gbf, block, batch, longest, prompts, ended):
    c = case(np.random.default_rng(batch + block), batch, block, longest, prompts, ended)
    check(c, run(gbf, c))
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("tokens_each", [3, 3000])
def test_in_place_and_tables_apart(gbf, tokens_each):
    """seq_lens on ctx_lens and ring_out on ring, small (one CTA) and large (a cluster)."""
    rng = np.random.default_rng(tokens_each)
    c = case(rng, 40, 16, tokens_each, prompts=20, ended=5)
    check(c, run(gbf, c, in_place=True, apart=10), apart=10)
    check(c, run(gbf, c, start=False))


def test_a_repeated_call_writes_the_same(gbf):
    c = case(np.random.default_rng(1), 50, 16, 200, prompts=5, ended=5)
    first = run(gbf, c)
    again = run(gbf, {**c, "table": first["table"], "free": first["free"]})
    for k in ("table", "free", "ring", "seq", "slots", "pos", "start"):
        assert np.array_equal(first[k], again[k]), k


@pytest.mark.parametrize("prompts", [0, 12])
def test_pool_runs_out(gbf, prompts):
    """The requests behind the last free block are refused, the others served."""
    rng = np.random.default_rng(2 + prompts)
    c = case(rng, 60, 4, 50, prompts=prompts, ended=6, spare=0)
    short = max(1, int(c["ring"][1]) // 2)
    keep = int(c["ring"][1]) - short
    gone = (c["ring"][0] + np.arange(keep, c["ring"][1])) % c["free"].size
    c["free"][gone] = -4
    c["ring"][1] = keep
    got = run(gbf, c)
    refused = check(c, got)
    assert refused.any() and not refused.all()
    s, msg = gbf.device_status()
    assert s == gbf.EDEVICE and "pool" in msg
    # no block is in two places
    served = got["seq"]
    used = np.concatenate([got["table"][b, :-(-served[b] // 4)] for b in range(60)])
    assert np.unique(used).size == used.size


def test_rows_too_short_and_bad_lengths(gbf):
    c = case(np.random.default_rng(3), 20, 16, 200, prompts=3, extra_width=0)
    c["new"][4] = 10 ** 6
    c["tokens"] = int(np.maximum(c["new"], 0).sum())
    got = run(gbf, c)
    assert check(c, got)[4]
    assert gbf.device_status()[0] == gbf.EDEVICE
    c = case(np.random.default_rng(4), 20, 16, 200)
    c["ctx"][7] = -1
    assert check(c, run(gbf, c))[7]
    assert gbf.device_status()[0] == gbf.EDEVICE


def test_more_tokens_than_rows(gbf):
    c = case(np.random.default_rng(5), 20, 16, 100, prompts=4)
    got = run(gbf, c, pad=0, tokens=c["tokens"] - 7)
    check(c, got, pad=0)
    assert gbf.device_status()[0] == gbf.EDEVICE


def test_bad_ids_and_ring_states(gbf):
    c = case(np.random.default_rng(6), 8, 16, 200, head=3)
    c["ctx"][:], c["new"][:] = 20, 1
    c = {**c, "ctx": np.full(8, 20, np.int32), "new": np.ones(8, np.int32), "tokens": 8}
    c["table"][:, 1] = np.arange(8)
    c["table"][2, 1] = 1 << 20
    got = run(gbf, c)
    assert got["slots"][2] == -1 and (got["slots"][[0, 1, 3, 4, 5, 6, 7]] >= 0).all()
    assert gbf.device_status()[0] == gbf.EDEVICE
    for ring in ([-1, 2], [c["free"].size, 2], [0, -2], [0, c["free"].size + 1]):
        run(gbf, {**c, "ring": np.array(ring, np.int32)})
        s, msg = gbf.device_status()
        assert s == gbf.EDEVICE and "pool" in msg


def test_graph_follows_the_lengths(gbf):
    """A captured step, replayed three times in place, walks the requests on."""
    rng = np.random.default_rng(8)
    c = case(rng, 10, 4, 30, spare=200, extra_width=20)
    c["new"][:] = 1
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()      # noqa: E731
    ctx, new, table, free, ring = (d(c[k]) for k in ("ctx", "new", "table", "free", "ring"))
    slots, pos = (torch.zeros(10, dtype=torch.int32, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gbf.paged_slots(ctx, new, table, free, ring, 4, ctx, ring, slots, pos)
    want = dict(c)
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        p, seq, s, q, _, _ = decode.paged_slots(want["ctx"], want["new"], want["table"], want["free"], want["ring"], 4)
        assert np.array_equal(slots.cpu().numpy(), s) and np.array_equal(pos.cpu().numpy(), q)
        want = {**want, "ctx": seq, "table": p.table, "free": p.free_ring, "ring": [p.head, p.count]}
    assert np.array_equal(ctx.cpu().numpy(), want["ctx"]) and ring.cpu().numpy().tolist() == want["ring"]
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,prompts,ended", [(512, 0, 3), (513, 0, 3), (900, 2, 20), (2040, 0, 0), (2300, 1, 60)])
def test_large_batches_of_decode_rows(gbf, batch, prompts, ended, in_place):
    """Batches scanned by 256 and by 1024 threads, with up to two tokens for each thread and with more."""
    c = case(np.random.default_rng(batch), batch, 16, 40, prompts, ended)
    check(c, run(gbf, c, in_place=in_place))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens", [3, 3000])
@pytest.mark.parametrize("batch", [5, 700])
def test_a_length_that_fills_the_sums(gbf, batch, tokens, in_place):
    """A request whose new length is 2^31 - 1 is refused; the ones behind it take their block and their length all the
    same, although their packed tokens lie past the end."""
    c = case(np.random.default_rng(batch), batch, 4, 40, ended=1, spare=2 * batch)
    c["ctx"][1:4], c["new"][0:4] = [0, 4, 6], [1, 2 ** 31 - 1, 1, 1]
    c["table"][2, 0], c["table"][3, :2] = c["free"][c["ring"][0]], c["free"][c["ring"][0]]     # (any block)
    got = run(gbf, c, tokens=tokens, pad=0, in_place=in_place)
    # (a new length that only just does not fit is refused alike, and can be counted out one by one)
    room = c["table"].shape[1] * 4
    p, seq, slots, pos, _, refused = decode.paged_slots(c["ctx"], np.where(c["new"] > room, room + 1, c["new"]), c["table"],
                                                        c["free"], c["ring"], 4)
    assert refused[1] and not refused[2] and not refused[3] and seq[2] == 5 and seq[3] == 7
    assert np.array_equal(got["seq"], seq) and np.array_equal(got["table"], p.table)
    assert np.array_equal(got["free"], p.free_ring) and got["ring"].tolist() == [p.head, p.count]
    assert got["slots"][0] == slots[0] and (got["slots"][1:] == -1).all()
    assert np.array_equal(got["pos"], np.concatenate([pos[:1], np.arange(tokens - 1)]))
    assert got["start"][:2].tolist() == [0, 1] and (got["start"][3:] == 2 ** 31 - 1).all()
    assert gbf.device_status()[0] == gbf.EDEVICE


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("prompts", [0, 20])
@pytest.mark.parametrize("state", ["head -1", "head n", "count -2", "count n + 1", "too many"])
def test_a_bad_ring_stays_as_it_is(gbf, state, prompts, in_place):
    """Nothing is taken from it or given back to it: the free ids are all there, ended requests keep their blocks and
    lengths, and a later call reports it again.  So too where more would go back than there are blocks."""
    c = case(np.random.default_rng(9), 40, 16, 200, prompts=prompts, ended=5)
    n = c["free"].size
    c["ring"][:] = {"head -1": [-1, 2], "head n": [n, 2], "count -2": [0, -2], "count n + 1": [0, n + 1],
                    "too many": [3, n]}[state]
    c["free"][:] = np.arange(n)
    ended = c["new"] < 0
    assert (c["ctx"][ended] > 0).any()
    for _ in range(2):
        got = run(gbf, c, in_place=in_place)
        refused = check(c, got)
        assert refused[ended & (c["ctx"] > 0)].all() and np.array_equal(got["free"], c["free"])
        assert np.array_equal(got["seq"][ended], c["ctx"][ended])
        if state != "too many":
            assert got["ring"].tolist() == c["ring"].tolist()
        s, msg = gbf.device_status()
        assert s == gbf.EDEVICE and "pool" in msg
        c = {**c, "ring": got["ring"].copy() if state != "too many" else c["ring"]}


@pytest.mark.parametrize("in_place", [False, True])
def test_a_cached_length_out_of_range_is_clamped(gbf, in_place):
    """Below 0 it counts as 0, above its table row as all of the row; the request is refused, ended or not."""
    c = case(np.random.default_rng(10), 12, 16, 100)
    room = c["table"].shape[1] * 16
    c["ctx"][[1, 4, 7, 9]], c["new"][[1, 4, 7, 9]] = [-1, -2 ** 31, room + 1, 2 ** 31 - 1], [1, -1, -1, 2]
    c["tokens"] = int(np.maximum(c["new"], 0).sum())
    got = run(gbf, c, in_place=in_place)
    assert check(c, got)[[1, 4, 7, 9]].all()
    assert got["seq"][[1, 4, 7, 9]].tolist() == [0, 0, room, room]
    s, msg = gbf.device_status()
    assert s == gbf.EDEVICE and "length" in msg


@pytest.mark.parametrize("prompts", [0, 20])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_a_bad_id_that_goes_back(gbf, bad, in_place, prompts):
    """An ended request's bad id is reported and keeps its place in the ring; the request that takes it gets slot -1 for
    its tokens there, reported again, and everyone else their blocks."""
    c = case(np.random.default_rng(12), 30, 16, 100, prompts=prompts, ended=1, spare=0)
    b = int(np.flatnonzero(c["new"] < 0)[0])
    if c["ctx"][b] == 0:
        c["ctx"][b] = 5
    c["table"][b, 0] = bad
    got = run(gbf, c, in_place=in_place)
    check(c, got)
    s, msg = gbf.device_status()
    assert s == gbf.EDEVICE and "block id" in msg
    head, count = got["ring"]
    assert count == -(-int(c["ctx"][b]) // 16) and got["free"][head] == bad          # all others are taken
    new = np.zeros(30, np.int32)
    new[b] = 16 * count
    again = {**c, "ctx": got["seq"], "new": new, "table": got["table"], "free": got["free"], "ring": got["ring"],
             "tokens": int(new.sum())}
    out = run(gbf, again, in_place=in_place)
    assert gbf.device_status()[0] == gbf.EDEVICE
    assert (out["slots"][:16] == -1).all() and (out["slots"][16:again["tokens"]] >= 0).all()
    ids = got["free"][(head + 1 + np.arange(count - 1)) % got["free"].size]
    assert np.array_equal(out["slots"][16:again["tokens"]], (ids[:, None] * 16 + np.arange(16)).ravel())
    assert np.array_equal(out["seq"], got["seq"] + new) and out["ring"][1] == 0


@pytest.mark.parametrize("more", [3, 1000])
def test_rows_for_two_to_the_31_tokens(gbf, more):
    """The longest slots and pos there may be (8.6 GB each), few of their entries used: the rest keep their values."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    slots, pos = (torch.full((2 ** 31 - 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    c = case(np.random.default_rng(more), 40, 16, 100)
    c["new"][3] = more
    c["table"] = np.pad(c["table"], ((0, 0), (0, 80)), constant_values=-3)
    c["free"] = np.pad(c["free"], (0, 100), constant_values=-4)
    held = np.unique(c["table"][c["table"] >= 0])
    spare = np.setdiff1d(np.arange(c["free"].size), held).astype(np.int32)
    c["free"][:spare.size], c["ring"][:] = spare, [0, spare.size]
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()      # noqa: E731
    table, seq, ring_out = d(c["table"]), d(np.zeros_like(c["ctx"])), d(np.zeros_like(c["ring"]))
    gbf.paged_slots(d(c["ctx"]), d(c["new"]), table, d(c["free"]), d(c["ring"]), 16, seq, ring_out, slots, pos)
    torch.cuda.synchronize()
    p, want, s, q, _, refused = decode.paged_slots(c["ctx"], c["new"], c["table"], c["free"], c["ring"], 16)
    assert not refused.any() and np.array_equal(seq.cpu().numpy(), want) and np.array_equal(table.cpu().numpy(), p.table)
    assert np.array_equal(slots[:s.size].cpu().numpy(), s) and np.array_equal(pos[:s.size].cpu().numpy(), q)
    assert bool((slots[s.size:s.size + 4096] == -9).all()) and bool((slots[-4096:] == -9).all())
    assert bool((pos[s.size:s.size + 4096] == -9).all()) and bool((pos[-4096:] == -9).all())
    assert gbf.device_status()[0] == gbf.OK


@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_at_the_end_of_int32(gbf, in_place):
    """Blocks so large that a table row has room for more tokens than a length can say."""
    top = 2 ** 31 - 1
    c = dict(ctx=np.array([top, top - 1, top - 5, 0, top], np.int32), new=np.array([1, 1, 6, 2, -1], np.int32),
             table=np.zeros((5, 3), np.int32), free=np.zeros(1, np.int32), ring=np.array([0, 1], np.int32), block=1 << 30,
             tokens=10)
    got = run(gbf, c, in_place=in_place)
    refused = check(c, got)
    assert refused.tolist() == [True, False, True, False, True] and got["seq"].tolist() == [top, top, top - 5, 2, top]
    assert gbf.device_status()[0] == gbf.EDEVICE
