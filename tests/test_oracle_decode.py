"""The decode oracle against closed forms, worked examples and brute force."""
import numpy as np

from oracle import decode


def test_slots_worked_example():
    """Blocks of 4.  Request 0: 3 cached in block 7, two more tokens -> one new
    block for position 4.  Request 1 ends and gives back 5 and 2.  Request 2 is a
    prompt of 5: two blocks."""
    table = np.array([[7, -1], [5, 2], [-1, -1]])
    p, seq, slots, pos, start, refused = decode.paged_slots([3, 6, 0], [2, -1, 5], table, [9, 0, 0, 0, 0, 1, 3, 8],
                                                            [5, 4], 4)
    assert p.table.tolist() == [[7, 1], [5, 2], [3, 8]]
    assert seq.tolist() == [5, 0, 5] and start.tolist() == [0, 2, 2, 7]
    assert pos.tolist() == [3, 4, 0, 1, 2, 3, 4]
    assert slots.tolist() == [31, 4, 12, 13, 14, 15, 32]
    assert (p.head, p.count) == (0, 3)                     # 9 was left, 5 and 2 follow
    assert p.free_ring[:3].tolist() == [9, 5, 2] and not refused.any()


def test_slots_pool_runs_out_in_request_order():
    table = np.full((3, 4), -1)
    p, seq, slots, _, _, refused = decode.paged_slots([0, 0, 0], [8, 5, 4], table, [0, 1, 2, 3, 4, 5], [0, 3], 4)
    assert refused.tolist() == [False, True, True] and seq.tolist() == [8, 0, 0]
    assert (slots[8:] == -1).all() and (p.head, p.count) == (2, 1)


def test_slots_of_a_bad_ring_or_too_many_blocks():
    """Nothing is taken or given back; who needs neither goes on."""
    table = np.array([[0, 1], [2, -1], [3, -1]])
    for ring in ([-1, 2], [6, 1], [0, -1], [0, 7], [0, 5]):
        p, seq, slots, _, _, refused = decode.paged_slots([5, 4, 1], [-1, 1, 1], table, [4, 5, 0, 0, 0, 0], ring, 4)
        dry = ring != [0, 5]                               # five are free, and two more would go back to a ring of six
        assert refused.tolist() == [True, dry, False] and seq.tolist() == [5, 4 if dry else 5, 2]
        assert slots.tolist() == [-1 if dry else 16, 13] and p.free_ring.tolist() == [4, 5, 0, 0, 0, 0]
        assert [p.head, p.count] == (ring if dry else [1, 4])
    p, seq, _, _, _, refused = decode.paged_slots([5, 4, 1], [-1, 0, 1], table, [4, 5, 0, 0, 0, 0], [0, 4], 4)
    assert seq.tolist() == [0, 4, 2] and not refused.any() and (p.head, p.count) == (0, 6)


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(12, 2, 8)), rng.normal(size=(12, 2, 8))
    table = np.array([[2, 0, 1], [1, 2, 0]])
    q = np.zeros((2, 4, 8))
    out, lse, _, _ = decode.paged_attention(q, k, v, table, [7, 0], 4, 0.5)
    rows = [8, 9, 10, 11, 0, 1, 2]
    assert np.allclose(out[0, 0], v[rows, 0].mean(0)) and np.allclose(out[0, 3], v[rows, 1].mean(0))
    assert np.allclose(lse[0], np.log(7)) and np.isneginf(lse[1]).all() and not out[1].any()
    out, lse, _, _ = decode.paged_attention(q, k, v, table, [7, 5], 4, 0.5, window=2)
    assert np.allclose(out[0, 0], v[[1, 2], 0].mean(0)) and np.allclose(lse[1], np.log(2))
    # one key far ahead of the others: its value
    q = np.broadcast_to(k[9, 0] * 200.0, (2, 4, 8))
    out, _, _, _ = decode.paged_attention(q, k, v, table, [7, 1], 4, 1.0)
    best = rows[int(np.argmax(k[rows, 0] @ k[9, 0]))]
    assert np.allclose(out[0, 0], v[best, 0])


def test_sample_worked_example():
    l = np.log([0.1, 0.4, 0.2, 0.3])
    for u, t in ((0.0, 0), (0.09, 0), (0.11, 1), (0.49, 1), (0.51, 2), (0.71, 3), (0.99, 3)):
        assert decode.sample_row(l, u)[0] == t
    for u, t in ((0.0, 1), (0.57, 1), (0.58, 3)):                      # two kept: 0.4 and 0.3 of 0.7
        assert decode.sample_row(l, u, top_k=2)[0] == t
        assert decode.sample_row(l, u, top_p=0.65)[0] == t
        assert decode.sample_row(l, u, min_p=0.6)[0] == t
    assert decode.sample_row(l, 0.99, top_p=0.0)[0] == 1
    assert decode.sample_row(l, 0.7, temperature=0.0)[0] == 1
    assert np.isclose(decode.sample_row(l, 0.2, top_k=2)[1], np.log(4 / 7))
    assert decode.sample_row([1.0, 2.0, 2.0], 0.99, top_k=1)[0] == 1   # lower index first among equals
    assert decode.sample_row([-np.inf, np.nan, -np.inf], 0.5)[0] == -1
    assert decode.sample_row([0.0, 1.0], 1.0)[0] == -1
    assert decode.sample_row([0.0, np.inf, np.inf], 0.6)[0] == 2


def test_sample_frequencies_follow_the_kept_distribution():
    l = np.array([0.0, 1.0, -0.5, 2.0, 1.5])
    u = (np.arange(20000) + 0.5) / 20000
    got = np.bincount([decode.sample_row(l, x, temperature=0.7, top_k=3)[0] for x in u], minlength=5) / u.size
    w = np.exp(l / 0.7) * (l >= 1.0)
    assert np.abs(got - w / w.sum()).max() < 1e-4
