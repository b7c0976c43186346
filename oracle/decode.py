"""The decode-step operators from their definitions: block tables and slot
maps, attention of one new token over a paged cache, sampling.  Plain loops
over requests, float64 (integers where the operator is integer).

Test infrastructure only: nothing in the product path imports this module.
"""
import numpy as np


class Pool:
    """State and outputs of paged_slots."""

    def __init__(self, table, free_ring, ring):
        self.table, self.free_ring = np.array(table), np.array(free_ring)
        self.head, self.count = (int(x) for x in ring)


def paged_slots(ctx, new, table, free_ring, ring, block_size):
    """One step: every request in turn takes the blocks its new tokens need from
    the front of the ring; then the ended ones' blocks go behind its end.  A ring
    state out of range stays as it is, nothing taken and nothing given back; where
    more would go back than there are blocks, nothing does.
    Returns (pool, seq_lens, slots, pos, start, refused)."""
    p = Pool(table, free_ring, ring)
    n, width = p.free_ring.size, p.table.shape[1]
    room = min(width * block_size, 2 ** 31 - 1)            # lengths are int32
    seq, slots, pos, start, refused = [], [], [], [0], []
    ring_ok = 0 <= p.head < n and 0 <= p.count <= n
    back = sum(-(-int(h) // block_size) for h, m in zip(ctx, new) if m < 0 and 0 <= h <= room)
    returns = ring_ok and p.count + back <= n
    left, taken, dry = p.count if ring_ok else 0, 0, False
    for b, (have, more) in enumerate(zip(ctx, new)):
        have, more = int(have), int(more)
        need = -(-(have + max(more, 0)) // block_size) - -(-have // block_size)
        bad = have < 0 or have + max(more, 0) > room or (more < 0 < have and not returns)
        if not bad and need > 0 and (dry or need > left):
            bad = dry = True
        refused.append(bad)
        have = min(max(have, 0), room)
        if not bad:
            for j in range(need):
                p.table[b, -(-have // block_size) + j] = p.free_ring[(p.head + taken) % n]
                taken, left = taken + 1, left - 1
        for i in range(max(more, 0)):
            at = have + i
            pos.append(at)
            slots.append(-1 if bad else int(p.table[b, at // block_size]) * block_size + at % block_size)
        start.append(len(slots))
        seq.append(have if bad else 0 if more < 0 else have + more)
    tail = p.head + p.count
    for b, (have, more) in enumerate(zip(ctx, new)):
        if more < 0 and not refused[b]:
            for j in range(-(-int(have) // block_size)):
                p.free_ring[tail % n] = p.table[b, j]
                tail += 1
    if ring_ok:
        p.head, p.count = (p.head + taken) % n, tail - p.head - taken
    return p, np.array(seq), np.array(slots, int), np.array(pos, int), np.array(start), np.array(refused)


def paged_attention(q, k_cache, v_cache, table, lens, block_size, scale, window=0):
    """out [B, Hq, D], lse [B, Hq], and for each output the sum of |p v| and the
    largest sum of |scale q k| that its rounding bounds are made of."""
    q, k_cache, v_cache = (np.asarray(a, np.float64) for a in (q, k_cache, v_cache))
    batch, hq, d = q.shape
    group = hq // k_cache.shape[1]
    out, size = np.zeros((batch, hq, d)), np.zeros((batch, hq, d))
    lse, reach = np.full((batch, hq), -np.inf), np.zeros((batch, hq))
    for b in range(batch):
        n = int(lens[b])
        j = np.arange(max(0, n - window) if window else 0, n)
        if j.size == 0:
            continue
        rows = np.asarray(table)[b, j // block_size].astype(np.int64) * block_size + j % block_size
        k, v = k_cache[rows], v_cache[rows]
        for h in range(hq):
            s = scale * (k[:, h // group] @ q[b, h])
            top = s.max()
            e = np.exp(s - top)
            p = e / e.sum()
            out[b, h] = p @ v[:, h // group]
            size[b, h] = p @ np.abs(v[:, h // group])
            lse[b, h] = top + np.log(e.sum())
            reach[b, h] = scale * (np.abs(k[:, h // group]) @ np.abs(q[b, h])).max()
    return out, lse, size, reach


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, margin, total) of one row: margin is the smallest distance
    of a running mass from a bound it is compared with, relative to the kept mass
    (a decision closer than the arithmetic's error may fall either way); total is
    the kept mass, with the largest weight as 1."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    bad = not (0.0 <= temperature < np.inf) or np.isnan(top_p) or not min_p <= 1.0 or not 0.0 <= u < 1.0
    if bad or not (l > -np.inf).any():
        return -1, np.nan, np.inf, 0.0
    top = l.max()
    if temperature == 0.0:
        return int(np.argmax(l)), 0.0, np.inf, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(l == top, 1.0, np.exp((l - top) / np.float64(temperature)))
    order = np.lexsort((np.arange(l.size), -l))
    order = order[l[order] > -np.inf]
    margin = np.inf
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1.0:
        total = w[order].sum()
        before = np.cumsum(w[order]) - w[order]
        if (w[order] < 1.0).any():                          # else the masses are whole numbers, free of rounding
            margin = min(margin, float(np.abs(before[1:] - top_p * total).min() / total))
        keep = before < top_p * total
        keep[0] = True
        order = order[keep]
    if min_p > 0.0:
        inexact = w[order][w[order] < 1.0]                 # the largest weight is 1 without any rounding
        margin = min(margin, float(np.abs(inexact / np.float64(min_p) - 1.0).min()) if inexact.size else np.inf)
        order = order[w[order] >= np.float64(min_p)]
    ids = np.sort(order)
    mass = np.cumsum(w[ids])
    if (w[ids] < 1.0).any():
        margin = min(margin, float(np.abs(mass - np.float64(u) * mass[-1]).min() / mass[-1]))
    at = min(int(np.searchsorted(mass, np.float64(u) * mass[-1], side="right")), ids.size - 1)
    return int(ids[at]), float(np.log(w[ids[at]] / mass[-1])), margin, float(mass[-1])
