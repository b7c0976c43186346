"""The CTA pair's walk after a wait that gave up (csrc/gemm_block_pair.cu): a model
of its hardware barriers, with every order of steps tried.

One half of one CTA: W epilogue warps and the issuer (or the relay) share two barriers
of W + 1 arrivals, K block i uses barrier i % 2.
  epilogue, block i   while its waits succeed: it goes on once block i's MMAs are done,
                      which were issued after block i - 2 was taken back, and arrives
                      without waiting.  From the wait that gives up on (at any block): it
                      arrives without one.
  issuer, block i     takes back block i - 2: arrives and waits for the barrier's phase;
                      at the end the last two.
A barrier counts arrivals, whoever they are from, and its phase ends at W + 1 of them.
"""
import os
import re

import pytest

from conftest import ROOT


def stuck(blocks, warps, ordered):
    """Whether some order of steps leaves a role waiting for ever.  `ordered`: a warp
    whose wait gave up still waits until block i - 2 was taken back, by the issuer's count."""
    # state: each warp's (next block, gave up), the issuer's (next block to take back, its phase while
    # it waits or -1), each barrier's (phase, arrivals)
    start = (tuple((0, False) for _ in range(warps)), (0, -1), ((0, 0), (0, 0)))
    seen, todo = {start}, [start]

    def arrive(bars, b):
        phase, n = bars[b]
        new = (phase + 1, 0) if n == warps else (phase, n + 1)
        return tuple(new if i == b else bars[i] for i in range(2))

    while todo:
        ws, (took, waits), bars = todo.pop()
        steps = []
        for w, (i, gone) in enumerate(ws):
            if i == blocks:
                continue
            if not gone:
                steps.append((ws[:w] + ((i, True),) + ws[w + 1:], (took, waits), bars))
            # MMAs of block i may be done once block i - 2 was taken back
            if i < 2 or took > i - 2 or (gone and not ordered):
                steps.append((ws[:w] + ((i + 1, gone),) + ws[w + 1:], (took, waits), arrive(bars, i % 2)))
        if took < blocks:
            b = took % 2
            if waits < 0:
                phase = bars[b][0]
                after = arrive(bars, b)
                steps.append((ws, (took + 1, -1) if after[b][0] != phase else (took, phase), after))
            elif bars[b][0] != waits:
                steps.append((ws, (took + 1, -1), bars))
        if not steps and (took < blocks or any(i < blocks for i, _ in ws)):
            return True
        for s in steps:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return False


def test_arrivals_out_of_step_can_hang():
    """Why the order is kept: with it left out some order of steps never ends."""
    assert stuck(4, 2, ordered=False)


@pytest.mark.parametrize("blocks,warps", [(1, 4), (2, 4), (3, 4), (5, 4), (6, 4), (9, 2), (12, 2)])
def test_every_order_of_steps_ends(blocks, warps):
    assert not stuck(blocks, warps, ordered=True)


def test_the_kernel_keeps_that_order():
    """A warp whose wait gave up waits for the count before each of its arrivals, and the two
    roles that take back publish theirs behind each barrier."""
    text = open(os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "csrc", "gemm_block_pair.cu")).read()
    epilogue = text[text.index("// ---------------------------------------------------------------- epilogue"):]
    arrivals = [m.start() for m in re.finditer(r"give_back\(", epilogue)]
    assert len(arrivals) == 2                              # while the waits succeed, and after one that gave up
    walk = epilogue[epilogue.index("if (!ok) {"):arrivals[1]]
    assert re.search(r"for \(; it < all; \+\+it\) \{\s+if \(it >= 2\) wait_taken\(&ctl->taken\[half\], it - 1\);", walk)
    assert "if (!ok) break;" in epilogue[:arrivals[0]]
    taken = re.findall(r"^ +(take_back|set_taken)\(", text, re.M)
    assert taken == ["take_back", "set_taken", "take_back", "set_taken", "take_back", "set_taken"]


def test_accumulators_change_hands_at_cluster_scope():
    """The barriers of an accumulator, which the pair's other CTA arrives on, are waited for at
    the scope that holds both CTAs, between the fences that order tensor memory."""
    read = lambda name: open(os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "csrc", name)).read()    # noqa: E731
    text = read("gemm_block_pair.cu")
    waits = re.findall(r"(\w+)(?:<[\w, ]*>)?\(&ctl->(acc_full|peer_gave)\[", text)
    waits = {(f, bar) for f, bar in waits if f not in ("mbar_init", "commit_pair", "smem_u32")}
    assert waits == {("wait_accumulator", "acc_full"), ("wait_accumulator", "peer_gave"), ("test_accumulator", "acc_full")}
    assert "mbar_wait<true, false, true>" in text and "mbarrier.test_wait.parity.relaxed.cluster" in text
    assert '".relaxed.cluster"' in read("tma.cuh") and "mbarrier.arrive.relaxed.cluster" in text
    relay = text[text.index("-- relay"):text.index("-- scales")]
    assert re.search(r"take_back\(.*?tc_fence_after\(\);\s+tc_fence_before\(\);\s+if \(elected\) mbar_arrive_relaxed", relay, re.S)
