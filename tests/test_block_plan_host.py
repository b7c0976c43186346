"""Which kernel takes a call of the block-scaled Linear (csrc/block_plan.h), compiled for the
host: the estimates against the same formulas in Python's integers, up to the largest
sizes that the entry point admits, and the choice on the documented sizes."""
import os
import random
import subprocess

import pytest

from conftest import ROOT
from test_decode_host import A, call, gbf, last   # noqa: F401

PROGRAM = r"""
#include <cstdio>
#include "block_plan.h"
int main() {
  long long m, n, k;
  gbf::LinearBlockRoom r = {};
  while (scanf("%lld %lld %lld %d %d %d %d %d", &m, &n, &k, &r.sms, &r.clusters[1], &r.clusters[2], &r.clusters[3],
               &r.clusters[4]) == 8) {
    const gbf::LinearBlockPlan p = gbf::plan_linear_block(m, n, k, r);
    printf("%lld %lld %lld %d %d %lld\n", static_cast<long long>(gbf::linear_block_ns(m, n, k, 64, r.sms)),
           static_cast<long long>(gbf::linear_block_ns(m, n, k, 128, r.sms)),
           static_cast<long long>(gbf::linear_block_pair_ns(m, n, k, r)), p.rows, p.split, static_cast<long long>(p.tiles));
  }
}
"""
GB300 = (152, 76, 36, 22, 16)          # SMs; clusters of one to four pairs (the larger ones fit a few fewer on some GPUs)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "csrc"), str(d / "plan.cpp"),
                    "-o", str(d / "plan")], check=True)

    def run(sizes, room=GB300):
        text = "".join(" ".join(map(str, (*s, *room))) + "\n" for s in sizes)
        out = subprocess.run([str(d / "plan")], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def up(a, b):
    return -(-a // b)


def expected(m, n, k, room=GB300):
    sms, fits, blocks = room[0], room[1:], up(k, 128)

    def single(rows):
        tiles, split = up(m, rows) * up(n, 128), 1
        while split < 8 and tiles * split * 2 <= sms and blocks >= split * 8:
            split *= 2
        extra = 0 if split == 1 else 1500 if rows == 64 else 3000
        return up(tiles, sms) * (2200 + up(blocks, split) * (270 if rows == 64 else 335)) + extra, split, tiles

    tiles = up(m, 256) * up(n, 256)
    split = next(s for s in (4, 3, 2, 1) if s == 1 or (blocks >= s * 6 and tiles <= fits[s - 1]))
    pair = up(tiles, fits[split - 1]) * (up(blocks, split) * 390 + 2200) + 5000 + (0 if split == 1 else 4000)
    t64, t128 = single(64)[0], single(128)[0]
    if m <= 32:
        rows = 16 if m <= 16 else 32
    else:
        rows = 256 if pair < t64 and pair < t128 else 64 if t64 <= t128 else 128
    return t64, t128, pair, rows, *((split, tiles) if rows == 256 else single(rows)[1:])


def test_estimates_do_not_wrap(plans):
    """K up to 2^31 (2^24 blocks, 335 ns each, are beyond 32 bits), and all tiles that are admitted."""
    top = (1 << 31) - 16
    sizes = [(33, 8, top), (64, 4096, top), (64, 4096, 820_000_000), (300, 128, 700_000_000), (5000, 4096, 1_000_000_000),
             (top, 128, top), ((1 << 31) - 1, 8064, 16), (64, top, top), (1 << 20, 1 << 17, 16)]
    for s, got in zip(sizes, plans(sizes)):
        assert got == expected(*s), s
        assert all(t > 0 for t in got[:3]) and got[4] * got[5] < 1 << 31, s


def test_choice_over_the_sizes_of_use(plans):
    rng = random.Random(5)
    size = lambda step, hi: step * int(round((hi / step) ** rng.random()))            # noqa: E731
    sizes = [(size(1, 16384), size(8, 32768), size(16, 32768)) for _ in range(400)]
    for room in (GB300, (148, 74, 35, 20, 14), (20, 9, 4, 2, 1)):
        for s, got in zip(sizes, plans(sizes, room)):
            assert got == expected(*s, room), (s, room)


def test_choice_on_the_documented_sizes(plans):
    sizes = [(1, 4096, 4096), (32, 16384, 4096), (512, 4096, 4096), (333, 4096, 11008), (1024, 4096, 4096), (8192, 16384, 4096),
             (256, 5120, 8192), (256, 4096, 14336)]
    assert [p[3:5] for p in plans(sizes)] == [(16, 4), (32, 1), (128, 1), (256, 2), (256, 1), (256, 1), (256, 3), (256, 4)]


def test_without_room_for_pairs_single_ctas_work(plans):
    for p in plans([(333, 4096, 11008), (8192, 16384, 4096)], (152, 0, 0, 0, 0)):
        assert p[3] in (64, 128)


def test_tiles_past_the_grid_are_refused(gbf):                                        # noqa: F811
    """Fewer than 2^31 tiles of 128 x 128, but not of the 64 x 128 that a call may be cut into."""
    names = [("x", A(0)), ("sx", A(1 << 20)), ("w", A(2 << 20)), ("sw", A(3 << 20)), ("bias", None), ("y", A(4 << 20)),
             ("m", (1 << 31) - 1), ("n", 12800), ("k", 16), ("act", 0), ("stream", None)]
    assert call(gbf.raw().gbfb_linear_fp8, names, {}) == gbf.EUNSUPPORTED and "64 x 128" in last(gbf)


def test_the_librarys_answer(gbf):                                                    # noqa: F811
    plan = gbf.linear_fp8_block_plan
    assert plan(0, 64, 256) == (0, 0)
    for bad in ((-1, 64, 256), (4, 0, 256), (4, 64, 0), (4, 60, 256), (4, 64, 136), (1 << 31, 64, 256)):
        with pytest.raises(gbf.GbfError):
            plan(*bad)
    assert gbf.raw().gbfb_linear_fp8_plan(4, 64, 256, None, None) == gbf.EINVAL
