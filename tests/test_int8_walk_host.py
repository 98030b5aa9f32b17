"""The walk of the large int8 tiles over ragged groups, on the host: the plan and the order of the tiles are csrc/int8_plan.h's,
the search among the groups is modelled as the kernel does it, 64 groups at a time and forward only."""
import random

import pytest

import int8_plan as P

LT = 256


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return P.load(str(tmp_path_factory.mktemp("plan")))


def _walk(lib, M, cols, K, off, swiglu):
    """Every tile (group, first row, column tile) that some workgroup takes; asserts that each lies where a group's rows are."""
    G = len(off) - 1
    kind, most, _ = P.plan(lib, M, cols, K, G, swiglu)
    if kind != P.LARGE:
        return None
    width = LT // 2 if swiglu else LT
    tiles_n = (cols + width - 1) // width
    clamp = lambda v, lo: lo if v < lo else min(v, M)  # noqa: E731
    lo = [clamp(v, 0) for v in off[:-1]]
    hi = [clamp(v, a) for a, v in zip(lo, off[1:])]
    count = [(b - a + LT - 1) // LT for a, b in zip(lo, hi)]
    T, grid, taken = lib.tiles(sum(count), tiles_n, most), lib.groups(most), []
    assert 0 <= T <= most
    for workgroup in range(grid):
        base = before = 0
        for b in range(workgroup, T, grid):
            v = lib.tile(b, T)
            assert 0 <= v < T
            row = v // tiles_n
            while row - before >= sum(count[base:base + 64]):
                before += sum(count[base:base + 64])
                base += 64
                assert base < G
            at = row - before
            assert at >= 0, (workgroup, b, v)                 # else no group of the 64 begins ahead of it
            grp = base
            while at >= count[grp]:
                at -= count[grp]
                grp += 1
            assert 0 <= lo[grp] + at * LT < hi[grp] <= M
            taken.append((grp, lo[grp] + at * LT, v % tiles_n))
    return taken, [(g, m, n) for g in range(G) for m in range(lo[g], hi[g], LT) for n in range(tiles_n)]


@pytest.mark.parametrize("swiglu", [False, True])
def test_every_tile_once(lib, swiglu):
    rng, seen = random.Random(3), 0
    for _ in range(60):
        G = rng.choice([1, 2, 3, 8, 64, 65, 130, 200])
        sizes = [rng.choice([0, 1, 65, 100, 256, 257, rng.randrange(1500)]) for _ in range(G)]
        off = [rng.randrange(20)]
        for s in sizes:
            off.append(off[-1] + s)
        r = _walk(lib, off[-1] + rng.randrange(300), rng.randrange(300, 5000), 256, off, swiglu)
        if r:
            seen += 1
            assert sorted(r[0]) == r[1]
    assert seen > 20


@pytest.mark.parametrize("swiglu", [False, True])
def test_offsets_that_break_the_rule_stay_among_the_groups(lib, swiglu):
    """Groups that overlap, run backwards or leave the rows: at most the plan's tiles, none outside its group, no workgroup ever
    looks for a group behind it."""
    rng, seen = random.Random(4), 0
    cases = [(4161, 350 if swiglu else 700, [0 if i % 2 == 0 else 4161 for i in range(66)])]       # 65 groups, 246 workgroups
    for _ in range(80):
        G, M = rng.choice([1, 5, 64, 65, 70, 129, 260]), rng.randrange(500, 20000)
        cases.append((max(M, 65 * G), rng.randrange(100, 4000), [rng.randrange(-50, 2 * M) for _ in range(G + 1)]))
    for M, cols, off in cases:
        r = _walk(lib, M, cols, 256, off, swiglu)
        if r:
            seen += 1
            assert set(r[0]) <= set(r[1])
    assert seen > 20
