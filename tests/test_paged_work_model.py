"""The cut of paged attention's work list, checked on the CPU: every key tile of
every segment is worked on once, partial results never overlap and stay within
the rows that the workspace is sized for, and the join finds each segment's
partials by its formula."""

import random

import pytest

from tests import paged_work_model as M


@pytest.mark.parametrize("seed", range(250))
def test_pieces_cover_and_partials_are_apart(seed):
    r = random.Random(seed)
    bn, most = r.choice([(64, 64), (32, 16), (128, 256), (64, 128)])
    hkv, ctas = r.choice([1, 2, 3, 8]), r.choice([1, 7, 148, 296, 444])
    items = []
    for _ in range(r.randint(1, 30)):
        lo = r.choice([0, 0, r.randint(0, 3000)])
        items.append((r.choice([0, 1, 4, 16, 17, 40, 64, 65, 128, 129, 256, 257, 500]), lo, max(lo, lo + r.randint(-100, 4000))))
    snap, extra = r.choice([(0, 0), (0, 1), (0, 3), (4, 0), (40, 0)])
    got, sp, total, chunk, extra = M.pieces(items, hkv, bn, most, ctas, snap, extra)
    rows_total = sum(s[1] for s in sp) + ctas * most
    taken, intervals = {}, []
    for c, i, seg, kt, count, row, rows in got:
        assert count > 0 and 0 <= seg < hkv * sp[i][3] and kt + count <= sp[i][4]
        for x in range(kt, kt + count):
            assert (i, seg, x) not in taken
            taken[i, seg, x] = c
        intervals.append((row, row + rows))
        assert 0 <= row and row + rows <= rows_total
    assert len(taken) == sum(s[0] for s in sp)
    if chunk:
        assert total <= chunk * ctas and len({g[0] for g in got}) == len(got)
    intervals.sort()
    assert all(a[1] <= b[0] for a, b in zip(intervals, intervals[1:]))
    # the join's view
    unit = base = 0
    by = {(c, i, seg): row for c, i, seg, _, _, row, _ in got}
    for i, (_, part, pm, rt, nt) in enumerate(sp):
        units = M.padded(sp[i], most, chunk, extra)
        for seg in range(hkv * rt if nt else 0):
            u0 = unit + seg * units
            last = u0 + (nt - 1) * M.weight(sp[i], most, extra)
            c0, c1 = M.owner(u0, total, chunk, ctas), M.owner(last, total, chunk, ctas)
            first = c0 * most + base + seg * pm
            for c in range(c0, c1 + 1):
                assert by[c, i, seg] == first + (c - c0) * most
                assert any(taken[i, seg, x] == c for x in range(nt))
        unit, base = unit + hkv * rt * units, base + part


def test_division_by_a_product():
    """FastDiv of csrc/serving.h: exact for every 31-bit number, at the ends and borders of each divisor."""
    r = random.Random(0)
    for d in list(range(1, 3000)) + [2 ** i + j for i in range(12, 31) for j in (-1, 0, 1)] + [2 ** 31 - 1]:
        shift = 0
        while (1 << shift) < d:
            shift += 1
        mul = (((1 << shift) - d) << 32) // d + 1
        assert mul < 2 ** 32
        top = 2 ** 31 - 1
        ns = [0, 1, d - 1, d, d + 1, top, top - 1, top // d * d, top // d * d - 1] + [r.randint(0, top) for _ in range(20)]
        for n in ns:
            if 0 <= n <= top:
                assert (((n * mul) >> 32) + n) < 2 ** 32 and (((n * mul) >> 32) + n) >> shift == n // d, (n, d)
