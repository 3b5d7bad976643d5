"""The work list of paged attention in plain integers (csrc/paged.cuh): items,
segments, the cut among the CTAs, and where the partial results lie."""


def tile_rows(rows, most):
    m = 16
    while m < most and m < rows:
        m *= 2
    return m


def part_tile(tm, most):
    """Rows of a segment's partials: two partials of small tiles where tiles reach 256 rows."""
    return 2 * tm if most == 256 and tm <= 128 else tm


def spans(items, hkv, bn, most):
    """items: (rows, lo, hi).  Per item: (units, part rows, partial rows of a segment, row tiles, key tiles)."""
    out = []
    for rows, lo, hi in items:
        tm = tile_rows(rows, most)
        rt = -(-rows // tm)
        nt = (hi + bn - 1) // bn - lo // bn if hi > lo and rows > 0 else 0
        pm = part_tile(tm, most)
        out.append((hkv * rt * nt, hkv * rt * pm, pm, rt, nt))
    return out


def pieces(items, hkv, bn, most, ctas):
    """Every piece of every CTA: (cta, item, segment, first key tile, tiles, first partial row, rows)."""
    sp = spans(items, hkv, bn, most)
    total = sum(s[0] for s in sp)
    ctas = min(ctas, total)
    got = []
    for c in range(ctas):
        u0, u1 = c * total // ctas, (c + 1) * total // ctas
        left = u1 - u0
        if left <= 0:
            continue
        unit = row = i = 0
        while not (sp[i][0] > 0 and unit <= u0 < unit + sp[i][0]):
            unit, row, i = unit + sp[i][0], row + sp[i][1], i + 1
        seg, kt = divmod(u0 - unit, sp[i][4])
        count = min(sp[i][4] - kt, left)
        while True:
            got.append((c, i, seg, kt, count, c * most + row + seg * sp[i][2], sp[i][2]))
            left -= count
            if left <= 0:
                break
            kt, seg = 0, seg + 1
            if seg == hkv * sp[i][3]:
                seg = 0
                row, i = row + sp[i][1], i + 1
                while sp[i][4] == 0:
                    row, i = row + sp[i][1], i + 1
            count = min(sp[i][4], left)
    return got, sp, total


def owner(unit, total, ctas):
    ctas = min(ctas, total)
    return ((unit + 1) * ctas - 1) // total
