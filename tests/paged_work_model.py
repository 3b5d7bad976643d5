"""The work list of paged attention in plain integers (csrc/paged.cuh): items,
segments, the cut among the CTAs, and where the partial results lie."""


def tile_rows(rows, most):
    m = 16
    while m < most and m < rows:
        m *= 2
    return m


def tile_units(tm, most):
    """Units of a key tile (where segments count extra tiles)."""
    return {16: 1, 32: 2, 64: 3}[tm] if most == 64 else 1


def spans(items, hkv, bn, most):
    """items: (rows, lo, hi).  Per item: (key tiles of all segments, part rows, rows of a segment's partials,
    row tiles, key tiles)."""
    out = []
    for rows, lo, hi in items:
        tm = tile_rows(rows, most)
        rt = -(-rows // tm)
        nt = (hi + bn - 1) // bn - lo // bn if hi > lo and rows > 0 else 0
        out.append((hkv * rt * nt, hkv * rt * tm, tm, rt, nt))
    return out


def cut(items, hkv, bn, most, ctas, snap, extra):
    """(total units, chunk, extra tiles of a segment): as paged_schedule decides them."""
    sp = spans(items, hkv, bn, most)
    total, segs = sum(x[0] for x in sp), sum(hkv * x[3] for x in sp if x[4] > 0)
    chunk = 0
    if snap > 0:
        if 2 * segs < ctas and total > 0:
            want = -(-total // (ctas - segs))
            if want <= total // ctas + snap:
                chunk = want
        extra = 0
    else:
        full = sum(hkv * x[3] * (x[4] + extra) * tile_units(x[2], most) for x in sp if x[4] > 0)
        if total <= ctas or full < tile_units(64, most) * ctas:
            extra = 0
    return sum(hkv * x[3] * padded(x, most, chunk, extra) for x in sp), chunk, extra


def weight(span, most, extra):
    """Units of one of its key tiles."""
    return tile_units(span[2], most) if extra > 0 else 1


def padded(span, most, chunk, extra):
    """Units of a segment."""
    nt = span[4]
    return -(-nt // chunk) * chunk if chunk else (nt + extra) * weight(span, most, extra) if nt else 0


def first(c, total, chunk, ctas):
    if chunk:
        return min(c * chunk, total)
    n = min(ctas, total)
    return c * total // n if c < n else total


def owner(unit, total, chunk, ctas):
    return unit // chunk if chunk else ((unit + 1) * min(ctas, total) - 1) // total


def pieces(items, hkv, bn, most, ctas, snap=0, extra=0):
    """Every piece of every CTA: (cta, item, segment, first key tile, tiles, first partial row, rows)."""
    sp = spans(items, hkv, bn, most)
    total, chunk, extra = cut(items, hkv, bn, most, ctas, snap, extra)
    got = []
    for c in range(ctas):
        u0 = first(c, total, chunk, ctas)
        left = first(c + 1, total, chunk, ctas) - u0
        if left <= 0:
            continue
        unit = row = i = 0
        units = lambda x: hkv * sp[x][3] * padded(sp[x], most, chunk, extra)  # noqa: E731
        tiles = lambda n: -(-n // weight(sp[i], most, extra))  # noqa: E731
        while not (units(i) > 0 and unit <= u0 < unit + units(i)):
            unit, row, i = unit + units(i), row + sp[i][1], i + 1
        seg, skip = divmod(u0 - unit, padded(sp[i], most, chunk, extra))
        kt = tiles(skip)
        count = min(sp[i][4], tiles(skip + left)) - kt
        while True:
            if count > 0:
                got.append((c, i, seg, kt, count, c * most + row + seg * sp[i][2], sp[i][2]))
            left -= padded(sp[i], most, chunk, extra) - skip
            if chunk or left <= 0:
                break
            kt, skip, seg = 0, 0, seg + 1
            if seg == hkv * sp[i][3]:
                seg = 0
                row, i = row + sp[i][1], i + 1
                while sp[i][4] == 0:
                    row, i = row + sp[i][1], i + 1
            count = min(sp[i][4], tiles(left))
    return got, sp, total, chunk, extra
