"""Batches in which the kernels of paged attention run for many key tiles (test
code only): rings that wrap several times, CTAs with several pieces, maxima that
grow along the keys.  What each case has to reach is counted by the work list's
model (tests/paged_work_model.py) with the kernels' constants."""

import numpy as np
import torch

from tests import paged_work_model as M
from tests import serving_cases as C

BF16, F32 = torch.bfloat16, torch.float32
SMS = 148
CTAS = {64: 3, 128: 2, 256: 1}  # of the list kernels on an SM
SNAP, EXTRA = 4, 2
OWN_ROWS, OWN_WORK = 32, 1 << 30


def _drafted(groups, seqs, n, prefix, step=1):
    """groups of `seqs` sequences with n new tokens each behind prefixes of about `prefix` tokens."""
    ptr = [g * seqs for g in range(groups + 1)]
    lens = [prefix + 13 * g for g in range(groups)]
    held = [lens[b // seqs] + n + step * (b % 7) for b in range(groups * seqs)]
    return [n] * (groups * seqs), held, (ptr, lens)


# name: (dtype, hq, hkv, d, page, (new, held, groups), what the case has to reach)
#   pieces: of some CTA, in the prefixes' list ("prefix") or the other ("list"); tiles: of some piece;
#   apart: whether the prefix kernel's lanes share their rows (None: d 256 has one lane)
CASES = {
    # several pieces a CTA: segments enough that no chunk is chosen
    "pieces_d128": (BF16, 32, 8, 128, 16, _drafted(5, 15, 5, 2800), dict(kind="prefix", pieces=2, tiles=12, apart=False)),
    "pieces_d128_apart": (BF16, 32, 8, 128, 32, _drafted(10, 6, 4, 1500), dict(kind="prefix", pieces=2, tiles=5, apart=True)),
    "pieces_d64": (BF16, 32, 8, 64, 16, _drafted(5, 15, 5, 2800), dict(kind="prefix", pieces=2, tiles=12, apart=False)),
    "pieces_d64_apart": (BF16, 16, 8, 64, 64, _drafted(10, 9, 4, 1600), dict(kind="prefix", pieces=2, tiles=5, apart=True)),
    "pieces_d256": (BF16, 16, 8, 256, 16, _drafted(5, 15, 5, 1300), dict(kind="prefix", pieces=2, tiles=12, apart=None)),
    # one long piece a CTA
    "long_d128": (BF16, 32, 4, 128, 64, _drafted(5, 5, 6, 9300), dict(kind="prefix", pieces=1, tiles=10, apart=False)),
    "long_d128_apart": (BF16, 32, 4, 128, 16, _drafted(5, 8, 2, 9300), dict(kind="prefix", pieces=1, tiles=10, apart=True)),
    "long_d64_apart": (BF16, 16, 4, 64, 128, _drafted(5, 8, 3, 9300), dict(kind="prefix", pieces=1, tiles=10, apart=True)),
    "long_d256": (BF16, 16, 4, 256, 32, _drafted(5, 6, 5, 4700), dict(kind="prefix", pieces=1, tiles=10, apart=None)),
    # sequences with keys of their own: 16, 32 and 64 rows a tile
    "own_16": (BF16, 16, 4, 128, 16, ([1] * 7, [7001 + 311 * b for b in range(7)], None),
               dict(kind="list", pieces=2, tiles=10)),
    "own_32": (BF16, 16, 4, 128, 64, ([6] * 7, [7001 + 311 * b for b in range(7)], None),
               dict(kind="list", pieces=2, tiles=10)),
    "own_64": (BF16, 16, 4, 64, 32, ([16] * 8, [8001 + 1311 * b for b in range(8)], None),
               dict(kind="list", pieces=2, tiles=10)),
    "own_d256": (BF16, 8, 4, 256, 16, ([1] * 6, [3001 + 911 * b for b in range(6)], None),
                 dict(kind="list", pieces=2, tiles=10)),
    "own_64_d256": (BF16, 8, 4, 256, 128, ([31] * 6, [3001 + 911 * b for b in range(6)], None),
                    dict(kind="list", pieces=2, tiles=10)),
    "own_many_rows": (BF16, 16, 2, 128, 16, ([300, 1, 70], [1900, 5000, 2070], None),
                      dict(kind="list", pieces=2, tiles=8)),
    "f32_d128": (F32, 16, 4, 128, 16, ([1] * 5, [4001 + 711 * b for b in range(5)], None),
                 dict(kind="list", pieces=2, tiles=10)),
    "f32_d64": (F32, 16, 4, 64, 64, ([9] * 5, [3001 + 511 * b for b in range(5)], None),
                dict(kind="list", pieces=2, tiles=10)),
    # contexts of 20 to 128 thousand tokens
    "prefix_128k": (BF16, 16, 2, 128, 16, _drafted(1, 16, 1, 131072), dict(kind="prefix", pieces=1, tiles=10, apart=True)),
    "prefix_128k_rows": (BF16, 32, 2, 128, 64, _drafted(1, 16, 1, 131059), dict(kind="prefix", pieces=1, tiles=10, apart=False)),
    "prefix_40k_d256": (BF16, 16, 2, 256, 16, _drafted(1, 12, 1, 40001), dict(kind="prefix", pieces=1, tiles=8, apart=None)),
    "own_60k": (BF16, 8, 2, 128, 128, ([1, 2, 1], [60001, 41007, 128], None), dict(kind="list", pieces=2, tiles=10)),
    "f32_20k": (F32, 8, 2, 128, 16, _drafted(1, 6, 1, 20011), dict(kind="list", pieces=2, tiles=8)),
    "f32_d256_group": (F32, 8, 2, 256, 32, _drafted(1, 5, 3, 6000), dict(kind="list", pieces=2, tiles=10)),
}


def room(name):
    """Tokens that the table has room for: as many as send the prefixes to their own kernel, where the case is about it."""
    dtype, hq, hkv, d, page, (new, held, groups), reach = CASES[name]
    if reach["kind"] != "prefix":
        return 0
    return -(-OWN_WORK // (sum(new) * hq // hkv * hkv * d)) + page


def lists(name):
    """The items of both lists: (of the prefixes' own list, of the other)."""
    dtype, hq, hkv, d, page, (new, held, groups), _ = CASES[name]
    gh = hq // hkv
    cap = max(max(held), room(name))
    own, rest = [], []
    prefix_of = [0] * len(new)
    if groups is not None:
        ptr, lens = groups
        rows = [sum(new[ptr[g]:ptr[g + 1]]) * gh for g in range(len(lens))]
        mine = dtype == BF16 and max(rows) > OWN_ROWS and sum(rows) * hkv * d * cap >= OWN_WORK
        (own if mine else rest).extend((rows[g], 0, lens[g]) for g in range(len(lens)))
        for g in range(len(lens)):
            prefix_of[ptr[g]:ptr[g + 1]] = [lens[g]] * (ptr[g + 1] - ptr[g])
    most_items = [r[0] for r in rest] + [n * gh for n in new]
    rest += [(n * gh, min(prefix_of[b], held[b]), held[b]) for b, n in enumerate(new)]
    return own, rest, max(most_items)


def reached(name):
    """(most pieces of a CTA, most key tiles of a piece, rows a tile of the longest pieces) of the list that the case is about."""
    dtype, hq, hkv, d, page, _, reach = CASES[name]
    own, rest, most_rows = lists(name)
    if reach["kind"] == "prefix":
        assert own
        got = M.pieces(own, hkv, 64 if d == 256 else 128, 128 if d == 256 else 256, SMS, snap=SNAP)[0]
    else:
        bn, most = (64, 16 if most_rows <= 16 else 64) if dtype == BF16 else (32, 16)
        got = M.pieces(rest, hkv, bn, most, SMS * CTAS[d], extra=EXTRA)[0]
    per = {}
    for c, *_ in got:
        per[c] = per.get(c, 0) + 1
    tiles = max(g[4] for g in got)
    return max(per.values()), tiles, {g[6] for g in got if g[4] == tiles}


def build(name, seed=0):
    """The case's cache and queries.  Some query rows see keys that rise in three steps of 9 bits along the
    sequence, some the other way, some neither: running maxima grow in the middle of a piece, and what was
    gathered before still counts."""
    dtype, hq, hkv, d, page, (new, held, groups), _ = CASES[name]
    st = C.Step(seed, dtype, hq, hkv, d, page, new, held, groups, extra_rows=1, values="peaks", room=room(name))
    g = torch.Generator().manual_seed(seed + 1)
    u = torch.randn(hkv, d, generator=g)
    u /= u.norm(dim=-1, keepdim=True)
    steps, height = 3, 1.5  # a step of the keys along u
    kp = st.k_pages.float()
    done = set()
    for b in range(len(new)):
        first, shared = b, 0
        if groups is not None:
            x = int(np.searchsorted(groups[0], b, side="right") - 1)
            first, shared = groups[0][x], groups[1][x]
        n = max(held[b], shared if first == b else 0)
        for i in range(-(-n // page)):
            p = int(st.table[b, i])
            if p in done:
                continue
            done.add(p)
            s = torch.arange(i * page, (i + 1) * page)
            level = torch.clamp((steps + 1) * s // max(held[b], 1), max=steps).float() * height
            kp[p] += level[None, :, None] * u[:, None, :]
    st.k_pages = kp.to(dtype)
    # a row's coefficient: its logits rise by 9 bits a step, fall, or stay
    c = torch.tensor([1.0, 0.0, -1.0])[torch.randint(0, 3, (st.q.shape[0], hq), generator=g)]
    rise = 9 * np.log(2) / height * d ** 0.5
    q = st.q.float().reshape(-1, hkv, hq // hkv, d)
    q += (c.reshape(q.shape[:3]) * rise)[..., None] * u[None, :, None, :]
    st.q = q.reshape(-1, hq, d).to(dtype)
    return st


def want(st, device, scale=None):
    """(out, lse, mean of |v|) of the definition in 64 bits, a sequence at a time, on `device`."""
    f64 = torch.float64
    kp, vp, q = st.k_pages.to(device), st.v_pages.to(device), st.q.to(device)
    T, hq, d, hkv, page = st.cu[-1], st.hq, st.d, st.hkv, st.page
    scale = d ** -0.5 if scale is None else scale
    out, mean = (torch.zeros(T, hq, d, dtype=f64, device=device) for _ in range(2))
    lse = torch.full((T, hq), -float("inf"), dtype=f64, device=device)
    for b in range(len(st.new)):
        n, held, first, shared = st.new[b], st.held[b], b, 0
        if n == 0 or held <= 0:
            continue
        if st.groups is not None:
            x = int(np.searchsorted(st.groups[0], b, side="right") - 1)
            first, shared = st.groups[0][x], st.groups[1][x]
        s = torch.arange(held)
        rows = torch.from_numpy(st.table).long()
        pages = torch.where(s < shared, rows[first, s // page], rows[b, s // page]).to(device)
        slots = (s % page).to(device)
        k, v = kp[pages, :, slots].to(f64), vp[pages, :, slots].to(f64)  # [held, hkv, d]
        t0 = st.cu[b]
        x = torch.einsum("tgrd,sgd->tgrs", q[t0:t0 + n].to(f64).reshape(n, hkv, hq // hkv, d), k) * scale
        seen = held - n + 1 + torch.arange(n, device=device)
        x = x.masked_fill((torch.arange(held, device=device) >= seen[:, None])[:, None, None], -float("inf"))
        live = seen > 0
        p = torch.softmax(x[live], -1)
        out[t0:t0 + n][live] = torch.einsum("tgrs,sgd->tgrd", p, v).reshape(-1, hq, d)
        mean[t0:t0 + n][live] = torch.einsum("tgrs,sgd->tgrd", p, v.abs()).reshape(-1, hq, d)
        lse[t0:t0 + n][live] = torch.logsumexp(x[live], -1).reshape(-1, hq)
    return tuple(t.cpu().numpy() for t in (out, lse, mean))
