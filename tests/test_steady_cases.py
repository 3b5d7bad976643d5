"""Paged attention over many key tiles: by the work list's model the cases reach
several pieces a CTA and rings that wrap (CPU), and the results hold (GPU)."""

import os
import random
import re

import numpy as np
import pytest
import torch

from dynamic_hierarchical_sparse_b200 import api
from tests import paged_work_model as M, serving_cases as C, steady_cases as T

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "dynamic_hierarchical_sparse_b200", "csrc")


@pytest.mark.parametrize("name", T.CASES)
def test_case_reaches_what_it_is_for(name):
    d, want = T.CASES[name][3], T.CASES[name][6]
    pieces, tiles, rows = T.reached(name)
    assert pieces >= want["pieces"] and tiles >= want["tiles"], (pieces, tiles)
    if want["pieces"] == 1:
        assert pieces == 1
    if want["kind"] == "prefix" and want["apart"] is not None:
        assert all((r < 256) == want["apart"] for r in rows), rows


def test_constants_are_the_kernels():
    src = {f: open(os.path.join(CSRC, f)).read() for f in ("paged_attention.cu", "paged_prefix.cu", "serving.h", "paged.cuh")}
    const = lambda f, n: re.search(r"%s = ([^;]+);" % n, src[f]).group(1)  # noqa: E731
    assert int(const("paged_attention.cu", "kSegmentTiles")) == T.EXTRA
    assert int(const("paged_prefix.cu", "kSnapTiles")) == T.SNAP
    assert int(const("paged_attention.cu", "kOwnPrefixRows")) == T.OWN_ROWS
    assert const("paged_attention.cu", "kOwnPrefixWork") == "1ll << 30"
    assert src["paged_attention.cu"].count("kCtas = D == 64 ? 3 : D == 128 ? 2 : 1;") == 2
    assert int(const("paged_attention.cu", "kBN")) == 64 and int(const("paged_attention.cu", "kFBN")) == 32
    assert int(const("paged_attention.cu", "kFRows")) == 16
    assert "paged_prefix_keys(int head_dim) { return head_dim == 256 ? 64 : 128; }" in src["serving.h"]
    assert "paged_prefix_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }" in src["serving.h"]
    assert "return kMax != 64 ? 1 : ts - 3;" in src["paged.cuh"]


@pytest.mark.parametrize("seed", range(120))
def test_work_list_with_the_kernels_constants(seed):
    """Every key tile once, partials apart and within the rows they are sized for, each where the join looks, with
    the extra tiles, chunks, tile sizes and CTAs that the kernels use."""
    r = random.Random(seed)
    d, form = r.choice([64, 128, 256]), r.choice(["list", "small", "f32", "prefix"])
    bn, most, ctas, snap, extra = {
        "list": (64, 64, T.SMS * T.CTAS[d], 0, T.EXTRA), "small": (64, 16, T.SMS * T.CTAS[d], 0, T.EXTRA),
        "f32": (32, 16, T.SMS * T.CTAS[d], 0, T.EXTRA),
        "prefix": (64 if d == 256 else 128, 128 if d == 256 else 256, T.SMS, T.SNAP, 0)}[form]
    hkv = r.choice([1, 2, 4, 8])
    span = r.choice([300, 4000, 30000])
    items = []
    for _ in range(r.choice([1, 3, 12, 60])):
        lo = 0 if form == "prefix" else r.choice([0, r.randint(0, span)])
        items.append((r.choice([0, 1, 4, 5, 16, 17, 32, 40, 64, 65, 200, 257, 700]), lo, lo + r.randint(0, span)))
    got, sp, total, chunk, extra = M.pieces(items, hkv, bn, most, ctas, snap, extra)
    taken, intervals, by = {}, [], {}
    for c, i, seg, kt, count, row, rows in got:
        assert count > 0 and 0 <= seg < hkv * sp[i][3] and kt + count <= sp[i][4]
        for x in range(kt, kt + count):
            assert (i, seg, x) not in taken
            taken[i, seg, x] = c
        intervals.append((row, row + rows))
        by[c, i, seg] = row
    assert len(taken) == sum(s[0] for s in sp)
    intervals.sort()
    assert all(a[1] <= b[0] for a, b in zip(intervals, intervals[1:]))
    assert not intervals or (intervals[0][0] >= 0 and intervals[-1][1] <= sum(s[1] for s in sp) + ctas * most)
    unit = base = 0
    for i, (_, part, pm, rt, nt) in enumerate(sp):
        units = M.padded(sp[i], most, chunk, extra)
        for seg in range(hkv * rt if nt else 0):
            u0 = unit + seg * units
            c0 = M.owner(u0, total, chunk, ctas)
            c1 = M.owner(u0 + (nt - 1) * M.weight(sp[i], most, extra), total, chunk, ctas)
            for c in range(c0, c1 + 1):
                assert by.pop((c, i, seg)) == c * most + base + seg * pm
        unit, base = unit + hkv * rt * units, base + part
    assert not by


def test_definition_is_the_oracles():
    """The definition used for the large cases against the serving operators' oracle."""
    for seed, groups in ((0, None), (1, ([0, 2, 4], [20, 37])), (2, ([0, 4], [50]))):
        st = C.Step(seed, torch.bfloat16, 6, 2, 64, 16, [1, 3, 0, 9], [40, 2, 60, 70], groups, extra_rows=2)
        for got, want in zip(T.want(st, "cpu", 0.2), st.want(0.2)):
            assert np.allclose(got, want, rtol=0, atol=1e-12)


LONG = ["prefix_128k", "prefix_128k_rows", "prefix_40k_d256", "own_60k", "f32_20k"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", [n for n in T.CASES if n not in LONG])
def test_many_tiles(name):
    api.lib()
    st = T.build(name)
    cache, batch, q, rows = st.cache(), st.batch(), st.q.cuda(), st.cu[-1]
    att = api.PagedAttention(cache, batch, st.hq)
    att.ws[256:].fill_(0xFF)  # NaN wherever a partial is read that no CTA wrote
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 5.0, device="cuda")
    att(q, out, lse=lse)
    assert att.status() == 0
    want, want_lse, mean = T.want(st, "cuda")
    bound, lse_bound = st.bounds(want, want_lse, mean)
    off = np.abs(out[:rows].double().cpu().numpy() - want)
    assert np.all(off <= bound), float((off / bound).max())
    assert np.all(np.abs(lse[:rows].double().cpu().numpy() - want_lse) <= lse_bound)
    assert torch.all(out[rows:] == 5.0) and torch.all(lse[rows:] == 5.0)
    first = out.clone()
    assert torch.equal(att(q, out), first)  # the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("name", LONG + ["long_d128"])
def test_long_contexts_closely(name):
    """Long contexts within bounds that count the additions in a row: a piece's keys, then the partials, where
    Step.bounds takes all keys; and f16's steps below its normal numbers, 2^-36 of the largest weight."""
    dt, hq, hkv, d = T.CASES[name][:4]
    st = T.build(name, seed=5)
    st.v_pages += 1.0
    q, rows = st.q.cuda(), st.cu[-1]
    att = api.PagedAttention(st.cache(), st.batch(), st.hq)
    out, lse = torch.zeros_like(q), torch.empty(q.shape[:2], device="cuda")
    att(q, out, lse=lse)
    assert att.status() == 0
    want, want_lse, mean = T.want(st, "cuda")
    fin = lambda t: np.nan_to_num(t.double().numpy(), nan=0.0)  # noqa: E731
    qn = np.linalg.norm(fin(st.q[:rows]), axis=-1).reshape(rows, hkv, -1)
    kn = np.linalg.norm(fin(st.k_pages), axis=-1).max(axis=(0, 2))
    x = (qn * kn[:, None]).reshape(rows, hq) * d ** -0.5
    chain = T.reached(name)[1] * 128 + T.SMS * 3
    dx = (d + 4) * C.F32 * x + 3 * 2.0 ** -22 + chain * C.F32
    f16 = dt == torch.bfloat16
    err = (2 * dx + (2.0 ** -11 if f16 else 0.0))[..., None] * mean
    err = err + (max(st.held) * 2.0 ** -36 * np.abs(fin(st.v_pages)).max() if f16 else 0.0)
    bound = C.half_step(dt) * (np.abs(want) + err) + err
    off = np.abs(out[:rows].double().cpu().numpy() - want)
    assert np.all(off <= bound), float((off / bound).max())
    off = np.abs(lse[:rows].double().cpu().numpy() - want_lse)
    assert np.all(off <= dx + 2 * C.F32 * np.abs(want_lse)), float((off / dx).max())
    first = out.clone()
    assert torch.equal(att(q, out), first)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["pieces_d128", "long_d256", "own_64", "f32_d128"])
def test_an_earlier_report_does_not_end_a_call(name):
    """The status word gathers reports; a timeout that an earlier call left there changes no later result."""
    st = T.build(name)
    cache, batch, q = st.cache(), st.batch(), st.q.cuda()
    att = api.PagedAttention(cache, batch, st.hq)
    want = att(q, torch.zeros_like(q))[:st.cu[-1]].clone()
    assert att.status() == 0
    att.ws[:4].view(torch.int32).fill_(1)  # as a wait that ran out would leave it
    att.ws[256:].fill_(0xFF)
    got = att(q, torch.zeros_like(q))[:st.cu[-1]]
    assert torch.equal(got, want) and att.status() == 5
    att.reset()
    assert att.status() == 0
