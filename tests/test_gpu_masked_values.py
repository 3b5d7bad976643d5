"""Values that are not finite (or close to the largest fp32 number): where a row does
not see them they change nothing, where it does the result is that of plain
arithmetic, row by row, as the 64-bit oracle has it."""

import numpy as np
import pytest
import torch

from dynamic_hierarchical_sparse_b200 import api
from oracle import serving_oracle as S
from tests import serving_cases as C

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def _room(st_args):
    dt, hq, hkv, d, page, new = st_args[:6]
    return -(-(1 << 30) // (sum(new) * hq // hkv * hkv * d)) + 128


def _run(st):
    cache, batch, q = st.cache(), st.batch(), st.q.cuda()
    att = api.PagedAttention(cache, batch, st.hq)
    att.ws[256:].fill_(0xFF)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    att(q, out, lse=lse)
    assert att.status() == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _same_kind(got, want):
    """NaN where NaN is due, the same infinity where one is."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    odd = np.isinf(want)
    assert np.array_equal(np.isinf(got), odd) and np.array_equal(got[odd], want[odd])
    return np.isfinite(want)


def _check(st, clean, wild=()):
    """The result against the oracle on these inputs; bounds from the same batch with finite ones (`clean`).
    wild: rows whose finite inputs are so large that only the kind of their results is checked."""
    got, got_lse = _run(st)
    with np.errstate(all="ignore"):
        want, want_lse, _ = st.want()
    c_out, c_lse, mean = clean.want()
    bound, lse_bound = clean.bounds(c_out, c_lse, mean)
    # the weighted mean of |v| of these rows may differ from the clean batch's: the largest value stands for it
    top = np.abs(np.nan_to_num(clean.v_pages.double().numpy(), nan=0.0)).max()
    bound = bound + (2.0 ** -8 if st.dtype == BF16 else 2.0 ** -18) * top
    calm = np.ones(want.shape[0], dtype=bool)
    calm[list(wild)] = False
    fin = _same_kind(got, want) & calm[:, None, None]
    assert fin.any() and np.all(np.abs(got[fin] - want[fin]) <= bound[fin])
    keep = np.isfinite(want_lse) & calm[:, None]
    assert np.array_equal(np.isnan(got_lse), np.isnan(want_lse))
    assert np.all(np.abs(got_lse[keep] - want_lse[keep]) <= lse_bound[keep])
    return got


def _slot(st, b, s):
    """(page, slot) of key s of sequence b."""
    if st.groups is not None:
        g = int(np.searchsorted(st.groups[0], b, side="right") - 1)
        if s < st.groups[1][g]:
            b = st.groups[0][g]
    return int(st.table[b, s // st.page]), s % st.page


DRAFTED = {
    # name: (dtype, hq, hkv, d, page, new, held, groups)
    "rows_16": (BF16, 8, 2, 128, 16, [4, 3], [200, 130], None),
    "rows_4": (BF16, 4, 2, 64, 32, [2, 2], [75, 300], None),
    "rows_32": (BF16, 16, 2, 128, 16, [4, 3], [200, 130], None),
    "rows_64": (BF16, 16, 2, 64, 16, [8, 7], [190, 700], None),
    "rows_64_d256": (BF16, 16, 2, 256, 64, [8, 7], [190, 700], None),
    "next_part": (BF16, 8, 2, 128, 16, [150, 40], [400, 41], None),
    "f32": (F32, 8, 2, 128, 16, [4, 3], [200, 130], None),
    "f32_rows": (F32, 16, 2, 64, 32, [8, 30], [190, 700], None),
    "f32_d256": (F32, 8, 2, 256, 16, [3, 2], [90, 333], None),
}


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("name", DRAFTED)
def test_values_of_later_tokens_stay_with_them(name, value):
    """A value that is not finite in the slot of a drafted token: its row and the later ones have it, earlier ones not."""
    args = DRAFTED[name]
    clean, st = C.Step(7, *args), C.Step(7, *args)
    for b in range(2):
        n, held = st.new[b], st.held[b]
        for j in (n - 1, n // 2):
            page, slot = _slot(st, b, held - n + j)
            st.v_pages[page, 0, slot, 3 + 20 * j % 32] = value
            st.v_pages[page, 1, slot, ::9] = -value
    got = _check(st, clean)
    first = min(st.new[0] - 1, st.new[0] // 2)
    assert np.isfinite(got[:first]).all() and not np.isfinite(got[first:st.new[0]]).all(-1).any()


@pytest.mark.parametrize("name", ["rows_16", "rows_64", "f32_rows"])
def test_both_infinities_and_several_tokens(name):
    args = DRAFTED[name]
    clean, st = C.Step(8, *args), C.Step(8, *args)
    for j, value in enumerate((INF, -INF, NAN)):
        page, slot = _slot(st, 1, st.held[1] - 3 + j)
        st.v_pages[page, :, slot, 5 * j] = value
        st.v_pages[page, :, slot, 40] = value if j < 2 else 1.0
    _check(st, clean)


PREFIX = {
    # sequences that hold less than the group's prefix, and drafted tokens inside it; table room for the kernel of long prefixes
    "apart_d128": (BF16, 8, 2, 128, 16, [1] * 14, [700] * 8 + [300, 350, 30, 0, 513, 129], ([0, 14], [690])),
    "wide_d128": (BF16, 32, 2, 128, 32, [1] * 14, [700] * 8 + [300, 350, 30, 0, 513, 129], ([0, 14], [690])),
    "apart_d64": (BF16, 16, 2, 64, 16, [1] * 10, [500] * 7 + [257, 128, 60], ([0, 10], [450])),
    "wide_d64": (BF16, 16, 1, 64, 128, [2] * 10, [500] * 7 + [257, 128, 60], ([0, 10], [450])),
    "d256": (BF16, 8, 1, 256, 16, [1] * 10, [500] * 7 + [257, 128, 60], ([0, 10], [450])),
    "drafted": (BF16, 16, 2, 128, 16, [7] * 6, [305, 303, 320, 290, 301, 400], ([0, 6], [300])),
}


@pytest.mark.parametrize("long", [False, True], ids=["one_list", "long_prefix_kernel"])
@pytest.mark.parametrize("name", PREFIX)
def test_prefix_values_behind_a_sequences_end(name, long):
    """Prefix values that are not finite, behind the end of some of the group's sequences: those do not have them."""
    args = PREFIX[name]
    kw = dict(room=_room(args)) if long else {}
    clean, st = C.Step(9, *args, **kw), C.Step(9, *args, **kw)
    n = st.groups[1][0]
    for i, s in enumerate((n - 1, n - 2, n // 2 + 60)):
        page, slot = _slot(st, 0, s)
        st.v_pages[page, 0, slot, 7 * i:7 * i + 2] = (NAN, INF, -INF)[i]
        st.v_pages[page, -1, slot, st.d - 1 - 2 * i] = (INF, NAN, -INF)[i]
    got = _check(st, clean)
    assert np.isfinite(got).any() and not np.isfinite(got).all()


def test_short_prefix_rows_in_fp32():
    args = (F32, 8, 2, 128, 16, [1] * 9, [300] * 5 + [100, 30, 0, 222], ([0, 9], [290]))
    clean, st = C.Step(10, *args), C.Step(10, *args)
    for i, s in enumerate((289, 288, 200)):
        page, slot = _slot(st, 0, s)
        st.v_pages[page, i % 2, slot, 4 * i] = (NAN, INF, -INF)[i]
    _check(st, clean)


@pytest.mark.parametrize("what", ["key", "query"])
@pytest.mark.parametrize("dt,d", [(BF16, 64), (BF16, 256), (F32, 64), (F32, 128), (F32, 256)])
def test_infinite_logits(dt, d, what):
    """Logits of -infinity have no weight, +infinity makes the row NaN; the others as without."""
    args = (dt, 4, 1, d, 16, [1, 1, 1], [40, 500, 60], None)
    clean, st = C.Step(11, *args), C.Step(11, *args)
    for s in (clean, st):
        s.q[:, :, 0] = s.q[:, :, 0].abs() + 0.5  # the number that meets the infinity: its sign is the logit's
        s.q[1, 1::2, 0] *= -1
    if what == "key":
        page, slot = _slot(st, 1, 300)
        st.k_pages[page, 0, slot, 0] = -INF  # heads 0 and 2: weight 0; heads 1 and 3: +infinity
        with np.errstate(all="ignore"):
            want = st.want()[0]
        assert np.isfinite(want[1, ::2]).all() and np.isnan(want[1, 1::2]).all()
    else:
        st.q[1, 2, 5] = INF
    _check(st, clean)


def test_every_logit_minus_infinity():
    for dt in (BF16, F32):
        args = (dt, 2, 1, 64, 16, [1, 1], [30, 3], None)
        clean, st = C.Step(12, *args), C.Step(12, *args)
        st.q[1, :, 0] = 1.0
        for s in range(3):
            page, slot = _slot(st, 1, s)
            st.k_pages[page, 0, slot, 0] = -INF
        got, lse = _run(st)
        want, _, mean = clean.want()
        bound = clean.bounds(want, _, mean)[0]
        assert np.isnan(got[1]).all() and np.all(lse[1] == -INF)  # no weight at all: a mean of nothing
        assert np.all(np.abs(got - want)[0] <= bound[0])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_numbers_next_to_the_largest(d):
    """fp32 numbers that would round to infinity in fewer bits are numbers like others."""
    big = torch.finfo(F32).max
    args = (F32, 4, 2, d, 16, [1, 2, 1], [40, 500, 60], None)
    clean, st = C.Step(13, *args), C.Step(13, *args)
    # keys: against a query number of 0 nothing, against a tiny one a plain logit
    for s in (clean, st):
        s.q[1, :, 0] = 0.0
        s.q[2, :, 0] = 2.0 ** -127
    page, slot = _slot(st, 1, 250)
    st.k_pages[page, :, slot, 0] = torch.tensor([big, -big])
    got = _check(st, clean)
    assert np.isfinite(got).all()
    # a value: the row's output is that large (or more than the clean bound knows of), and finite where its weight allows
    page, slot = _slot(st, 0, 17)
    st.v_pages[page, 0, slot, 9] = big
    got = _check(st, clean, wild=[0])
    with np.errstate(all="ignore"):
        want = st.want()[0]
    assert np.allclose(got[0], want[0], rtol=1e-4, atol=1e-4)


def test_finite_batches_are_left_alone():
    """Rows that see part of a tile, all finite: the same bits as when the unseen slots hold something else."""
    for name in ("rows_16", "rows_64", "next_part"):
        a, b = C.Step(14, *DRAFTED[name]), C.Step(14, *DRAFTED[name])
        page, slot = _slot(b, 0, b.held[0] - 1)
        b.v_pages[page, :, slot] = 3.0
        x, y = _run(a)[0], _run(b)[0]
        assert np.array_equal(x[:a.new[0] - 1], y[:a.new[0] - 1])
