"""GPU parity of the operators around the prefill path (rotary positions, paged
append, paged attention) against their fp64 oracle, through the public binding."""

import ctypes

import numpy as np
import pytest
import torch

from dynamic_hierarchical_sparse_b200 import api, workloads as W
from oracle import dhsa_oracle as O, serving_oracle as S
from oracle.dhsa_oracle import as_f64
from tests import serving_cases as C

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LLAMA3 = W.RopeScaling("llama3", 8.0, 8192.0)
YARN = W.RopeScaling("yarn", 16.0, 4096.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    api.lib()


def _np(t):
    return as_f64(t.detach().cpu())


# ------------------------------------------------------------------- rope

ROPE_CASES = [
    # tokens, hq, hkv, d, rotary, interleaved, scaling, base, dtype
    (1, 32, 8, 128, 128, False, None, 10000.0, BF16),
    (5, 8, 8, 64, 64, True, LLAMA3, 500000.0, BF16),
    (33, 3, 1, 256, 64, False, YARN, 10000.0, BF16),
    (17, 6, 2, 128, 104, False, None, 10000.0, BF16),   # halves not on vector borders
    (17, 6, 2, 128, 90, True, None, 10000.0, BF16),     # odd number of pairs
    (9, 2, 2, 64, 2, False, None, 10000.0, BF16),
    (5000, 32, 8, 128, 128, False, LLAMA3, 500000.0, BF16),   # many heads a thread
    (3001, 9, 3, 256, 128, True, YARN, 10000.0, BF16),
    (4999, 13, 1, 64, 36, False, None, 10000.0, BF16),
    (1, 4, 4, 64, 64, False, None, 10000.0, F32),
    (2049, 8, 4, 256, 64, True, YARN, 10000.0, F32),
    (3000, 32, 8, 128, 128, False, LLAMA3, 500000.0, F32),
    (40, 5, 5, 128, 30, False, None, 10000.0, F32),
    (55, 7, 3, 128, 100, False, None, 10000.0, BF16),   # vectors of 4 bytes
    (55, 7, 3, 256, 36, True, None, 10000.0, F32),      # vectors of 8 bytes
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "t%d_d%d_r%d_%s" % (c[0], c[3], c[4], str(c[8])[6:]))
def test_rope(case):
    T, hq, hkv, d, rd, inter, scaling, base, dt = case
    g = torch.Generator().manual_seed(T + d)
    q, k = torch.randn(T, hq, d, generator=g).to(dt), torch.randn(T, hkv, d, generator=g).to(dt)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    if T > 4:
        pos[1], pos[2], pos[3] = 2 ** 31 - 1, -12345, -2 ** 31
    r = api.Rope(rd, base, inter, scaling)
    qo, ko = api.rope(q.cuda(), k.cuda(), pos.cuda(), r)
    f, a = S.rope_frequencies(rd, base, scaling)
    for got, x in ((qo, q), (ko, k)):
        want = S.rope(x, pos.numpy(), f, a, inter)
        bound = C.rope_bound(x, want, pos.numpy(), f, a, inter, dt)
        assert np.all(np.abs(_np(got) - want) <= bound)
        assert torch.equal(got[..., rd:].cpu(), x[..., rd:])


def test_rope_slices_in_place_and_one_alone():
    """Slices of one fused tensor, in place: the same bits as packed ones, and nothing else is touched."""
    g = torch.Generator().manual_seed(3)
    T, hq, hkv, d = 77, 4, 2, 128
    fused = torch.randn(T + 5, hq + 2 * hkv + 1, d, generator=g).to(BF16).cuda()
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).cuda()
    for rd in (128, 64, 50):
        r = api.Rope(rd)
        x = fused.clone()
        q, k = x[:T, :hq], x[:T, hq:hq + hkv]
        qo, ko = api.rope(q.contiguous(), k.contiguous(), pos, r)
        got = api.rope(q, k, pos, r, q, k)
        assert got[0] is q and torch.equal(q, qo) and torch.equal(k, ko)
        assert torch.equal(x[:, hq + hkv:], fused[:, hq + hkv:]) and torch.equal(x[T:], fused[T:])
        assert torch.equal(api.rope(fused[:T, :hq], None, pos, r)[0], qo)
        assert torch.equal(api.rope(None, fused[:T, hq:hq + hkv], pos, r)[1], ko)


def test_rope_nothing_to_do():
    q = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    qo, ko = api.rope(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), api.Rope(64))
    assert qo.shape == q.shape and ko is None


# ----------------------------------------------------------------- append

APPEND_CASES = [
    # dtype, hq, hkv, d, page, new, held, rotary, interleaved
    (BF16, 32, 8, 128, 16, [1] * 9, [1, 2, 16, 17, 33, 300, 15, 4000, 64], 128, False),
    (BF16, 8, 4, 256, 64, [1, 3, 0, 130], [1, 3, 77, 200], 256, False),
    (BF16, 6, 2, 64, 128, [5, 200, 1], [128, 200, 1000], 34, True),
    (BF16, 4, 1, 128, 32, [1000, 1, 2500], [1000, 31, 2600], 128, False),
    (BF16, 16, 16, 128, 16, [700, 900], [700, 1500], 128, True),
    (F32, 6, 2, 64, 32, [1, 40, 7], [33, 40, 70], 32, True),
    (F32, 4, 4, 256, 16, [900, 33], [950, 33], 256, False),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "%s_d%d_p%d" % (str(c[0])[6:], c[3], c[4]))
@pytest.mark.parametrize("given", [False, True], ids=["own_positions", "given_positions"])
def test_append(case, given):
    dt, hq, hkv, d, page, new, held, rd, inter = case
    st = C.Step(len(new) + d, dt, hq, hkv, d, page, new, held, extra_rows=3)
    g = torch.Generator().manual_seed(d)
    T = st.cu[-1]
    k, v = (torch.randn(T + 3, hkv, d, generator=g).to(dt) for _ in range(2))
    cache, batch = st.cache(), st.batch()
    k0, v0 = cache.k_pages.clone(), cache.v_pages.clone()
    r = api.Rope(rd, 10000.0, inter)
    at = np.concatenate([np.arange(h - n, h) for n, h in zip(new, held)])
    pos = torch.from_numpy(at * 3 + 5).to(torch.int32) if given else None
    qo = torch.full((T + 3, hq, d), 7.0, dtype=dt, device="cuda")
    ko = torch.full((T + 3, hkv, d), 7.0, dtype=dt, device="cuda")
    app = api.KvAppender(cache, batch, r)
    app(k.cuda(), v.cuda(), st.q.cuda(), qo, ko, None if pos is None else pos.cuda())
    assert app.status() == 0
    f, a = S.rope_frequencies(rd, 10000.0)
    p = at if pos is None else pos.numpy()
    for got, x in ((qo, st.q), (ko, k)):
        want = S.rope(x[:T], p, f, a, inter)
        assert np.all(np.abs(_np(got[:T]) - want) <= C.rope_bound(x[:T], want, p, f, a, inter, dt))
        assert torch.all(got[T:] == 7.0)  # rows behind the last sequence
    # K pages hold the very bits of k_out, V pages the converted v, and no other slot changed
    kp, vp = k0.clone(), v0.clone()
    for b in range(len(new)):
        for j in range(new[b]):
            s = held[b] - new[b] + j
            kp[st.table[b, s // page], :, s % page] = ko[st.cu[b] + j]
            vp[st.table[b, s // page], :, s % page] = v[st.cu[b] + j].cuda().to(vp.dtype)
    bits = torch.int16 if dt == BF16 else torch.int32
    assert torch.equal(cache.k_pages.view(bits), kp.view(bits))
    assert torch.equal(cache.v_pages.view(bits), vp.view(bits))


def test_append_without_rotation_and_by_slices():
    """No rotation: keys are stored as they are.  k, v as slices of one fused tensor, pages that lie apart."""
    st = C.Step(5, BF16, 4, 2, 128, 16, [3, 20], [40, 20], gap=64)
    T = st.cu[-1]
    qkv = torch.randn(T, 8, 128, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    cache = st.cache()
    api.append_kv(cache, st.batch(), qkv[:, 4:6], qkv[:, 6:], check=True)
    for b, n in enumerate(st.new):
        for j in range(n):
            s, t = st.held[b] - n + j, st.cu[b] + j
            assert torch.equal(cache.k_pages[st.table[b, s // 16], :, s % 16], qkv[t, 4:6])
            assert torch.equal(cache.v_pages[st.table[b, s // 16], :, s % 16], qkv[t, 6:].half())
    # rotated in place, in the fused tensor
    want = api.append_kv(st.cache(), st.batch(), qkv[:, 4:6], qkv[:, 6:], api.Rope(128), qkv[:, :4],
                         k_out=torch.empty(T, 2, 128, dtype=BF16, device="cuda"))
    x = qkv.clone()
    api.append_kv(st.cache(), st.batch(), x[:, 4:6], x[:, 6:], api.Rope(128), x[:, :4], x[:, :4], x[:, 4:6])
    assert torch.equal(x[:, :4], want[0]) and torch.equal(x[:, 4:6], want[1]) and torch.equal(x[:, 6:], qkv[:, 6:])


def test_append_reports_large_values_and_bad_tables():
    st = C.Step(6, BF16, 2, 1, 64, 16, [1, 1, 1], [5, 6, 40])
    cache, batch = st.cache(), st.batch()
    k = torch.ones(3, 1, 64, dtype=BF16, device="cuda")
    v = torch.ones(3, 1, 64, dtype=BF16, device="cuda")
    app = api.KvAppender(cache, batch)
    v[0, 0, 3], v[1, 0, 4], v[2, 0, 5] = 1e6, float("nan"), float("-inf")
    app(k, v)
    assert app.status() == 6
    at = lambda b, s: cache.v_pages[st.table[b, s // 16], 0, s % 16]  # noqa: E731
    assert at(0, 4)[3] == 65504 and torch.isnan(at(1, 5)[4]) and at(2, 39)[5] == -65504
    app(k, k)
    assert app.status() == 6  # reports gather ...
    app.reset()
    app(k, k)
    assert app.status() == 0  # ... until they are cleared
    # a page outside the cache, a length beyond the table, a negative length: reported, nothing stored
    for change in ("page", "long", "short"):
        bad = C.Step(6, BF16, 2, 1, 64, 16, [1, 1, 1], [5, 6, 40])
        cache, batch = bad.cache(), bad.batch()
        before = cache.k_pages.clone()
        if change == "page":
            batch.block_table[2, 2] = bad.pages
        else:
            batch.kv_lens[2] = 49 if change == "long" else -3
        app = api.KvAppender(cache, batch)
        app(k, k)
        assert app.status() == 6
        assert torch.equal(before[bad.table[2, 2]].view(torch.int16), cache.k_pages[bad.table[2, 2]].view(torch.int16))
        assert torch.all(cache.k_pages[bad.table[0, 0], 0, 4] == 1)


def test_append_padding_tokens_are_not_stored():
    """Positions below zero: no report, no page written, q and k rotated all the same."""
    st = C.Step(15, BF16, 4, 2, 128, 16, [3, 1, 2], [1, 0, 9])
    cache, batch = st.cache(), st.batch()
    k0 = cache.k_pages.clone()
    k, v = (torch.randn(6, 2, 128, generator=torch.Generator().manual_seed(i)).to(BF16).cuda() for i in range(2))
    app = api.KvAppender(cache, batch, api.Rope(128))
    qo, ko = app(k, v, st.q.cuda(), k_out=torch.empty_like(k))
    assert app.status() == 0
    pos = torch.tensor([-2, -1, 0, -1, 7, 8], dtype=torch.int32, device="cuda")
    want = api.rope(st.q.cuda(), k, pos, api.Rope(128))
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    k0[st.table[0, 0], :, 0], k0[st.table[2, 0], :, 7], k0[st.table[2, 0], :, 8] = ko[2], ko[4], ko[5]
    assert torch.equal(k0.view(torch.int16), cache.k_pages.view(torch.int16))


# -------------------------------------------------------------- attention

ATTEND_CASES = {
    # name: (dtype, hq, hkv, d, page, new, held, groups, values)
    "one_token": (BF16, 4, 1, 128, 16, [1], [1], None, "normal"),
    "lengths": (BF16, 8, 2, 128, 16, [1] * 10, [1, 2, 15, 16, 17, 63, 64, 65, 129, 1000], None, "normal"),
    "empty_rows": (BF16, 8, 2, 64, 32, [1, 0, 2, 1], [0, 50, 1, 70], None, "normal"),
    "ragged_new": (BF16, 6, 2, 128, 64, [3, 1, 17, 0, 40], [3, 90, 200, 5, 41], None, "peaks"),
    "d64_heads": (BF16, 24, 8, 64, 128, [1] * 5, [700, 3, 128, 129, 2000], None, "peaks"),
    "d256_group": (BF16, 8, 4, 256, 16, [1] * 6, [70, 65, 100, 200, 129, 300], ([0, 6], [64]), "peaks"),
    "d256_many_rows": (BF16, 16, 2, 256, 32, [5] * 4, [150, 130, 200, 160], ([0, 4], [120]), "normal"),
    "prefix_in_page": (BF16, 8, 2, 128, 16, [1] * 7, [102, 200, 103, 101, 164, 165, 166], ([0, 7], [101]), "peaks"),
    "prefix_long": (BF16, 8, 2, 128, 16, [1] * 6, [5001, 5100, 5020, 5333, 5007, 5064], ([0, 6], [5000]), "peaks"),
    "prefix_all": (BF16, 4, 4, 128, 32, [1, 1, 1], [96, 97, 96], ([0, 3], [96]), "normal"),
    "prefix_beyond": (BF16, 4, 2, 128, 16, [1, 2, 1], [200, 30, 0], ([0, 3], [100]), "normal"),
    "two_groups": (BF16, 8, 1, 128, 64, [1] * 7, [300, 280, 257, 500, 66, 70, 64], ([0, 4, 7], [256, 33]), "peaks"),
    "empty_group": (BF16, 4, 2, 64, 16, [1] * 3, [40, 50, 60], ([0, 0, 2, 3, 3], [77, 32, 0, 16]), "normal"),
    "prefix_rows": (BF16, 8, 2, 128, 16, [1] * 40, [600 + 7 * i for i in range(40)], ([0, 40], [600]), "peaks"),
    # many rows on one prefix: d 64 / 128 / 256, rows beyond one tile, a prefix that ends inside a tile, in a page
    "many_d64": (BF16, 16, 2, 64, 128, [1] * 30, [1300 + 11 * i for i in range(30)], ([0, 30], [1291]), "peaks"),
    "many_d128": (BF16, 32, 4, 128, 32, [2] * 21, [2600 + 7 * i for i in range(21)], ([0, 21], [2590]), "peaks"),
    "many_d256": (BF16, 8, 2, 256, 16, [3] * 25, [900 + 3 * i for i in range(25)], ([0, 25], [833]), "peaks"),
    "many_groups": (BF16, 8, 1, 128, 64, [1] * 41, [700 + i for i in range(41)],
                    ([0, 6, 6, 36, 41], [500, 9, 640, 1]), "peaks"),
    "many_short_rows": (BF16, 8, 2, 128, 16, [1] * 20, [300] * 5 + [20] * 5 + [0] * 5 + [129] * 5,
                        ([0, 20], [150]), "normal"),
    "many_drafted": (BF16, 12, 4, 128, 16, [6] * 16, [130 + i for i in range(16)], ([0, 16], [128]), "normal"),
    "drafted": (BF16, 32, 8, 128, 16, [5] * 5, [405, 431, 410, 500, 417], ([0, 5], [400]), "peaks"),
    "drafted_in_prefix": (BF16, 8, 2, 128, 16, [7] * 4, [205, 203, 220, 190], ([0, 4], [200]), "normal"),
    "heads_odd": (BF16, 21, 3, 128, 16, [1, 2, 3], [33, 77, 150], None, "normal"),
    "one_kv_head": (BF16, 40, 1, 64, 16, [1, 1], [900, 1000], ([0, 2], [890]), "peaks"),
    "f32": (F32, 8, 2, 64, 32, [1, 0, 3, 1, 1], [1, 4, 90, 500, 0], None, "peaks"),
    "f32_d128_group": (F32, 6, 2, 128, 16, [1] * 9, [300 + 5 * i for i in range(9)], ([0, 9], [290]), "peaks"),
    "f32_d256": (F32, 4, 4, 256, 64, [2, 2], [100, 1500], ([0, 1, 2], [0, 1000]), "normal"),
    "f32_prefix_beyond": (F32, 4, 2, 128, 16, [1, 2, 1], [200, 30, 0], ([0, 3], [101]), "normal"),
}


def _attend(st, scale=None, extra=0, gap_rows=False):
    cache, batch = st.cache(), st.batch()
    q = st.q.cuda()
    att = api.PagedAttention(cache, batch, st.hq)
    att.ws[256:].fill_(0xFF)  # NaN wherever a partial is read that no CTA wrote
    out = torch.full(q.shape, 5.0, dtype=st.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    att(q, out, scale, lse)
    assert att.status() == 0
    return out, lse


def _check(st, out, lse, scale=None):
    T = st.cu[-1]
    want, want_lse, mean = st.want(scale)
    bound, lse_bound = st.bounds(want, want_lse, mean, scale)
    off = np.abs(_np(out[:T]) - want)
    assert np.all(off <= bound), float((off / bound).max())
    got = _np(lse[:T])
    fin = np.isfinite(want_lse)
    assert np.array_equal(fin, np.isfinite(got)) and np.all(got[~fin] == -np.inf)
    assert np.all(np.abs(got[fin] - want_lse[fin]) <= lse_bound[fin])
    assert torch.all(out[T:] == 5.0) and torch.all(lse[T:] == 5.0)


@pytest.mark.parametrize("name", ATTEND_CASES)
def test_paged_attention(name):
    dt, hq, hkv, d, page, new, held, groups, values = ATTEND_CASES[name]
    st = C.Step(len(name), dt, hq, hkv, d, page, new, held, groups, extra_rows=2, values=values)
    _check(st, *_attend(st))


def _room(hq, hkv, d, rows):
    """Tokens of table room from which a group's prefix goes to the tensor-core kernel (2^30 of rows x Hkv x d x room)."""
    return -(-(1 << 30) // (rows * hkv * d)) + 128


GROUPED = [n for n, c in ATTEND_CASES.items()
           if c[0] == BF16 and c[7] is not None and
           max(sum(c[5][a:b]) for a, b in zip(c[7][0], c[7][0][1:])) * c[1] // c[2] > 32]


@pytest.mark.parametrize("name", GROUPED)
def test_paged_attention_with_room_for_long_prefixes(name):
    """The same batches with wide tables, whose prefixes go to the tensor-core kernel."""
    dt, hq, hkv, d, page, new, held, groups, values = ATTEND_CASES[name]
    rows = sum(new) * hq // hkv
    st = C.Step(len(name) + 1, dt, hq, hkv, d, page, new, held, groups, extra_rows=2, values=values,
                room=_room(hq, hkv, d, rows))
    a = _attend(st)
    _check(st, *a)
    for x, y in zip(a, _attend(st)):  # the same bits again
        assert torch.equal(x, y)


def test_long_prefix_reports_and_neighbours():
    """A page outside the cache in a long prefix: reported, read as zeros; the other group's rows as they were."""
    st = C.Step(31, BF16, 8, 1, 128, 16, [1] * 12, [150 + i for i in range(12)], ([0, 6, 12], [140, 150]),
                room=_room(8, 1, 128, 96))
    cache, batch, q = st.cache(), st.batch(), st.q.cuda()
    att = api.PagedAttention(cache, batch, 8)
    good = att(q, torch.empty_like(q)).clone()
    assert att.status() == 0
    for bad in (st.pages, -1, -2 ** 31, 2 ** 31 - 1):
        batch.block_table[0, 3] = bad
        out = att(q, torch.empty_like(q))
        assert att.status() == 6
        assert torch.equal(out[6:], good[6:]) and torch.isfinite(out).all()
        att.reset()
    batch.prefix_lens[0] = 10 ** 9
    att(q, torch.empty_like(q))
    assert att.status() == 6


@pytest.mark.parametrize("dt", [BF16, F32])
def test_paged_attention_scale_strides_and_page_gaps(dt):
    st = C.Step(4, dt, 8, 2, 128, 16, [2, 1, 3], [60, 200, 100], ([0, 3], [50]), gap=128, values="peaks")
    cache, batch = st.cache(), st.batch()
    fused = torch.zeros(st.cu[-1], 12, 128, dtype=dt, device="cuda")
    fused[:, 2:10] = st.q.cuda()
    out = torch.zeros(st.cu[-1], 9, 128, dtype=dt, device="cuda")
    got = api.PagedAttention(cache, batch, 8)(fused[:, 2:10], out[:, :8], scale=0.3)
    want, lse, mean = st.want(0.3)
    assert np.all(np.abs(_np(got) - want) <= st.bounds(want, lse, mean, 0.3)[0])
    assert torch.all(out[:, 8] == 0)


def test_paged_attention_one_shot_and_padding():
    st = C.Step(8, BF16, 4, 2, 64, 16, [1, 1], [20, 30], extra_rows=6)
    out = api.paged_attention(st.q.cuda(), st.cache(), st.batch(), check=True)
    want, lse, mean = st.want()
    assert np.all(np.abs(_np(out[:2]) - want) <= st.bounds(want, lse, mean)[0])
    assert torch.all(out[2:] == 0)


def test_paged_attention_nothing_to_do():
    st = C.Step(9, BF16, 4, 2, 64, 16, [0, 0], [20, 30])
    out = torch.full((3, 4, 64), 2.0, dtype=BF16, device="cuda")
    api.PagedAttention(st.cache(), st.batch(), 4)(torch.zeros_like(out), out)
    assert torch.all(out == 2.0)
    none = api.PagedBatch([0], torch.empty(0, dtype=torch.int32, device="cuda"),
                          torch.empty(0, 1, dtype=torch.int32, device="cuda"))
    api.PagedAttention(st.cache(), none, 4)(torch.zeros_like(out), out)
    assert torch.all(out == 2.0)


def test_paged_attention_same_bits_every_time():
    st = C.Step(10, BF16, 8, 2, 128, 16, [1] * 12, [900 + 31 * i for i in range(12)], ([0, 12], [896]), values="peaks")
    a, la = _attend(st)
    for _ in range(3):
        b, lb = _attend(st)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_paged_attention_extreme_logits(dt):
    """Infinite logits and NaN keys as in exact arithmetic on the row that sees them, nothing on the others."""
    st = C.Step(11, dt, 2, 1, 64, 16, [1, 1, 1], [40, 50, 60])
    kp = st.k_pages
    kp[st.table[0, 1], 0, 3] = float("nan")     # seen by sequence 0 alone
    kp[st.table[1, 2], 0, 5] = 3e38             # logits of +-infinity or NaN for sequence 1
    out, lse = _attend(st)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    want, want_lse, mean = st.want()
    bound, _ = st.bounds(want, want_lse, mean)
    # the bound counts the largest key; take it for the third sequence from its own keys
    kp[st.table[0, 1], 0, 3] = 0
    kp[st.table[1, 2], 0, 5] = 0
    bound, _ = st.bounds(want, want_lse, mean)
    assert np.all(np.abs(_np(out)[2] - want[2]) <= bound[2])


@pytest.mark.parametrize("bits", [0x7FFFFFFF, 0x7FC00000, 0x7F810000, -1, -0x7F0000])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_paged_attention_any_nan(dt, bits):
    """Every NaN, whatever its bits, in a query, key or value makes the rows that meet it NaN."""
    def nan(dtype):
        if dtype == F32:
            return torch.tensor([bits], dtype=torch.int32).view(F32)[0]
        t = torch.tensor([bits >> 16], dtype=torch.int16).view(BF16)[0]
        return t if dtype == BF16 else t.to(dtype)
    st = C.Step(31, dt, 8, 2, 64, 16, [1, 1, 2], [40, 33, 90])
    clean, _ = _attend(st)
    st.q[1, 3, 7] = nan(st.q.dtype)                                # a query head of sequence 1
    st.k_pages[st.table[0, 1], 1, 3, 9] = nan(st.k_pages.dtype)    # a key of sequence 0, heads 4 to 7
    st.v_pages[st.table[2, 2], 0, 5, 11] = nan(st.v_pages.dtype)   # a value of sequence 2, heads 0 to 3
    assert st.q[1, 3, 7].isnan() and st.k_pages[st.table[0, 1], 1, 3, 9].isnan()
    got, lse = _attend(st)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, 3] = hit[0, 4:] = hit[2:, :4, 11] = True
    assert torch.equal(torch.isnan(got), hit)
    assert torch.equal(torch.isnan(lse), (hit.all(-1)))
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_paged_attention_reports_bad_tables(dt):
    for change in ("page", "negative", "long", "short", "prefix"):
        st = C.Step(12, dt, 4, 2, 64, 16, [1, 2, 1], [30, 40, 70], ([0, 3], [16]))
        cache, batch = st.cache(), st.batch()
        att = api.PagedAttention(cache, batch, 4)
        if change in ("page", "negative"):
            batch.block_table[2, 2] = st.pages if change == "page" else -1
        elif change == "prefix":
            batch.prefix_lens[0] = -1
        else:
            batch.kv_lens[2] = 10 ** 6 if change == "long" else -4
            if change == "long":  # all of the row's pages exist, the length alone is wrong
                batch.block_table[2] = batch.block_table[2, 0]
        q = st.q.cuda()
        out = torch.empty_like(q)
        att(q, out)
        assert att.status() == 6, change
        if change != "prefix":
            want, lse, mean = st.want()
            bound = st.bounds(want, lse, mean)[0]
            assert np.all(np.abs(_np(out)[:3] - want[:3]) <= bound[:3]), change
        if change == "short":
            assert torch.all(out[3] == 0)
        att.reset()
        assert att.status() == 0


@pytest.mark.parametrize("heads", [(8, 2), (32, 2)], ids=["one_list", "own_prefix_list"])
def test_captured_steps_follow_the_device_arrays(heads):
    """A captured append and attention, replayed while lengths and tables go on: each step as an eager one."""
    hq, hkv = heads
    d, page, B, P = 128, 16, 3, 40
    g = torch.Generator().manual_seed(0)
    st = C.Step(13, BF16, hq, hkv, d, page, [1] * B, [P + 4, P + 1, P + 30], ([0, B], [P]),
                room=_room(hq, hkv, d, B * hq // hkv) if hq == 32 else 0)
    st.k_pages, st.v_pages = st.k_pages.nan_to_num(0.0), st.v_pages.nan_to_num(0.0)
    # room for more pages: every sequence gets two more
    extra = 2 * B
    grow = lambda t: torch.cat([t, torch.zeros(extra, *t.shape[1:], dtype=t.dtype)])  # noqa: E731
    n0 = st.pages
    st.k_pages, st.v_pages, st.pages = grow(st.k_pages), grow(st.v_pages), n0 + extra
    table = np.concatenate([st.table, np.full((B, 2), -7, np.int32)], axis=1)
    for b in range(B):
        used = -(-st.held[b] // page)
        table[b, used:used + 2] = [n0 + 2 * b, n0 + 2 * b + 1]
    st.table = table
    cache, batch = st.cache(), st.batch()
    eager_cache = st.cache()
    rope = api.Rope(d)
    app, att = api.KvAppender(cache, batch, rope), api.PagedAttention(cache, batch, hq)
    qkv = torch.zeros(B, hq + 2 * hkv, d, dtype=BF16, device="cuda")
    q_rot, out = torch.zeros(B, hq, d, dtype=BF16, device="cuda"), torch.zeros(B, hq, d, dtype=BF16, device="cuda")

    def step():
        app(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], qkv[:, :hq], q_rot)
        att(q_rot, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(20):
        qkv.copy_(torch.randn(B, hq + 2 * hkv, d, generator=g).to(BF16))
        batch.kv_lens.copy_(torch.tensor([h + i for h in st.held], dtype=torch.int32))
        graph.replay()
        got = out.clone()
        eb = st.batch()
        eb.kv_lens.copy_(batch.kv_lens)
        q2, _ = api.append_kv(eager_cache, eb, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], rope, qkv[:, :hq])
        want = api.paged_attention(q2, eager_cache, eb)
        assert torch.equal(got, want), i
    assert app.status() == 0 and att.status() == 0


def test_other_streams_and_overlapping_calls():
    """Two calls at once on two streams, each with its own workspace."""
    sts = [C.Step(20 + i, BF16, 8, 2, 128, 16, [1] * 6, [700 + 50 * j for j in range(6)], ([0, 6], [640]))
           for i in range(2)]
    alone = [_attend(st)[0] for st in sts]
    streams = [torch.cuda.Stream() for _ in sts]
    calls = [(api.PagedAttention(st.cache(), st.batch(), 8), st.q.cuda(), torch.zeros_like(st.q, device="cuda"))
             for st in sts]
    torch.cuda.synchronize()
    for _ in range(5):
        for (att, q, out), s in zip(calls, streams):
            att(q, out, stream=s)
    torch.cuda.synchronize()
    for a, (_, _, out) in zip(alone, calls):
        assert torch.equal(a, out)
    # one-shot calls on a stream are ordered against the current one
    s = torch.cuda.Stream()
    for st, a in zip(sts, alone):
        assert torch.equal(api.paged_attention(st.q.cuda(), st.cache(), st.batch(), stream=s), a)
        pos = torch.arange(6, dtype=torch.int32, device="cuda")
        r = api.Rope(128)
        assert torch.equal(api.rope(st.q.cuda(), None, pos, r, stream=s)[0], api.rope(st.q.cuda(), None, pos, r)[0])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_many_sequences_and_groups(dt):
    """More items than a CTA has threads: 700 sequences in 233 groups, some of them idle."""
    B = 700
    new = [1 if b % 7 else 0 for b in range(B)]
    held = [(b * 37) % 90 + (b % 5 != 0) for b in range(B)]
    ptr = list(range(0, B, 3)) + [B]
    prefix = [(g * 11) % 40 for g in range(len(ptr) - 1)]
    st = C.Step(40, dt, 4, 2, 64, 16, new, held, (ptr, prefix), values="peaks")
    _check(st, *_attend(st))


def test_overlapping_calls_with_long_prefixes():
    """Two calls at once on two streams through the tensor-core kernel, each as alone."""
    sts = [C.Step(50 + i, BF16, 32, 2, 128, 16, [1] * 5, [300 + j for j in range(5)], ([0, 5], [290]),
                  room=_room(32, 2, 128, 80)) for i in range(2)]
    alone = [_attend(st)[0] for st in sts]
    streams = [torch.cuda.Stream() for _ in sts]
    calls = [(api.PagedAttention(st.cache(), st.batch(), 32), st.q.cuda(), torch.zeros_like(st.q, device="cuda"))
             for st in sts]
    torch.cuda.synchronize()
    for _ in range(6):
        for (att, q, out), s in zip(calls, streams):
            att(q, out, stream=s)
    torch.cuda.synchronize()
    for a, (att, _, out) in zip(alone, calls):
        assert torch.equal(a[:5], out[:5]) and att.status() == 0


def test_append_makes_its_output_on_another_stream():
    st = C.Step(60, BF16, 4, 2, 128, 16, [2, 3], [20, 30])
    k = torch.randn(5, 2, 128, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    want = api.KvAppender(st.cache(), st.batch(), api.Rope(128))(k, k, st.q.cuda())[0]
    app, s, q = api.KvAppender(st.cache(), st.batch(), api.Rope(128)), torch.cuda.Stream(), st.q.cuda()
    torch.cuda.synchronize()
    got = app(k, k, q, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_far_pages():
    """Pages whose element offsets pass 32 bits."""
    page, hkv, d = 16, 1, 64
    stride = (1 << 31) + 64
    n = 3
    k = torch.empty((n - 1) * stride + hkv * page * d, dtype=BF16, device="cuda")
    v = torch.empty((n - 1) * stride + hkv * page * d, dtype=torch.float16, device="cuda")
    view = lambda t: t.as_strided((n, hkv, page, d), (stride, page * d, d, 1))  # noqa: E731
    cache = api.PagedCache(view(k), view(v))
    table = torch.tensor([[2, 1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([45], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(45, 4, d, generator=g).to(BF16).cuda()
    api.append_kv(cache, api.PagedBatch([0, 45], lens, table), qkv[:, 2:3], qkv[:, 3:], check=True)
    out = api.paged_attention(qkv[:, :2], cache, api.PagedBatch([0, 45], lens, table), check=True)
    small = api.PagedCache(cache.k_pages.contiguous(), cache.v_pages.contiguous())
    assert torch.equal(out, api.paged_attention(qkv[:, :2], small, api.PagedBatch([0, 45], lens, table)))
    want, _ = S.paged_attention(qkv[:, :2].cpu(), small.k_pages.cpu(), small.v_pages.cpu(), [0, 45], [45], [[2, 1, 0]])
    assert np.abs(_np(out) - want).max() < 2e-2


def test_binding_refusals():
    st = C.Step(14, BF16, 4, 2, 64, 16, [1, 1], [20, 30])
    cache, batch, q = st.cache(), st.batch(), st.q.cuda()
    att = api.PagedAttention(cache, batch, 4)
    with pytest.raises(TypeError):
        att(q.float(), torch.empty_like(q))
    for bad in (q[:1], q[:, :3], q.transpose(0, 1).contiguous().transpose(0, 1), q.cpu()):
        with pytest.raises(ValueError):
            att(bad, torch.empty_like(q))
    with pytest.raises(ValueError):
        att(q, torch.empty_like(q), lse=torch.empty(2, 4, dtype=torch.float64, device="cuda"))
    with pytest.raises(api.DhsaError):
        att(q, q)
    with pytest.raises(api.DhsaError):
        api.PagedAttention(cache, batch, 3)
    with pytest.raises(TypeError):
        api.PagedCache(cache.k_pages, cache.k_pages)
    with pytest.raises(ValueError):
        api.PagedCache(cache.k_pages.transpose(1, 2), cache.v_pages.transpose(1, 2))
    with pytest.raises(ValueError):
        api.KvAppender(cache, batch, api.Rope(64))(q[:, :2], q[:, 2:], q_out=torch.empty_like(q))
    with pytest.raises(api.DhsaError):
        api.KvAppender(cache, batch)(q[:, :2], q[:, 2:], q)  # q needs a rotation
    with pytest.raises(ValueError):
        api.rope(q, None, torch.zeros(3, dtype=torch.int32, device="cuda"), api.Rope(64))
    with pytest.raises(ValueError):
        api.PagedBatch([0, 1, 2], batch.kv_lens, batch.block_table, [0, 2])
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError):
            att(q.to("cuda:1"), torch.empty_like(q))


# ------------------------------------------------ the operators in a row


def test_prefill_then_answers_of_a_shared_prompt():
    """As used: a prompt's q, k, v are rotated and its keys and values stored in
    one call; the rotated q and k go through the plan and the sparse attention;
    then four answers grow over the shared pages, one token at a time."""
    inp = W.random_problem(30, [400], 8, 2, 128, "bf16", 30, 90, W.Budget.topk(10 ** 6))
    P, page, hq, hkv, d, B = 400, 16, 8, 2, 128, 4
    dev = torch.device("cuda")
    rope = api.Rope(d, 500000.0, scaling=LLAMA3)
    cache = api.PagedCache.empty(25 + B, page, hkv, d, BF16)
    prompt = torch.arange(25, dtype=torch.int32, device=dev)[None]
    q, k, v = inp.q.to(dev), inp.k.to(dev), inp.v.to(dev)
    q_rot, k_rot = api.append_kv(cache, api.PagedBatch([0, P], torch.tensor([P], dtype=torch.int32, device=dev), prompt),
                                 k, v, rope, q, k_out=torch.empty_like(k), check=True)
    pos = torch.arange(P, dtype=torch.int32, device=dev)
    qr, kr = api.rope(q, k, pos, rope)
    assert torch.equal(qr, q_rot) and torch.equal(kr, k_rot)
    prob = api.Problem.from_inputs(inp, dev)
    out = api.attention(q_rot, k_rot, v, prob, api.plan(q_rot, k_rot, prob, inp.budget, check=True), check=True)
    # every chunk kept: the prompt's own paged attention, all tokens at once, is the same function
    paged = api.paged_attention(q_rot, cache, api.PagedBatch([0, P], torch.tensor([P], dtype=torch.int32, device=dev),
                                                             prompt), check=True)
    f, a = S.rope_frequencies(d, 500000.0, LLAMA3)
    want = O.attention_gather(q_rot.cpu(), k_rot.cpu(), inp.v, inp.chunk_bounds,
                              *[np.asarray(x) for x in _all_chunks(inp, hq)])
    assert np.abs(_np(out) - want).max() <= 2e-2 and np.abs(_np(paged) - want).max() <= 2e-2
    table = torch.cat([prompt.expand(B, -1), torch.arange(25, 25 + B, dtype=torch.int32, device=dev)[:, None]], 1)
    table = table.contiguous()
    lens = torch.full((B,), P, dtype=torch.int32, device=dev)
    batch = api.PagedBatch(list(range(B + 1)), lens, table, [0, B], torch.tensor([P], dtype=torch.int32, device=dev))
    app, att = api.KvAppender(cache, batch, rope), api.PagedAttention(cache, batch, hq)
    g = torch.Generator().manual_seed(5)
    keys, vals = [k_rot.cpu()[None].expand(B, -1, -1, -1)], [inp.v[None].expand(B, -1, -1, -1)]
    for step in range(7):
        qkv = torch.randn(B, hq + 2 * hkv, d, generator=g).to(BF16)
        x = qkv.to(dev)
        lens += 1
        q_new, _ = app(x[:, hq:hq + hkv], x[:, hq + hkv:], x[:, :hq])
        got = att(q_new, torch.empty_like(q_new))
        at = np.full(B, P + step)
        qw = S.rope(qkv[:, :hq], at, f, a)
        keys.append(torch.from_numpy(S.rope(qkv[:, hq:hq + hkv], at, f, a))[:, None].to(BF16))
        vals.append(qkv[:, None, hq + hkv:])
        kk, vv = as_f64(torch.cat(keys, 1)), as_f64(torch.cat(vals, 1))
        s = np.einsum("bgrd,bsgd->bgrs", as_f64(torch.from_numpy(qw).to(BF16)).reshape(B, hkv, -1, d), kk) / d ** 0.5
        e = np.exp(s - s.max(-1, keepdims=True))
        want = np.einsum("bgrs,bsgd->bgrd", e / e.sum(-1, keepdims=True), vv).reshape(B, hq, d)
        assert np.abs(_np(got) - want).max() <= 2e-2
    assert app.status() == 0 and att.status() == 0


def _all_chunks(inp, hq):
    n = inp.num_chunks
    row_ptr, col = [0], []
    for _ in range(hq):
        for i in range(n):
            col += list(range(i + 1))
            row_ptr.append(len(col))
    return row_ptr, col
