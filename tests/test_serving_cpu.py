"""CPU checks of the operators around the prefill path: the rotation's table,
refusals on the host (no kernel runs), and pins of their oracle."""

import ctypes
import math

import numpy as np
import pytest
import torch

from dynamic_hierarchical_sparse_b200 import api, build, workloads as W
from oracle import serving_oracle as S

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# ------------------------------------------------------------ oracle pins


def test_oracle_rope_is_relative():
    """q rotated at p + s and k at s have a product that depends on p alone."""
    g = np.random.default_rng(0)
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    f, _ = S.rope_frequencies(16, 10000.0)
    for inter in (False, True):
        want = np.sum(S.rope(q, [7], f, interleaved=inter) * S.rope(k, [0], f, interleaved=inter))
        for s in (1, 100, 12345):
            got = np.sum(S.rope(q, [7 + s], f, interleaved=inter) * S.rope(k, [s], f, interleaved=inter))
            assert abs(got - want) < 1e-9


def test_oracle_rope_by_hand():
    # one pair of frequency 1 at position 1: a plain turn by one radian; the third and fourth number stay
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    c, s = math.cos(1.0), math.sin(1.0)
    assert np.allclose(S.rope(x, [1], [1.0]), [[[c - 2 * s, 2 * c + s, 3, 4]]])
    # two pairs: halves (1,3) (2,4), interleaved (1,2) (3,4)
    y = S.rope(x, [1], [1.0, 0.0])
    assert np.allclose(y, [[[c - 3 * s, 2, 3 * c + s, 4]]])
    assert np.allclose(S.rope(x, [1], [1.0, 0.0], interleaved=True), [[[c - 2 * s, 2 * c + s, 3, 4]]])


def test_oracle_scalings_by_hand():
    f0, _ = S.rope_frequencies(8, 10000.0)
    assert np.allclose(f0, [1, 0.1, 0.01, 0.001])
    assert np.allclose(S.rope_frequencies(8, 10000.0, W.RopeScaling("linear", 4))[0], f0 / 4)
    # 1000 tokens make 159, 15.9, 1.59 and 0.159 turns: above 4 kept, below 1 stretched, 1.59 mixed
    f, a = S.rope_frequencies(8, 10000.0, W.RopeScaling("llama3", 8, 1000.0, 1.0, 4.0))
    mix = (10 / (2 * math.pi) - 1) / 3
    assert a == 1.0 and np.allclose(f, [1, 0.1, 0.01 * mix + 0.01 / 8 * (1 - mix), 0.001 / 8])
    f, a = S.rope_frequencies(8, 10000.0, W.RopeScaling("yarn", 16, 1000.0, beta_fast=20.0, beta_slow=1.0))
    # pair indexes 8 ln(1000 / (2 pi b)) / (2 ln 10^4): 0.9 for 20 turns, 2.2 for one, so 0 and 3
    want = [f0[i] / 16 * (i / 3) + f0[i] * (1 - i / 3) for i in range(4)]
    assert abs(a - (0.1 * math.log(16) + 1)) < 1e-15 and np.allclose(f, want)


def test_oracle_paged_attention_is_dense_attention():
    """Pages in any order, with and without a shared prefix, against torch's attention in fp64."""
    g = np.random.default_rng(1)
    hkv, r, d, page = 2, 2, 8, 4
    kp, vp = g.standard_normal((9, hkv, page, d)), g.standard_normal((9, hkv, page, d))
    table = [[3, 1, 7], [3, 0, 5]]
    cu, lens = [0, 2, 3], [10, 6]
    q = g.standard_normal((3, hkv * r, d))
    out, lse = S.paged_attention(q, kp, vp, cu, lens, table, [0, 2], [4])
    assert np.allclose(out, S.paged_attention(q, kp, vp, cu, lens, table)[0])
    for b in range(2):
        n, L = cu[b + 1] - cu[b], lens[b]
        k = np.concatenate([kp[p] for p in table[b]], axis=1)[:, :L].repeat(r, axis=0)
        v = np.concatenate([vp[p] for p in table[b]], axis=1)[:, :L].repeat(r, axis=0)
        mask = torch.arange(L)[None] <= torch.arange(L - n, L)[:, None]
        qq = torch.from_numpy(q[cu[b]:cu[b + 1]]).transpose(0, 1)
        want = torch.nn.functional.scaled_dot_product_attention(qq, torch.from_numpy(k), torch.from_numpy(v),
                                                                attn_mask=mask)
        assert np.allclose(out[cu[b]:cu[b + 1]], want.transpose(0, 1).numpy(), atol=1e-12)
        x = (qq @ torch.from_numpy(k).transpose(1, 2) / math.sqrt(d)).masked_fill(~mask, -math.inf)
        assert np.allclose(lse[cu[b]:cu[b + 1]], x.logsumexp(-1).transpose(0, 1).numpy(), atol=1e-12)


def test_oracle_planted_slips_show():
    """A prefix that is read through the wrong row, or a mask that is off by one, changes the oracle's result."""
    g = np.random.default_rng(2)
    kp, vp = g.standard_normal((6, 1, 4, 8)), g.standard_normal((6, 1, 4, 8))
    q = g.standard_normal((2, 1, 8))
    good, _ = S.paged_attention(q, kp, vp, [0, 1, 2], [7, 6], [[0, 1], [2, 3]], [0, 2], [4])
    own, _ = S.paged_attention(q, kp, vp, [0, 1, 2], [7, 6], [[0, 1], [2, 3]])
    late, _ = S.paged_attention(q, kp, vp, [0, 1, 2], [8, 6], [[0, 1], [2, 3]], [0, 2], [4])
    assert np.allclose(good[0], own[0]) and not np.allclose(good[1], own[1])
    assert not np.allclose(good[0], late[0])


# ------------------------------------------------------- rotation's table

SCALINGS = [None, W.RopeScaling("linear", 4.0), W.RopeScaling("llama3", 8.0, 8192.0),
            W.RopeScaling("yarn", 16.0, 4096.0), W.RopeScaling("yarn", 1.0, 4096.0)]


@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: "none" if s is None else s.kind)
@pytest.mark.parametrize("rotary,base", [(2, 10000.0), (64, 10000.0), (104, 500000.0), (128, 500000.0), (256, 10000.0)])
def test_rope_table_matches_the_oracle(rotary, base, scaling):
    r = api.Rope(rotary, base, True, scaling)
    f, a = S.rope_frequencies(rotary, base, scaling)
    assert r.c.rotary_dim == rotary and r.c.interleaved == 1 and abs(r.c.factor - a) <= 2.0 ** -24 * a
    turns = np.array([int(x) for x in r.c.turns[:rotary // 2]], dtype=object)
    for p in (1, 77, 1000003, -5):
        got = np.array([(int(t) * p % 2 ** 64) / 2.0 ** 64 for t in turns])
        off = got - np.array(p * f / (2 * math.pi))
        # fp64: the frequency is off by a few 2^-53 of itself, and so is p times it
        assert np.all(np.abs(off - np.round(off)) <= 16 * 2.0 ** -53 * abs(p))
    assert all(int(t) == 0 for t in r.c.turns[rotary // 2:])


def test_rope_table_from_frequencies():
    r = api.Rope(8, inv_freq=[1.0, -0.5, 7.0, 0.0], factor=1.25)
    want = [(x / (2 * math.pi)) % 1.0 for x in (1.0, -0.5, 7.0, 0.0)]
    assert np.allclose([int(t) / 2.0 ** 64 for t in r.c.turns[:4]], want, atol=1e-15) and r.c.factor == 1.25
    with pytest.raises(ValueError):
        api.Rope(8, inv_freq=[1.0])
    for bad in ([math.nan, 0, 0, 0], [math.inf, 0, 0, 0]):
        with pytest.raises(api.DhsaError):
            api.Rope(8, inv_freq=bad)


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(base=1.0),
                                dict(base=math.nan), dict(scaling=W.RopeScaling("linear", 0.5)),
                                dict(scaling=W.RopeScaling("llama3", 8.0, 0.0)),
                                dict(scaling=W.RopeScaling("llama3", 8.0, 8192.0, 4.0, 4.0)),
                                dict(scaling=W.RopeScaling("yarn", 8.0, 8192.0, beta_fast=1.0, beta_slow=2.0)),
                                dict(scaling=W.RopeScaling("yarn", math.inf, 8192.0))])
def test_rope_table_refusals(kw):
    with pytest.raises(api.DhsaError) as e:
        api.Rope(**dict(dict(rotary_dim=64), **kw))
    assert e.value.code == INVALID


def test_unknown_scaling_is_refused():
    with pytest.raises(ValueError):
        api.Rope(64, scaling=W.RopeScaling("other", 2.0))


# --------------------------------------------------------------- refusals
# Addresses are made up: every call below is refused before anything is launched.

A = 1 << 20


def _tok(data=A, stride=0):
    return api._Tokens(data, stride)


NONE = api._Tokens(None, 0)


def _rope_call(**kw):
    r = api.Rope(kw.pop("rotary", 64))
    v = dict(dtype=0, d=128, T=10, pos=A, q=_tok(A), hq=4, qo=_tok(2 * A), k=_tok(3 * A), hk=2, ko=_tok(4 * A))
    v.update(kw)
    return api.lib().dhsa_rope(ctypes.byref(r.c), v["dtype"], v["d"], v["T"], v["pos"], v["q"], v["hq"], v["qo"],
                               v["k"], v["hk"], v["ko"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(d=64, rotary=128), INVALID),
    (dict(T=-1), INVALID), (dict(pos=None), INVALID), (dict(hq=0), INVALID), (dict(hk=-2), INVALID),
    (dict(hq=70000), UNSUPPORTED), (dict(qo=NONE), INVALID), (dict(ko=NONE), INVALID), (dict(q=NONE), INVALID),
    (dict(q=_tok(A + 8)), INVALID), (dict(q=_tok(A, 511)), INVALID), (dict(q=_tok(A, 516)), INVALID),
    (dict(q=_tok(A, -1024)), INVALID), (dict(qo=_tok(A + 1024)), INVALID), (dict(qo=_tok(A, 1024)), INVALID),
    (dict(ko=_tok(2 * A)), INVALID), (dict(qo=_tok(3 * A)), INVALID), (dict(ko=_tok(A + 16)), INVALID),
])
def test_rope_refusals(kw, code):
    assert _rope_call(**kw) == code


def test_rope_accepts_nothing_to_do():
    assert _rope_call(T=0, pos=None) == OK
    assert _rope_call(q=NONE, qo=NONE, k=NONE, ko=NONE) == OK
    # two slices of one fused tensor, each rotated in place, do not overlap
    fused = dict(q=_tok(A, 768), qo=_tok(A, 768), k=_tok(A + 4 * 128 * 2, 768), ko=_tok(A + 4 * 128 * 2, 768))
    assert _rope_call(T=0, **fused) == OK


class _Step:
    """A cache and batch with made-up device addresses and real host mirrors."""

    def __init__(self, **kw):
        v = dict(dtype=0, hkv=2, d=128, page=16, pages=50, stride=2 * 16 * 128, kp=A, vp=2 * A, cu=[0, 1, 4],
                 groups=None, max_pages=10, table_stride=10, table=A, lens=A, d_cu=A, d_groups=A, prefix=A, seqs=None)
        v.update(kw)
        self.h_cu = np.asarray(v["cu"], dtype=np.int32)
        self.h_g = None if v["groups"] is None else np.asarray(v["groups"], dtype=np.int32)
        self.cache = api._PagedCache(v["dtype"], v["hkv"], v["d"], v["page"], v["pages"], v["stride"], v["kp"], v["vp"])
        n = len(self.h_cu) - 1 if v["seqs"] is None else v["seqs"]
        self.batch = api._PagedBatch(n, v["max_pages"], v["table_stride"],
                                     0 if self.h_g is None else len(self.h_g) - 1, v["d_cu"], v["lens"], v["table"],
                                     v["d_groups"], v["prefix"], self.h_cu.ctypes.data,
                                     None if self.h_g is None else self.h_g.ctypes.data)

    def size(self, hq=4):
        n = ctypes.c_size_t(0)
        code = api.lib().dhsa_paged_attention_workspace_size(ctypes.byref(self.cache), ctypes.byref(self.batch), hq,
                                                             ctypes.byref(n))
        return code, n.value

    def attend(self, q=_tok(4 * A), hq=4, out=_tok(8 * A), ws=16 * A, nbytes=None):
        nbytes = self.size(hq)[1] if nbytes is None else nbytes
        return api.lib().dhsa_paged_attention(ctypes.byref(self.cache), ctypes.byref(self.batch), q, hq, 0.0, out,
                                              None, ws, nbytes, None)

    def append(self, k=_tok(4 * A), v=_tok(5 * A), ko=NONE, q=NONE, qo=NONE, hq=4, rope=True, rotary=64, ws=16 * A,
               nbytes=256):
        r = api.Rope(rotary)
        return api.lib().dhsa_kv_append(ctypes.byref(self.cache), ctypes.byref(self.batch),
                                        ctypes.byref(r.c) if rope else None, None, k, v, ko, q, qo, hq, ws, nbytes,
                                        None)


STEP_REFUSALS = [
    (dict(dtype=3), INVALID), (dict(d=80), UNSUPPORTED), (dict(d=-1), INVALID), (dict(hkv=0), INVALID),
    (dict(page=24), UNSUPPORTED), (dict(page=256), UNSUPPORTED), (dict(page=0), INVALID), (dict(pages=0), INVALID),
    (dict(stride=2 * 16 * 128 - 8), INVALID), (dict(stride=2 * 16 * 128 + 4), INVALID),
    (dict(stride=2 ** 37), UNSUPPORTED), (dict(kp=None), INVALID), (dict(vp=A + 2), INVALID),
    (dict(max_pages=0), INVALID), (dict(table_stride=9), INVALID), (dict(max_pages=2 ** 27, table_stride=2 ** 27), UNSUPPORTED),
    (dict(cu=[1, 2, 3]), INVALID), (dict(cu=[0, 3, 2]), INVALID), (dict(d_cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(table=None), INVALID), (dict(seqs=-1), INVALID),
]


@pytest.mark.parametrize("kw,code", STEP_REFUSALS)
def test_paged_step_refusals(kw, code):
    s = _Step(**kw)
    assert s.size()[0] == code
    assert s.attend(nbytes=1 << 30) == code
    assert s.append() == code


@pytest.mark.parametrize("kw", [dict(groups=[0, 1]), dict(groups=[1, 2]), dict(groups=[0, 2, 1, 2]),
                                dict(groups=[0, 2], prefix=None), dict(groups=[0, 2], d_groups=None)])
def test_group_refusals(kw):
    assert _Step(**kw).size()[0] == INVALID
    assert _Step(**kw).attend(nbytes=1 << 30) == INVALID


def test_paged_attention_refusals():
    s = _Step(groups=[0, 2])
    assert s.size() [0] == OK and s.size()[1] > 256
    assert s.size(hq=3)[0] == INVALID and s.size(hq=0)[0] == INVALID
    assert s.attend(ws=None) == WORKSPACE and s.attend(ws=16 * A + 64) == WORKSPACE
    assert s.attend(nbytes=s.size()[1] - 1) == WORKSPACE
    assert s.attend(q=NONE) == INVALID and s.attend(out=NONE) == INVALID
    assert s.attend(q=_tok(4 * A + 4)) == INVALID and s.attend(out=_tok(8 * A, 520 // 8 * 8 + 4)) == INVALID
    assert s.attend(out=_tok(4 * A)) == INVALID and s.attend(out=_tok(4 * A + 1024)) == INVALID
    assert _Step(cu=[0, 2 ** 30, 2 ** 31 - 1]).size(hq=4)[0] == UNSUPPORTED
    # more row and key tiles than the kernels count in 32 bits
    many = _Step(cu=list(range(2049)), max_pages=2 ** 22, table_stride=2 ** 22)
    assert many.size()[0] == UNSUPPORTED and many.attend(nbytes=1 << 40) == UNSUPPORTED
    assert _Step(cu=list(range(2049)), max_pages=2 ** 13, table_stride=2 ** 13).size()[0] == OK
    assert _Step(cu=[0, 0, 0]).attend(q=NONE, out=NONE) == OK  # nothing to do
    assert _Step(cu=[0]).attend(q=NONE, out=NONE) == OK


def test_kv_append_refusals():
    s = _Step()
    assert s.append(ws=None) == WORKSPACE and s.append(nbytes=255) == WORKSPACE
    assert s.append(k=NONE) == INVALID and s.append(v=NONE) == INVALID
    assert s.append(q=_tok(6 * A)) == INVALID and s.append(qo=_tok(6 * A)) == INVALID
    assert s.append(q=_tok(6 * A), qo=_tok(7 * A), rope=False) == INVALID
    assert s.append(q=_tok(6 * A), qo=_tok(7 * A), hq=0) == INVALID
    assert s.append(rotary=256) == INVALID
    assert s.append(k=_tok(4 * A, 100)) == INVALID and s.append(ko=_tok(4 * A + 512)) == INVALID
    assert s.append(ko=_tok(5 * A)) == INVALID  # k_out on v
    assert _Step(cu=[0, 0, 0]).append(k=NONE, v=NONE) == OK
    # groups are not read by the append
    assert _Step(cu=[0, 0, 0], groups=[0, 1]).append(k=NONE, v=NONE) == OK


def test_binding_refusals_without_a_gpu():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        api.PagedCache(torch.zeros(3, 1, 16, 64), torch.zeros(3, 1, 16, 64))
    with pytest.raises(ValueError):
        api.rope(None, None, torch.zeros(4, dtype=torch.int32), api.Rope(64))
    with pytest.raises(ValueError):
        api.rope(x, None, torch.zeros(4, dtype=torch.int32), api.Rope(64))
    with pytest.raises(ValueError):
        api.PagedBatch([0, 1], torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32))


def test_struct_layouts_match_the_header():
    """sizeof as a C compiler lays the header's structs out."""
    import os
    import subprocess
    import tempfile

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"dhsa_rope_scaling": api._RopeScaling, "dhsa_rope_table": api._RopeTable, "dhsa_tokens": api._Tokens,
             "dhsa_paged_cache": api._PagedCache, "dhsa_paged_batch": api._PagedBatch}
    with tempfile.TemporaryDirectory() as t:
        src = os.path.join(t, "a.c")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include "dhsa.h"\nint main(void) {\n')
            for n in names:
                f.write('printf("%%zu\\n", sizeof(%s));\n' % n)
            f.write("return 0; }\n")
        exe = os.path.join(t, "a")
        subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I" + os.path.join(root, "include"), src, "-o", exe],
                       check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(c) for c in names.values()]


# ------------------------------------------------------------ operands of the binding


def test_broadcast_tokens_are_refused():
    """A tensor whose tokens share memory has the stride that would stand for packed tokens."""
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16).expand(3, 4, 64)
    with pytest.raises(ValueError, match="q overlap"):
        api._tokens(x, "q", 4, 64, torch.bfloat16, 3, x.get_device())
    half = torch.zeros(4 * 256, dtype=torch.bfloat16).as_strided((3, 4, 64), (128, 64, 1))
    with pytest.raises(ValueError, match="q overlap"):
        api._tokens(half, "q", 4, 64, torch.bfloat16, 3, half.get_device())
    with pytest.raises(ValueError, match="contiguous"):
        api._tokens(torch.zeros(3, 4, 128, dtype=torch.bfloat16)[:, :, ::2], "q", 4, 64, torch.bfloat16, 3, -1)
    one = torch.zeros(1, 4, 64, dtype=torch.bfloat16).expand(1, 4, 64)
    assert api._tokens(one, "q", 4, 64, torch.bfloat16, 1, -1).token_stride == 4 * 64
    apart = torch.zeros(3, 4, 128, dtype=torch.bfloat16)[:, :2].reshape(3, 4, 64)
    assert api._tokens(apart[:, :2], "q", 2, 64, torch.bfloat16, 3, -1).token_stride == 4 * 128
