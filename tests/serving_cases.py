"""Inputs and error bounds of the serving operators' GPU tests (test code only)."""

import random

import numpy as np
import torch

from dynamic_hierarchical_sparse_b200 import api
from oracle import serving_oracle as S
from oracle.dhsa_oracle import as_f64

F32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def v_type(dtype):
    return torch.float16 if dtype == torch.bfloat16 else dtype


def rope_bound(x, want, positions, freqs, factor, interleaved, dtype):
    """|y - exact|: the output's rounding, and per product x * cos (or sin): cos
    and sin off by 4 half steps of fp32 each (2 ulp of the function, the rounding
    of its argument of at most pi / 4, and of a * cos), the table by 2^-32 turns
    (1.5e-9 radians, under 2^-28), the product and the sum by one half step each.
    The oracle's and the table's frequencies (up to 1, or as given) and the
    oracle's angles are off by 2^-53 of themselves, so at position p by |p| 2^-53 each."""
    n = len(freqs)
    a = np.abs(as_f64(x))
    first = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    second = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    pair = np.zeros_like(a)
    pair[..., first] = pair[..., second] = factor * (a[..., first] + a[..., second])
    far = 4 * 2.0 ** -53 * np.abs(np.asarray(positions, dtype=np.float64))[:, None, None]
    return half_step(dtype) * np.abs(want) + (7 * F32 + far) * pair


class Step:
    """A paged cache whose unwritten slots hold NaN, one step's queries, and the
    tables (entries behind a sequence's pages are nonsense).

    groups: None, or (group_ptr, prefix_lens); the whole pages of a prefix are
    shared, the page that a prefix ends in is the first sequence's, while the
    others' own page holds NaN in the prefix's part.  room: tokens that a table
    row is wide enough for (long prefixes take another kernel, by that bound)."""

    def __init__(self, seed, dtype, hq, hkv, d, page, new, held, groups=None, extra_rows=0, gap=0, values="normal",
                 room=0):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        self.dtype, self.hq, self.hkv, self.d, self.page = dtype, hq, hkv, d, page
        self.new, self.held, self.groups = list(new), list(held), groups
        B = len(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        prefix_of = [0] * B
        first_of = list(range(B))
        if groups is not None:
            for x in range(len(groups[1])):
                for b in range(groups[0][x], groups[0][x + 1]):
                    prefix_of[b], first_of[b] = groups[1][x], groups[0][x]
        # a sequence's row covers what it holds; a group's first one covers the prefix too
        cover = [max(h, prefix_of[b] if first_of[b] == b else 0) for b, h in enumerate(held)]
        width = max([1, room // page] + [-(-c // page) for c in cover])
        pages = sum(-(-c // page) for c in cover) + 3
        ids = list(range(pages))
        r.shuffle(ids)
        self.table = np.full((B, width), 2 ** 30, dtype=np.int32)
        self.table[:, ::2] = -7
        for b in range(B):
            for i in range(-(-cover[b] // page)):
                shared = i < prefix_of[b] // page and first_of[b] != b
                self.table[b, i] = self.table[first_of[b], i] if shared else ids.pop()
        self.pages = pages
        kp = torch.full((pages, hkv, page, d), float("nan"))
        vp = torch.full((pages, hkv, page, d), float("nan"))
        mix = torch.randn(hkv, 4, d, generator=g)
        for b in range(B):
            lo = 0 if first_of[b] == b else prefix_of[b]
            for i in range(lo // page, -(-cover[b] // page)):
                a, e = max(lo, i * page), min(cover[b], (i + 1) * page)
                if e <= a:  # the sequence ends within the prefix
                    continue
                k = torch.randn(hkv, e - a, d, generator=g)
                if values == "peaks":
                    k += 0.5 * torch.randn(hkv, e - a, 4, generator=g) @ mix
                kp[self.table[b, i], :, a - i * page:e - i * page] = k
                vp[self.table[b, i], :, a - i * page:e - i * page] = torch.randn(hkv, e - a, d, generator=g)
        self.k_pages, self.v_pages = kp.to(dtype), vp.to(dtype).to(v_type(dtype))
        q = torch.randn(self.cu[-1] + extra_rows, hkv, hq // hkv, d, generator=g)
        if values == "peaks":
            q += 0.5 * torch.einsum("tgrc,gcd->tgrd", torch.randn(*q.shape[:3], 4, generator=g), mix)
        self.q = q.reshape(-1, hq, d).to(dtype)
        self.gap = gap

    def cache(self, dev="cuda"):
        if not self.gap:
            return api.PagedCache(self.k_pages.to(dev), self.v_pages.to(dev))
        # pages that lie apart: K and V in buffers with `gap` elements behind every page
        out = []
        for t in (self.k_pages, self.v_pages):
            n = t[0].numel()
            flat = torch.full((t.shape[0], n + self.gap), float("nan"), dtype=t.dtype, device=dev)
            flat[:, :n] = t.reshape(t.shape[0], -1).to(dev)
            out.append(flat[:, :n].unflatten(1, t.shape[1:]))
        return api.PagedCache(*out)

    def batch(self, dev="cuda"):
        kw = {}
        if self.groups is not None:
            kw = dict(group_ptr=self.groups[0],
                      prefix_lens=torch.tensor(self.groups[1], dtype=torch.int32, device=dev))
        return api.PagedBatch(self.cu, torch.tensor(self.held, dtype=torch.int32, device=dev),
                              torch.from_numpy(self.table).to(dev), **kw)

    def want(self, scale=None):
        kw = {} if self.groups is None else dict(group_ptr=self.groups[0], prefix_lens=self.groups[1])
        args = (self.cu, self.held, self.table.tolist())
        out, lse = S.paged_attention(self.q, self.k_pages, self.v_pages, *args, scale=scale, **kw)
        mean = S.paged_attention(self.q, self.k_pages, self.v_pages.abs(), *args, scale=scale, **kw)[0]
        # the largest sum over i of |q_i k_i| * scale that a row meets (an upper bound: the largest key of all)
        return out, lse, mean

    def bounds(self, out, lse, mean, scale=None):
        """|out - exact| and |lse - exact|.

        A logit x = scale * sum of d products is off by at most d half steps of
        fp32 of sum |q_i k_i| scale <= |q| |k| scale, by its scaling, the
        subtraction of the maximum and the fp32 log2(e) by another 4 of |x| (at
        most as large); ex2.approx by 2^-22; joining two partials takes two more
        such factors.  The weights then are off by dx (relative), in f16 by
        another 2^-11, or 2^-25 of the largest one seen where that is more;
        summing n of them in fp32 by n half steps at most.  Numerator and
        denominator together: twice that, times the weighted mean of |v|."""
        fin = lambda t: np.nan_to_num(as_f64(t), nan=0.0)  # noqa: E731
        scale = self.d ** -0.5 if scale is None else scale
        qn = np.linalg.norm(fin(self.q[:self.cu[-1]]), axis=-1).reshape(self.cu[-1], self.hkv, -1)
        kn = np.linalg.norm(fin(self.k_pages), axis=-1).max(axis=(0, 2))
        x = (qn * kn[:, None]).reshape(self.cu[-1], self.hq) * scale
        n = max(self.held + [1])
        dx = (self.d + 4) * F32 * x + 3 * 2.0 ** -22 + n * F32
        f16 = self.dtype == torch.bfloat16
        tiny = n * 2.0 ** -25 * np.abs(fin(self.v_pages)).max() if f16 else 0.0
        err = (2 * dx + (2.0 ** -11 if f16 else 0.0))[..., None] * mean + tiny
        return half_step(self.dtype) * (np.abs(out) + err) + err, dx + 2 * F32 * np.abs(np.where(np.isfinite(lse), lse, 0))
