"""Weights far below the largest one (bf16 attention takes them in f16): keys 15 to
20 nats under attention sinks whose values are zero, so that the output is theirs alone."""

import math

import numpy as np
import pytest
import torch

from dynamic_hierarchical_sparse_b200 import api
from tests import serving_cases as C, steady_cases as T

pytestmark = pytest.mark.gpu

LIFT = {"list": 15, "prefix": 11}  # log2 of the largest weight when its base is set


def _sinks(name, gap, every):
    """A case of steady_cases in which every `every`-th key is a sink: logits of `gap` above all others, values 0."""
    dtype, hq, hkv, d, page, (new, held, groups), _ = T.CASES[name]
    st = C.Step(3, dtype, hq, hkv, d, page, new, held, groups, room=T.room(name))
    g = torch.Generator().manual_seed(4)
    u = torch.randn(hkv, 1, d, generator=g)
    u /= u.norm(dim=-1, keepdim=True)
    k, v = 0.25 * st.k_pages.float(), st.v_pages.float().abs() + 0.25
    at = slice(3, None, every)
    k[:, :, at] = torch.where(k[:, :, at].isnan(), k[:, :, at], math.sqrt(d) * u)
    v[:, :, at] *= 0.0
    st.k_pages, st.v_pages = k.to(dtype), v.to(st.v_pages.dtype)
    q = 0.25 * st.q.float().reshape(-1, hkv, hq // hkv, d) + gap * u
    st.q = q.reshape(-1, hq, d).to(dtype)
    return st


@pytest.mark.parametrize("gap", [15.0, 17.0, 17.5, 20.0])
@pytest.mark.parametrize("name", ["own_16", "own_32", "own_64", "own_d256", "pieces_d128", "long_d128_apart",
                                  "pieces_d64_apart", "long_d256"])
def test_keys_far_below_a_sink_keep_their_weight(name, gap):
    st = _sinks(name, gap, 16)
    cache, batch, q = st.cache(), st.batch(), st.q.cuda()
    att = api.PagedAttention(cache, batch, st.hq)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    att(q, out, lse=lse)
    assert att.status() == 0
    want, want_lse, mean = T.want(st, "cuda")
    assert want.max() < 2.0 ** -15  # the sinks have nearly all the weight
    # the logits' error dx as in Step.bounds; a weight is off by 2^-11 of itself, or where f16 is subnormal by
    # 2^-25 of its base's largest, which is 2^-(25 + lift) of the row's: over the sum of the sinks' weights (within e^-1
    # of the largest each: q's other part moves their common logit by rounding alone), `every` of them a sink.
    # The output then rounds once.
    fin = lambda t: np.nan_to_num(t.double().numpy(), nan=0.0)  # noqa: E731
    qn = np.linalg.norm(fin(st.q), axis=-1).max()
    kn = np.linalg.norm(fin(st.k_pages), axis=-1).max()
    n = max(st.held)
    dx = (st.d + 4) * C.F32 * qn * kn * st.d ** -0.5 + 3 * 2.0 ** -22 + n * C.F32
    vmax = float(st.v_pages.float().nan_to_num(0.0).max())
    tiny = 16 * math.e * 2.0 ** -(25 + LIFT[T.CASES[name][6]["kind"]]) * vmax
    err = (2 * dx + 2.0 ** -11) * mean + tiny
    bound = C.half_step(st.dtype) * (np.abs(want) + err) + err
    off = np.abs(out.double().cpu().numpy() - want)
    print(name, gap, "worst error over bound %.3f, relative %.4f" % ((off / bound).max(), (off / want).max()))
    assert np.all(off <= bound), float((off / bound).max())
    assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= dx + 2 * C.F32 * np.abs(want_lse).max()
