"""Serving calls as programs make them: buffers that go on being used, handles that live on."""

import numpy as np
import pytest
import torch

from dynamic_hierarchical_sparse_b200 import api
from tests import serving_cases as C

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("make", [lambda x: np.array(x, np.int32), lambda x: torch.tensor(x, dtype=torch.int32)],
                         ids=["numpy", "torch"])
def test_a_batch_keeps_its_own_offsets(make):
    """A program that builds its next step's offsets in the same buffer changes no batch that it made before."""
    st = C.Step(1, BF16, 8, 2, 64, 16, [1, 2, 1], [40, 60, 50], ([0, 2, 3], [20, 0]))
    cu, ptr = make(st.cu), make(st.groups[0])
    lens = torch.tensor(st.held, dtype=torch.int32, device="cuda")
    batch = api.PagedBatch(cu, lens, torch.from_numpy(st.table).cuda(), ptr,
                           torch.tensor(st.groups[1], dtype=torch.int32, device="cuda"))
    cu += 1000
    ptr += 1000
    # (no call before this holds: offsets on the host beyond those on the device would be read there)
    assert batch.h_cu.tolist() == st.cu and batch.h_groups.tolist() == st.groups[0]
    q = st.q.cuda()
    got = api.PagedAttention(st.cache(), batch, 8)(q, torch.empty_like(q))
    assert torch.equal(got, api.PagedAttention(st.cache(), st.batch(), 8)(q, torch.empty_like(q)))


@pytest.mark.parametrize("room", [0, 1 << 18])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_batches_without_work(dt, room):
    """Every sequence idle, empty prefixes, prefixes behind idle sequences: zeros, lse of -infinity, nothing reported."""
    for held, prefix in (([0] * 9, [0]), ([0] * 9, [40]), ([5] * 9, [0]), ([0] * 8 + [41], [40])):
        st = C.Step(2, dt, 16, 2, 64, 16, [1] * 9, held, ([0, 9], prefix), room=room)
        q, att = st.q.cuda(), api.PagedAttention(st.cache(), st.batch(), 16)
        att.ws[256:].fill_(0xFF)
        out, lse = torch.full_like(q, 3.0), torch.empty(9, 16, device="cuda")
        att(q, out, lse=lse)
        want, want_lse, mean = st.want()
        bound, lse_bound = st.bounds(want, want_lse, mean)
        assert att.status() == 0
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
        idle = np.array(held) == 0
        got = lse.double().cpu().numpy()
        assert np.all(got[idle] == -np.inf) and np.all(np.abs(got[~idle] - want_lse[~idle]) <= lse_bound[~idle])
