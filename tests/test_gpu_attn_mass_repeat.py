"""Equal calls of sparse_attn_mass add equal bits."""

import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_attn_mass import SM, SPARSE, Case, _entries


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,lens,h,topk,fewest", SPARSE, ids=[f"{sum(c[0])}x{c[2]}-{c[3]}" for c in SPARSE])
def test_sparse_twice(dsa, rows, lens, h, topk, fewest):
    c = Case(rows, lens, h, seed=topk + h)
    idx = _entries(c, topk, fewest)
    lse = c.lse(lambda t: idx[t][idx[t] >= 0].long())
    d = c.cuda()
    args = (d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx.cuda(), lse.cuda(), SM)
    mass = torch.zeros(len(lens), c.max_ctx, dtype=torch.int64).cuda()
    out = dsa.sparse_attn_mass(*args, mass=mass)
    first = mass.clone()
    assert torch.equal(dsa.sparse_attn_mass(*args, mass=mass), out)
    assert torch.equal(mass, 2 * first) and (bool(first.any()) or not bool((idx >= 0).any()))
