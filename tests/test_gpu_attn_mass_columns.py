"""Columns of a chunk that are not the sequence's own must not reach its weights, whatever lies in them (attn_mass,
sparse_attn_mass).  Cases, formula and bounds are those of test_gpu_attn_mass."""

import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_attn_mass import SM, Case, _dense, _float


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _filled(dsa, c, byte):
    return torch.full((dsa.attn_mass_workspace_size(len(c.q), c.h, len(c.lens)),), byte, dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [0xFF, 0x7C, 0x7B, 0x00])     # two NaN, large numbers or zeros as fp16
@pytest.mark.parametrize("h", [5, 16, 64, 100])
def test_rows_that_see_nothing_whatever_the_workspace_holds(dsa, h, byte):
    """Rows with q_pos = -1 in the last and in another sequence, rows of an empty sequence, of none and of one that is too
    long; what the workspace held before makes no difference."""
    c = Case([3, 2, 1, 1], [150, 200, 0, 140], h, seed=h, max_ctx=200)
    for b, seen in ((0, [149, -1, 60]), (1, [-1, 199]), (3, [100])):
        c.q_pos[(c.q_seq == b).nonzero()[:, 0]] = torch.tensor(seen, dtype=torch.int32)
    lse = c.lse(c.seen)
    lse[torch.isneginf(lse)] = 1.0
    got = _dense(dsa, c, lse, workspace=_filled(dsa, c, byte))
    assert dsa.device_status() == 0
    want, tol = c.dense(lse)
    assert ((_float(got) - want).abs() <= tol).all()
    assert torch.equal(got, _dense(dsa, c, lse, workspace=_filled(dsa, c, 0)))
    c.q_seq[c.q_seq == 0] = torch.tensor([0, -1, 0], dtype=torch.int32)
    c.lens[3] = 201
    q_seq, lens = c.q_seq.clone(), c.lens.clone()
    c.q_pos[(c.q_seq == -1) | (c.q_seq == 3)], c.q_seq[c.q_seq == -1], c.lens[3] = -1, 0, 0     # (for the formula)
    want, tol = c.dense(lse)
    c.q_pos[(q_seq == -1) | (q_seq == 3)] = 50
    c.q_seq, c.lens = q_seq, lens
    got = _dense(dsa, c, lse, workspace=_filled(dsa, c, byte))
    assert set(dsa.status_names(dsa.device_status())) == {"BAD_SEQ", "BAD_LEN"}
    assert ((_float(got) - want).abs() <= tol).all()


@pytest.mark.gpu
def test_every_row_sees_nothing(dsa):
    c = Case([2, 1], [100, 90], 16, seed=1)
    c.q_pos[:] = -1
    lse = torch.ones(3, 16)
    assert not _dense(dsa, c, lse, workspace=_filled(dsa, c, 0xFF)).any() and dsa.device_status() == 0
