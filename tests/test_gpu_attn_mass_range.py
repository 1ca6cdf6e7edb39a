"""attn_mass and sparse_attn_mass where fp32 holds the logits but not every sum on the way to them: cached values up to the
largest that a record can hold, and queries down to the smallest.  Formula and bounds are those of test_gpu_attn_mass."""

import math

import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_attn_mass import SM, Case, _dense, _float, _sparse_want, _values


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _sparse(dsa, c, idx, lse):
    d = c.cuda()
    mass = torch.zeros(len(c.lens), c.max_ctx, dtype=torch.int64).cuda()
    w = dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx.cuda(), lse.cuda(), SM, mass=mass)
    return w.cpu().double(), _float(mass)


def _grow(c, b, positions, tile, exponent):
    """Values of a tile of the positions 2^exponent times as large."""
    for p in positions:
        slot = int(c.table[b, p // 64]) * 64 + p % 64
        at = slice(576 + 4 * tile, 580 + 4 * tile)
        s = c.rec[slot, at].clone().view(torch.float32) * 2.0 ** exponent
        assert torch.isfinite(s * 448).all()
        c.rec[slot, at] = s.view(torch.uint8)
    c.kv = _values(c.rec)


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale,kv_scale", [(2.0 ** -62, 2.0 ** 61), (2.0 ** -108, 2.0 ** 108), (2.0 ** -117, 2.0 ** 117)])
def test_small_queries_and_large_values(dsa, q_scale, kv_scale):
    c = Case([2, 3], [150, 300], 7, seed=5, q_scale=q_scale, kv_scale=kv_scale)
    lse = c.lse(c.seen)
    want, tol = c.dense(lse)
    assert ((_float(_dense(dsa, c, lse)) - want).abs() <= tol).all()
    idx = torch.stack([torch.randperm(150, generator=c.g)[:70] for _ in range(5)]).to(torch.int32)
    lse = c.lse(lambda t: idx[t].long())
    w, e, want, tol = _sparse_want(c, idx, lse)
    got, mass = _sparse(dsa, c, idx, lse)
    assert ((got - w).abs() <= e).all() and ((mass - want).abs() <= tol).all()
    assert dsa.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h", [5, 16, 100])
def test_large_values_that_only_another_sequences_queries_meet(dsa, h):
    """Positions of sequence 0 with a huge tile where its own queries are zero: the next rows' queries lie in the same
    chunk of columns, and products with them leave fp32."""
    c = Case([2, 2], [140, 200], h, seed=h)
    own = c.q_seq == 0
    c.q[own, :, 256:384] = 0
    c.q_pos[own] = 139
    _grow(c, 0, (0, 3, 77, 100, 139), 2, 118)
    lse = c.lse(c.seen)
    want, tol = c.dense(lse)
    assert torch.isfinite(tol).all()
    assert ((_float(_dense(dsa, c, lse)) - want).abs() <= tol).all()
    order = torch.argsort(c.q_seq, stable=True)               # sparse: the next row's, so sequence 0 first
    c.q, c.q_seq, c.q_pos = c.q[order], c.q_seq[order], c.q_pos[order]
    idx = torch.stack([torch.randperm(140, generator=c.g)[:100] for _ in range(4)]).to(torch.int32)
    idx[:2, :5] = torch.tensor([0, 3, 77, 100, 139], dtype=torch.int32)
    lse = c.lse(lambda t: idx[t].long())
    w, e, want, tol = _sparse_want(c, idx, lse)
    got, mass = _sparse(dsa, c, idx, lse)
    assert ((got - w).abs() <= e).all() and ((mass - want).abs() <= tol).all()
    assert dsa.device_status() == 0


@pytest.mark.gpu
def test_a_head_of_no_weight_over_large_values(dsa):
    """lse = -inf adds nothing where the head's own logits leave fp32; the other heads do not meet the large tile."""
    c = Case([1], [130], 6, seed=9)
    c.q_pos[:] = 129
    c.q[:, [0, 1, 2, 4, 5], 128:256] = 0
    _grow(c, 0, range(0, 130, 3), 1, 118)
    lse = c.lse(c.seen)
    lse[0, 3] = -math.inf
    want, tol = c.dense(lse)
    tol = tol.nan_to_num(0, 0, 0)
    keep = [0, 1, 2, 4, 5]
    alone = Case.weights(c, 0, c.seen(0), lse)                # (head 3's bound is inf * 0: taken from the others)
    l, size = c.terms(0, c.row(0))
    w = torch.exp(l[keep] - lse[0, keep].double()[:, None])
    rel = 2.0 ** -19 * size[keep] + 2.0 ** -22 * (l[keep].abs() + lse[0, keep].abs().double()[:, None] + 1) + 400 * 2.0 ** -24
    want[0, :130], tol[0, :130] = w.sum(0), (w * rel).sum(0) + 6 * 2.0 ** -37
    assert len(alone) == 2 and ((_float(_dense(dsa, c, lse)) - want).abs() <= tol).all()
    assert dsa.device_status() == 0
