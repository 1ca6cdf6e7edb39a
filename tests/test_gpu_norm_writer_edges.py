"""norm_rope_quant_kv at the ends of what it is given: rows without a norm."""

import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_norm_rope import _stored


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [False, True])
def test_rows_of_zeros_without_eps(dsa, weights):
    """0 / 0: NaN in both caches, as rows whose squares are all below fp32; the dims that are not normed stay."""
    g = torch.Generator().manual_seed(1)
    k, kv = torch.randn(5, 128, generator=g).to(torch.bfloat16), torch.randn(5, 576, generator=g).to(torch.bfloat16)
    k[1], kv[1, :512] = 0, 0
    k[2], kv[2, :512] = 1e-30, -1e-30
    k[3], kv[3] = 0, 0
    k[3, 7], kv[3, 9] = 1e-18, 1e-18              # (a square of 1e-36: a norm there is)
    turns, _ = dsa.rope_turns(64)
    kc, vc = dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)
    pos = torch.arange(5, dtype=torch.int32).cuda()
    w = dict(k_weight=torch.rand(128).cuda() + 0.5, k_bias=torch.ones(128).cuda(), kv_weight=torch.rand(512).cuda() + 0.5)
    dsa.norm_rope_quant_kv(k.cuda(), kv.cuda(), pos, torch.arange(5).cuda(), kc, vc, turns, eps=0.0, **(w if weights else {}))
    assert dsa.device_status() == 0
    codes, _, vcodes, vscales = _stored(kc, vc, torch.arange(5))
    values = vcodes * vscales.repeat_interleave(128, -1)[:, :576]
    for row in (1, 2):
        assert torch.isnan(codes[row]).all() and torch.isnan(values[row, :512]).all()
        assert torch.isfinite(values[row, 512:]).all()
    for row in (0, 3, 4):
        assert torch.isfinite(codes[row]).all() and torch.isfinite(values[row]).all()
