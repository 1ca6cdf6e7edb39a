"""norm_rope_quant_kv at the ends of what it is given: rows without a norm, and angles whose sines are tiny."""

import math

import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_norm_rope import U, _e4m3, _stored


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


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [-20, -28, -31, -34, -50])
def test_sines_of_small_angles_keep_their_relative_accuracy(dsa, exponent):
    """Keys that are zero in the first of the two parts which the turn mixes: its group of 32 then holds nothing but
    -s u of the other part, for angles of 2^exponent to 2^(exponent + 1) turns.  u w is off by 29 units of 2^-24 (the
    bound of test_gpu_norm_rope without a mean), the sine of so small an angle is the angle, of three roundings, the
    polynomial's two and the amplitude's one, the products take two: below 96 units of the value's own size."""
    n = 60
    g = torch.Generator().manual_seed(-exponent)
    k = torch.randn(n, 128, generator=g).to(torch.bfloat16)
    k[:, :32] = 0
    w = 1 + 0.2 * torch.rand(128, generator=g)
    turns = torch.tensor([round(2.0 ** (64 + exponent) * (1 + i / 32)) for i in range(32)])
    pos = torch.tensor([1, -1] * (n // 2), dtype=torch.int32)
    kc = dsa.alloc_k_cache(1)
    dsa.norm_rope_quant_kv(k.cuda(), None, pos.cuda(), torch.arange(n).cuda(), kc, None, turns.cuda(), k_weight=w.cuda(),
                           amplitude=1.25)
    codes, e8, _, _ = _stored(kc, dsa.alloc_kv_cache(1), torch.arange(n))
    u = k.double()
    u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    s = torch.sin(2 * math.pi * pos.double()[:, None] * turns.double() * 2.0 ** -64) * 1.25
    y = -u[:, 32:64] * s
    d = 96 * U * y.abs()
    top = y.abs().amax(-1)
    e = e8[:, 0] - 127
    e_lo, e_hi = (torch.frexp(v)[1] - 9 for v in (top * (1 - 96 * U), top * (1 + 96 * U)))
    assert ((e >= e_lo) & (e <= e_hi)).all()
    scale = torch.exp2(e.double())[:, None]
    assert ((codes[:, :32] >= _e4m3((y - d) / scale)) & (codes[:, :32] <= _e4m3((y + d) / scale))).all()
