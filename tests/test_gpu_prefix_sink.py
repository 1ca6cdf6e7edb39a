"""prefix_attn with one position far above the rest and nothing in it: the output is the rest's, by
far smaller than the largest weight, and has to be as good as any other.

Every logit comes from dim 512 alone (the query's other dims are 0), so the rest's weights are
equal and their roundings do not average out.  The sink's values are 0 and the others' positive, so
|o| is the size S that the tolerance of test_gpu_prefix is relative to: two roundings to fp16 (2^-11
each), 2 D for the logits, 2^-20 for 2^x, 2^-8 for the result."""

import numpy as np
import pytest
import torch

import oracle
from dsa_testlib import ensure_built
from test_gpu_prefix import Batch, SM, round11
from test_gpu_prefix_tiles import POWERS, SHAPES


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


FEW = {"few": (4, 16, [700, 650, 800, 1000], 0, 1000), "few_wide": (4, 32, [700, 650, 800, 1000], 640, 1000)}


@pytest.mark.gpu
# where the sink is, and how many powers of two it stands above the rest; a sink of a later tile raises
# the reference, behind which 11 bits reach 2^-19 of the largest weight
@pytest.mark.parametrize("at,gaps", [(0, (4.0, 11.3, 16.6, 20.6, 24.6, 26.6)), (37, (20.6, 24.6)), (200, (11.3, 16.6, 18.6)),
                                     (100, (9.3, 17.6))])
@pytest.mark.parametrize("shape", sorted(SHAPES) + sorted(FEW))
def test_the_rest_behind_a_sink(dsa, shape, at, gaps):
    n, h, lens, prefix, max_ctx, *plan = SHAPES[shape] if shape in SHAPES else FEW[shape]
    got = dsa.test_prefix_plan(n, h, len(lens), prefix, max_ctx)
    assert all(got[k] == v for k, v in plan[0].items()) if plan else got["few_parts"] > 0
    rows = [(i * len(lens) // n, lens[i * len(lens) // n] - 1 - i % 5) for i in range(n)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=at, max_ctx=max_ctx)
    vals = torch.randn(b.num_pages * 64, 576, generator=torch.Generator().manual_seed(at + 1)).abs() + 0.25
    vals[:, 512:] = 0
    for s in range(len(lens)):
        page = b.pages[at // 64] if at < prefix else b.table[s, at // 64]
        vals[int(page) * 64 + at % 64, :512] = 0
        vals[int(page) * 64 + at % 64, 512] = 1.0
    dsa.quant_kv_fp8(vals.to(torch.bfloat16).cuda(), torch.arange(b.num_pages * 64).cuda(), b.cache)
    gap = torch.tensor(gaps)[torch.arange(n * h) % len(gaps)].view(n, h)
    b.q[:] = 0
    b.q[..., 512] = (gap / POWERS).to(torch.bfloat16)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    rec = b.cache.cpu().numpy().reshape(-1, 608)
    o = out.double().cpu().numpy()
    for t in {0, n // 2, n - 1}:
        s, seen = int(b.q_seq[t]), np.arange(int(b.q_pos[t]) + 1)
        own = b.table.numpy()[s][seen // 64]
        pages = np.where(seen < prefix, np.r_[b.pages.numpy(), 0][np.minimum(seen // 64, len(b.pages))], own)
        r = rec[pages.astype(np.int64) * 64 + seen % 64]
        kv = oracle.fp8_tile_dequantize(r[:, :576], r[:, 576:596].copy().view(np.float32))
        kv = kv if h <= 32 else round11(kv)
        x = SM * (b.q[t].double().numpy() @ kv.T)
        assert np.array_equal(x.argmax(1), np.full(h, at))
        w = np.exp(x - x.max(1, keepdims=True))
        ref = w @ kv[:, :512] / w.sum(1, keepdims=True)
        d = np.abs(x).max() * 576 * 2.0 ** -24
        assert np.abs(o[t] / ref - 1).max() <= 2.0 ** -8 + 2.0 ** -10 + 2 * d + 2.0 ** -20


@pytest.mark.gpu
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_a_sinks_row_beside_rows_whose_logits_rise(dsa, shape):
    # even heads: a sink at position 0; odd heads, in the same warps: logits that rise from tile to tile
    # and raise their references again and again
    n, h, lens, prefix, max_ctx, plan = SHAPES[shape]
    got = dsa.test_prefix_plan(n, h, len(lens), prefix, max_ctx)
    assert all(got[k] == v for k, v in plan.items())
    rows = [(i * len(lens) // n, lens[i * len(lens) // n] - 1 - i % 5) for i in range(n)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=5, max_ctx=max_ctx)
    vals = torch.randn(b.num_pages * 64, 576, generator=torch.Generator().manual_seed(6)).abs() + 0.25
    vals[:, 512:] = 0
    for s in range(len(lens)):
        p = torch.arange(max_ctx)
        pages = torch.where(p < prefix, torch.cat([b.pages, b.pages.new_zeros(1)])[(p // 64).clamp(max=len(b.pages))],
                            b.table[s][p // 64]).long()
        vals[pages * 64 + p % 64, 513] = (p // 64).float()
        vals[pages[0] * 64, :512], vals[pages[0] * 64, 512] = 0, 1.0
    dsa.quant_kv_fp8(vals.to(torch.bfloat16).cuda(), torch.arange(b.num_pages * 64).cuda(), b.cache)
    b.q[:] = 0
    b.q[:, ::2, 512] = (torch.tensor([20.6, 24.6])[torch.arange(n * ((h + 1) // 2)) % 2].view(n, -1) / POWERS).to(torch.bfloat16)
    b.q[:, 1::2, 513] = 17.0 / POWERS
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    rec = b.cache.cpu().numpy().reshape(-1, 608)
    for t in {0, n // 2, n - 1}:
        s, seen = int(b.q_seq[t]), np.arange(int(b.q_pos[t]) + 1)
        pages = np.where(seen < prefix, np.r_[b.pages.numpy(), 0][np.minimum(seen // 64, len(b.pages))],
                         b.table.numpy()[s][seen // 64])
        r = rec[pages.astype(np.int64) * 64 + seen % 64]
        kv = round11(oracle.fp8_tile_dequantize(r[:, :576], r[:, 576:596].copy().view(np.float32)))
        x = SM * (b.q[t].double().numpy() @ kv.T)
        w = np.exp(x - x.max(1, keepdims=True))
        ref = w @ kv[:, :512] / w.sum(1, keepdims=True)
        d = np.abs(x).max(1, keepdims=True) * 576 * 2.0 ** -24
        bound = 2.0 ** -8 + 2.0 ** -10 + 2 * d + 2.0 ** -20
        assert np.all(np.abs(out[t].double().cpu().numpy() / ref - 1) <= bound), t
