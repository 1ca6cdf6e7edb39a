"""prefix_attn over caches whose scales lie at the ends of fp32, or far apart between tiles: the sums of
weights must neither overflow nor vanish.  Tolerances are those of test_gpu_prefix, without its
absolute term: S = sum_j p_j |v_j|,
|o - ref| <= (2^-10 + 2 D + 2^-20) S + n 2^-25 max|v| + 2^-8 |ref|, D = max|logit| 576 2^-24."""

import numpy as np
import pytest
import torch

import oracle
from dsa_testlib import ensure_built
from test_gpu_prefix import Batch, SM, round11
from test_gpu_prefix_sink import FEW
from test_gpu_prefix_tiles import SHAPES


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


# the exponents of the scales by position
SCALES = {
    "tiny": lambda p, r: -124.0 + 10 * r,
    "huge": lambda p, r: 100.0 + 10 * r,
    "tiny_then_plain": lambda p, r: np.where(p < 320, -104.0, -8.0) + r,
    "plain_then_tiny": lambda p, r: np.where(p < 320, -8.0, -104.0) + r,
    "every_second_tile_tiny": lambda p, r: np.where(p // 64 % 2 == 0, -104.0, -8.0) + r,
    # zeros alone, whose exponent is free
    "a_tile_of_zeros_then_tiny": lambda p, r: np.where(p < 64, -np.inf, -124.0 + 10 * r),
    "tiles_of_zeros_then_plain": lambda p, r: np.where(p < 192, -np.inf, -8.0 + r),
    "tiles_of_zeros_among_huge": lambda p, r: np.where(p // 64 % 3 == 1, -np.inf, 100.0 + r),
    "every_second_tile_zeros": lambda p, r: np.where(p // 64 % 2 == 0, -np.inf, -8.0 + r),
    "zeros_alone": lambda p, r: np.full(p.shape, -np.inf),
}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", sorted(SCALES))
@pytest.mark.parametrize("shape", sorted(SHAPES) + sorted(FEW))
def test_scales_at_the_ends_of_the_range(dsa, shape, kind):
    n, h, lens, prefix, max_ctx, *plan = SHAPES[shape] if shape in SHAPES else FEW[shape]
    got = dsa.test_prefix_plan(n, h, len(lens), prefix, max_ctx)
    assert all(got[k] == v for k, v in plan[0].items()) if plan else got["few_parts"] > 0
    rows = [(i * len(lens) // n, lens[i * len(lens) // n] - 1 - i % 5) for i in range(n)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=len(kind), max_ctx=max_ctx)
    rng = np.random.default_rng(len(shape) + len(kind))
    rec = b.cache.cpu().numpy().reshape(-1, 608).copy()
    for s in range(len(lens)):
        p = np.arange(max_ctx)
        pages = np.where(p < prefix, np.r_[b.pages.numpy(), 0][np.minimum(p // 64, len(b.pages))], b.table.numpy()[s][p // 64])
        scale = np.exp2(SCALES[kind](p, rng.random(max_ctx))).astype(np.float32)
        rec[pages.astype(np.int64) * 64 + p % 64, 576:596] = np.repeat(scale[:, None], 5, 1).view(np.uint8)
    b.cache.copy_(torch.from_numpy(rec).view(b.cache.shape))
    if "huge" in kind:
        b.q *= 2.0 ** -112     # logits of some units
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    o, e = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t in {0, n // 3, n - 1}:
        s, seen = int(b.q_seq[t]), np.arange(int(b.q_pos[t]) + 1)
        own = b.table.numpy()[s][seen // 64]
        pages = np.where(seen < prefix, np.r_[b.pages.numpy(), 0][np.minimum(seen // 64, len(b.pages))], own)
        r = rec[pages.astype(np.int64) * 64 + seen % 64]
        kv = oracle.fp8_tile_dequantize(r[:, :576], r[:, 576:596].copy().view(np.float32))
        kv = kv if h <= 32 else round11(kv)
        q = b.q[t].double().numpy()
        x = SM * (q @ kv.T)
        m = x.max(1, keepdims=True)
        w = np.exp(x - m)
        z = w.sum(1, keepdims=True)
        v = kv[:, :512]
        ref, size = w / z @ v, w / z @ np.abs(v)
        d = SM * (np.abs(q) @ np.abs(kv).T).max() * 576 * 2.0 ** -24
        tol = (2.0 ** -10 + 2 * d + 2.0 ** -20) * size + len(kv) * 2.0 ** -25 * np.abs(v).max() + 2.0 ** -8 * np.abs(ref)
        assert (np.abs(o[t] - ref) <= tol).all(), t
        assert np.abs(e[t] - (m + np.log(z))[:, 0]).max() <= 1e-4 + d


@pytest.mark.gpu
@pytest.mark.parametrize("shape", sorted(SHAPES) + sorted(FEW))
def test_a_nan_among_zeros(dsa, shape):
    # a tile of zeros with one poisonous position: NaN for the rows that see it, nothing to the others;
    # lse = ln 71 = 4.3 by a log2 and a product in fp32, each off by 2^-22 at most, times ln 2
    n, h, lens, prefix, max_ctx, *_ = SHAPES[shape] if shape in SHAPES else FEW[shape]
    rows = [(i * len(lens) // n, 70 if i % 2 else 130) for i in range(n)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=9, max_ctx=max_ctx)
    b.cache[:] = 0
    for s in range(len(lens)):
        page = b.pages[1] if prefix > 100 else b.table[s, 1]
        b.cache.view(-1, 608)[int(page) * 64 + 100 - 64, 7] = 0x7F
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    assert torch.isnan(out[::2]).all() and torch.isnan(lse[::2]).all()
    assert not out[1::2].any()
    assert (lse[1::2] - np.log(71.0)).abs().max() <= 1e-6
