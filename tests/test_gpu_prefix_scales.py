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
    if kind == "huge":
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
        assert (np.abs(o[t] - ref) / tol).max() <= 1, t
        assert np.abs(e[t] - (m + np.log(z))[:, 0]).max() <= 1e-4 + d
