"""NaN and infinities through the rotating cache writers: stored as dsa_quant_kv stores the turned
values, so that a row that went wrong upstream stays wrong for its reader.

At position 0 a pair (a, b) becomes (a - 0 b, 0 a + b): itself where both are finite, and NaN beside
an infinity or NaN.  These values are exact in bf16, so the plain writer's bytes are the reference."""

import math

import numpy as np
import pytest
import torch

from dsa_testlib import ensure_built

pytestmark = pytest.mark.gpu
NAN = math.nan


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _rows(seed, n):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, 128, generator=g), torch.randn(n, 576, generator=g)


def _turned_at_zero(x, offset, layout):
    y = x.clone()
    i = torch.arange(32)
    i0, i1 = (offset + i, offset + 32 + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
    a, b = x[:, i0], x[:, i1]
    y[:, i0], y[:, i1] = a - 0.0 * b, 0.0 * a + b
    return y


def _kv_cases(kv, top):
    """Each row wrong in its own way; the last two as they are."""
    kv[0, 128:256] = NAN                    # a whole tile
    kv[1, 256:384] = -NAN
    kv[2, 5] = NAN                          # one value
    kv[3, 128:132] = NAN                    # all of a thread's values
    kv[4, 384] = top
    kv[5, 0:128] = -top
    kv[6, 130], kv[6, 131] = top, NAN
    kv[7, 512:] = NAN                       # the whole rotary part
    kv[8, 512:544] = NAN                    # half of it
    kv[9, 515] = NAN
    kv[10, 520] = top
    kv[11, 512:] = -top
    kv[12, 512:576:2] = NAN
    kv[13] = NAN
    kv[14, 575], kv[14, 512] = -top, 3e38
    return kv


def _k_cases(k, top):
    k[0, 0:32] = NAN
    k[1, 96:128] = NAN
    k[2, 5] = NAN
    k[3, 100] = NAN
    k[4, 40] = top
    k[5, 127] = -top
    k[6, 32:64] = top
    k[7, :64] = NAN
    k[8] = NAN
    k[9, 64:128] = -top
    k[10, 66], k[10, 3] = top, top
    return k


@pytest.mark.parametrize("top", [1.0, math.inf])    # NaN alone, and infinities beside it
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("k_offset", [0, 20, 64])
def test_non_finite_values_are_stored_as_the_plain_writer_stores_them(dsa, k_offset, layout, top):
    n = 17
    k, kv = _rows(k_offset, n)
    k, kv = _k_cases(k, top).to(torch.bfloat16), _kv_cases(kv, top).to(torch.bfloat16)
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(1))[:n].cuda()
    turns, _ = dsa.rope_turns(64)
    got = [dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)]
    want = [dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)]
    dsa.rope_quant_kv(k.cuda(), kv.cuda(), torch.zeros(n, dtype=torch.int32).cuda(), slots, *got, turns,
                      k_offset=k_offset, k_layout=layout, kv_layout=layout)
    dsa.quant_kv(_turned_at_zero(k.float(), k_offset, layout).to(torch.bfloat16).cuda(),
                 _turned_at_zero(kv.float(), 512, layout).to(torch.bfloat16).cuda(), slots, *want)
    assert dsa.device_status() == 0
    rec_g, rec_w = (c[1].cpu().numpy().reshape(64, 608)[slots.cpu().numpy()] for c in (got, want))
    for row in range(n):
        assert np.array_equal(rec_g[row, 576:596].view(np.uint32), rec_w[row, 576:596].view(np.uint32)), row
        assert np.array_equal(rec_g[row, :576], rec_w[row, :576]), row
    pg, pw = (c[0].cpu().numpy() for c in (got, want))
    rows = slots.cpu().numpy()
    for row in range(n):
        at = rows[row]
        assert np.array_equal(pg[8192 + 4 * at:8196 + 4 * at], pw[8192 + 4 * at:8196 + 4 * at]), row
        assert np.array_equal(pg[128 * at:128 * at + 128], pw[128 * at:128 * at + 128]), row


@pytest.mark.parametrize("h", [16, 64])
def test_a_row_of_nan_shows_in_attention(dsa, h):
    # positions other than 0: every turned value of a NaN row is NaN, and the attention over it too
    k, kv = _rows(7, 40)
    kv[17] = NAN
    cache, keys = dsa.alloc_kv_cache(1), dsa.alloc_k_cache(1)
    turns, amp = dsa.rope_turns(64, scaling="yarn", factor=4.0)
    pos = torch.arange(40, dtype=torch.int32)
    dsa.rope_quant_kv(k.to(torch.bfloat16).cuda(), kv.to(torch.bfloat16).cuda(), pos.cuda(), pos.long().cuda(), keys, cache,
                      turns, amplitude=amp)
    scales = cache.cpu().numpy().reshape(64, 608)[:, 576:596].copy().view(np.float32)
    assert np.isnan(scales[17]).all() and np.isfinite(np.delete(scales, 17, 0)).all()
    q = torch.randn(2, h, 576, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    one = torch.zeros(1, dtype=torch.int32).cuda()
    out, _ = dsa.prefix_attn(q, cache, None, 0, one[None], one + 40, one.repeat(2), torch.tensor([39, 16], dtype=torch.int32).cuda(),
                             64, 0.07)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    assert dsa.device_status() == 0
