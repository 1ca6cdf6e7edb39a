"""The rotating writers' codes and rope's small sines to the last bit that the formula gives.

float64 throughout: the phase is the exact integer product, so an angle is off by 2^-53 of itself, and a
value by some 2^-51.  The kernel knows a value to 2^-41 of its pair's size where that matters; some
2^-10 of the 2^26 values here lie so close to a border between two codes."""

import math

import numpy as np
import pytest
import torch

import oracle
from dsa_testlib import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _cos_sin(turns, pos):
    phase = (pos.astype(np.int64)[:, None] * turns[None]).astype(np.float64)     # wraps at a whole turn
    angle = phase * (2.0 * math.pi / 2.0 ** 64)
    return np.cos(angle), np.sin(angle)


def _turned(x, turns, pos, layout):
    """x [n, 64] float64."""
    c, s = _cos_sin(turns, pos)
    i = np.arange(32)
    i0, i1 = (i, 32 + i) if layout == "half" else (2 * i, 2 * i + 1)
    y = np.empty_like(x)
    y[:, i0], y[:, i1] = x[:, i0] * c - x[:, i1] * s, x[:, i0] * s + x[:, i1] * c
    return y


def _e4m3(x):
    """Nearest E4M3 values, ties to even, of values within +-448 (a little above: saturated)."""
    e = np.maximum(np.frexp(np.where(x == 0, 1.0, x))[1] - 1, -6)
    step = np.exp2(e - 3.0)
    return np.clip(np.round(x / step) * step, -448, 448)


def _written(dsa, seed, k_layout, kv_layout):
    n = 65536
    g = torch.Generator().manual_seed(100 * seed + len(k_layout))
    k = torch.randn(n, 128, generator=g).to(torch.bfloat16)
    kv = torch.randn(n, 576, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 18, (n,), generator=g, dtype=torch.int32)
    turns, _ = dsa.rope_turns(64)
    kc, vc = dsa.alloc_k_cache(n // 64), dsa.alloc_kv_cache(n // 64)
    dsa.rope_quant_kv(k.cuda(), kv.cuda(), pos.cuda(), torch.arange(n).cuda(), kc, vc, turns, k_layout=k_layout,
                      kv_layout=kv_layout)
    assert dsa.device_status() == 0
    return n, k.double().numpy(), kv.double().numpy(), turns.cpu().numpy(), pos.numpy(), kc.cpu().numpy(), vc.cpu().numpy()


SEEDS = pytest.mark.parametrize("seed", range(4))
LAYOUTS = pytest.mark.parametrize("k_layout,kv_layout", [("half", "interleaved"), ("interleaved", "half")])


@SEEDS
@LAYOUTS
def test_every_code_of_a_keys_turned_dims(dsa, seed, k_layout, kv_layout):
    n, k, _, turns, pos, cache, _ = _written(dsa, seed, k_layout, kv_layout)
    y = _turned(k[:, :64], turns, pos, k_layout).reshape(n, 2, 32)
    e = np.frexp(np.abs(y).max(-1, keepdims=True))[1] - 9
    page = cache.reshape(-1, 8448)
    got = oracle.codecs.e4m3_decode(page[:, :8192].reshape(n, 128)[:, :64]).reshape(n, 2, 32)
    want = _e4m3(y * np.exp2(-1.0 * e))
    assert np.array_equal(page[:, 8192:].reshape(n, 4)[:, :2], (e[..., 0] + 127).astype(np.uint8))
    assert np.array_equal(got, want), np.argwhere(got != want)


@SEEDS
@LAYOUTS
def test_every_code_of_a_turned_tile(dsa, seed, k_layout, kv_layout):
    n, _, kv, turns, pos, _, cache = _written(dsa, seed, k_layout, kv_layout)
    y = _turned(kv[:, 512:], turns, pos, kv_layout)
    scale = (np.abs(y).max(1, keepdims=True) / 448).astype(np.float32).astype(np.float64)
    rec = cache.reshape(n, 608)
    got, want = oracle.codecs.e4m3_decode(rec[:, 512:576]), _e4m3(y / scale)
    assert np.array_equal(got, want), np.argwhere(got != want)
    # (the stored scale: the fp32 rotation's 4 roundings, and the quotient's)
    mine = rec[:, 592:596].copy().view(np.float32).astype(np.float64)
    assert np.all(np.abs(mine - scale) <= 5 * 2.0 ** -24 * scale)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d", [64, 66])
def test_small_angles_keep_their_relative_accuracy(dsa, layout, d):
    # (a, 0) becomes (a cos, a sin): no other term hides what the sine has lost.  fp32: the angle, the
    # sine, its product with a (and with 1, the amplitude): 5 roundings of 2^-24 at most
    pos = torch.tensor([1, 2, 3, 7, 100, 1000, -1, -5], dtype=torch.int32)
    turns, _ = dsa.rope_turns(64)
    x = torch.zeros(len(pos), 5, d)
    i = np.arange(32)
    i0, i1 = (i, 32 + i) if layout == "half" else (2 * i, 2 * i + 1)
    x[..., i0] = torch.randn(len(pos), 5, 32, generator=torch.Generator().manual_seed(d))
    y = dsa.rope(x.cuda(), pos.cuda(), turns, layout=layout).double().cpu().numpy()
    c, s = _cos_sin(turns.cpu().numpy(), pos.numpy())
    a = x[..., i0].double().numpy()
    assert np.abs(y[..., i1] / (a * s[:, None]) - 1).max() <= 5 * 2.0 ** -24
    assert np.abs(y[..., i0] / (a * c[:, None]) - 1).max() <= 5 * 2.0 ** -24
