"""rope's small sines, from the exact integer phase in float64 (off by 2^-53 of itself)."""

import math

import numpy as np
import pytest
import torch

from dsa_testlib import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _cos_sin(turns, pos):
    phase = (pos.astype(np.int64)[:, None] * turns[None]).astype(np.float64)     # wraps at a whole turn
    angle = phase * (2.0 * math.pi / 2.0 ** 64)
    return np.cos(angle), np.sin(angle)


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
