"""The accuracy that the header of norm_rope_quant_kv promises, derived from its arithmetic in units of 2^-24.

The factor: squares and their sums take 8 roundings (a key: 4 dims a lane, five exchanges) or 14 (a latent row: chains of
8), the product with 1 / n and eps one, halved by the root, rsqrt 4: 9 or 11.5.  The normed value takes two more and its
bias one of the result: 12 (key), 13.5 (latent) of |u w| + |b|.  The sines are good to 8 units, the turn takes two:
22 < 2^-19 of a key's own and its pair's sizes; the latent row's quotient takes two: 15.5 < 2^-20, which is below it; its
scales one: 14.5 < 2^-20.  With a mean its sum takes 7 roundings: 7 units < 2^-21 of mean|x| / sigma |w|, and the difference one
of |u w|, which the 2^-19 have room for.  The turned 64 dims of a latent row: 10 units of the pair's sizes, two for the quotient."""

import math

import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_norm_rope import _e4m3, _spread, _stored, _turn, _unit

N = 4096


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _inside(codes, y, d, scale):
    return bool(((codes >= _e4m3((y - d) / scale)) & (codes <= _e4m3((y + d) / scale))).all())


@pytest.mark.gpu
@pytest.mark.parametrize("k_norm,mean", [("rms", 0.0), ("layer", 0.0), ("layer", 2.0), ("layer", -90.0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_codes_and_scales(dsa, k_norm, mean, layout):
    g = torch.Generator().manual_seed(int(abs(mean)) + len(layout))
    k = (torch.randn(N, 128, generator=g) + mean).to(torch.bfloat16)
    kv = (torch.randn(N, 576, generator=g) * 3).to(torch.bfloat16)
    kw, kb = 1 + 0.2 * torch.randn(128, generator=g), 0.3 * torch.randn(128, generator=g)
    vw = 1 + 0.2 * torch.randn(512, generator=g)
    pos = torch.randint(0, 1 << 20, (N,), generator=g, dtype=torch.int32)
    turns, amp = dsa.rope_turns(64, scaling="yarn", factor=8.0, device="cpu")
    kc, vc = dsa.alloc_k_cache(N // 64), dsa.alloc_kv_cache(N // 64)
    dsa.norm_rope_quant_kv(k.cuda(), kv.cuda(), pos.cuda(), torch.arange(N).cuda(), kc, vc, turns.cuda(), kw.cuda(), kb.cuda(),
                           vw.cuda(), k_norm=k_norm, amplitude=amp, k_layout=layout, kv_layout=layout)
    codes, e8, vcodes, vscales = _stored(kc, vc, torch.arange(N))
    k, kv, turns, pos = k.double()[:, None], kv.double()[:, None], turns.tolist(), pos.tolist()
    u, r = _unit(k, 128, k_norm == "layer", 1e-6)
    y = _turn(u * kw.double() + kb.double(), turns, pos, 0, layout, amp)[:, 0]
    size = 2.0 ** -19 * ((u * kw.double()).abs() + kb.double().abs())
    if k_norm == "layer":
        size = size + 2.0 ** -21 * kw.double().abs() * k.abs().mean(-1, keepdim=True) * r
    d = _spread(size, turns, 0, layout, amp)[:, 0]
    grp = lambda t: t.view(N, 4, 32).amax(-1)  # noqa: E731
    top, far = grp(y.abs() - d), grp(y.abs() + d)
    e = e8 - 127
    assert ((e >= torch.frexp(top)[1] - 9) & (e <= torch.frexp(far)[1] - 9)).all()
    assert _inside(codes, y, d, torch.exp2(e.double()).repeat_interleave(32, -1))
    u, _ = _unit(kv, 512, False, 1e-6)
    z = torch.cat([u * vw.double(), kv[..., 512:]], -1)
    y = _turn(z, turns, pos, 512, layout, amp)[:, 0]
    d = 2.0 ** -20 * _spread(z.abs(), turns, 512, layout, amp)[:, 0]
    for t in range(5):
        part = slice(128 * t, min(128 * t + 128, 576))
        s, top = vscales[:, t:t + 1], y[:, part].abs().amax(-1, keepdim=True)
        slack = d[:, part].amax(-1, keepdim=True) if t == 4 else 2.0 ** -20 * top
        assert ((s - top / 448).abs() <= slack / 448 + 2.0 ** -24 * s).all()
        assert _inside(vcodes[:, part], y[:, part], d[:, part], s)


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [-30, -36, -45, -55])
@pytest.mark.parametrize("sign", [1, -1])
def test_small_angles_of_any_bits(dsa, exponent, sign):
    """Sines alone in their group (keys zero in the part that meets the cosines), of angles of 2^exponent turns and any
    lower bits, on both sides of 0: good to 2^-19 of their own."""
    n = 64
    g = torch.Generator().manual_seed(-exponent)
    k = torch.randn(n, 128, generator=g).to(torch.bfloat16)
    k[:, 32:64] = 0
    turns = sign * torch.randint(1 << (63 + exponent), 1 << (64 + exponent), (32,), generator=g)
    kc = dsa.alloc_k_cache(1)
    dsa.norm_rope_quant_kv(k.cuda(), None, torch.ones(n, dtype=torch.int32).cuda(), torch.arange(n).cuda(), kc, None, turns.cuda())
    codes, e8, _, _ = _stored(kc, dsa.alloc_kv_cache(1), torch.arange(n))
    u, _ = _unit(k.double(), 128, False, 1e-6)
    y = u[:, :32] * torch.sin(2 * math.pi * turns.double() * 2.0 ** -64)
    top, e = y.abs().amax(-1), e8[:, 1] - 127
    assert ((e >= torch.frexp(top * (1 - 2.0 ** -19))[1] - 9) & (e <= torch.frexp(top * (1 + 2.0 ** -19))[1] - 9)).all()
    assert _inside(codes[:, 32:64], y, 2.0 ** -19 * y.abs(), torch.exp2(e.double())[:, None])
