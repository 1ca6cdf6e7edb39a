"""Rotary positions (rope) and the rotating cache writers (rope_quant_kv) against the
formula in 64 bits.

Tolerances.  rope computes in fp32: the phase is exact but for 2^-31 of a half turn and its
rounding to fp32 (at most 2^-25 relative of a value below 1, times pi: 9.4e-8 rad), the
sine and cosine add about an ulp (2^-23 of values up to 1), the amplitude's product, the
table's product and the final sum three roundings of 2^-24 each.  Against
m = amplitude (|a| + |b|) that is below 9.4e-8 + 1.2e-7 + 3 * 6e-8 = 4e-7 =: FP32; a bf16 or
fp16 result adds half a step, eps / 2 of its value, and a subnormal fp16 result half of 2^-24.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from dsa_testlib import ensure_built

FP32 = 4e-7


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _phase(turns, pos):
    """cos, sin of every position and frequency, in float64 from the exact integer phase."""
    out = np.empty((len(pos), len(turns)))
    for i, p in enumerate(pos):
        for j, f in enumerate(turns):
            x = (int(p) * int(f)) % (1 << 64)
            out[i, j] = (x - (1 << 64) if x >= 1 << 63 else x) / 2.0 ** 64 * 2 * math.pi
    return np.cos(out), np.sin(out)


def _ref(x, turns, pos, offset, layout, amplitude, sign=1.0):
    """x float64 [n, h, d] turned; returns (y, m): m the size the tolerance is relative to."""
    c, s = _phase(turns, pos)
    c, s = amplitude * c[:, None], amplitude * sign * s[:, None]
    y, m = x.copy(), np.zeros_like(x)
    half = len(turns)
    i = np.arange(half)
    i0, i1 = (offset + i, offset + half + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    m[..., i0] = m[..., i1] = abs(amplitude) * (np.abs(a) + np.abs(b))
    return y, m


def _table(rot, seed=0, base=10000.0):
    return [round(base ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64) for i in range(rot // 2)]


# ---- the table (no GPU) ------------------------------------------------------------------

def test_turns_are_the_frequencies():
    import dsa_sparse_attention_topk_gb300 as dsa
    t, amp = dsa.rope_turns(64, device="cpu")
    assert amp == 1.0 and t.dtype == torch.int64
    f = t.double().numpy() / 2.0 ** 64 * 2 * math.pi
    np.testing.assert_allclose(f, 10000.0 ** (-np.arange(32) / 32.0), rtol=1e-12)


def test_scaled_tables():
    import dsa_sparse_attention_topk_gb300 as dsa
    f = lambda **kw: dsa.rope_turns(64, device="cpu", **kw)[0].double().numpy()  # noqa: E731
    plain = f()
    np.testing.assert_allclose(f(scaling="linear", factor=8.0), plain / 8, rtol=1e-12)
    ntk = f(scaling="ntk", factor=8.0)
    assert ntk[0] == plain[0]
    np.testing.assert_allclose(ntk[-1], plain[-1] / 8, rtol=1e-9)
    yarn, amp = dsa.rope_turns(64, scaling="yarn", factor=40.0, device="cpu")
    yarn = yarn.double().numpy()
    assert abs(amp - (0.1 * math.log(40.0) + 1)) < 1e-12
    turns_made = plain / 2.0 ** 64 * 4096           # turns in the original 4096 positions
    assert np.array_equal(yarn[turns_made > 64], plain[turns_made > 64])
    np.testing.assert_allclose(yarn[turns_made < 0.5], plain[turns_made < 0.5] / 40, rtol=1e-12)
    assert np.all(np.diff(yarn) < 0)
    # f (1 - r) + f r: at most four roundings of 2^-53
    np.testing.assert_allclose(f(scaling="yarn", factor=1.0), plain, rtol=4 * 2.0 ** -53)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(rot=64, base=1.0), dict(rot=64, factor=0.5),
                                dict(rot=64, scaling="other"), dict(rot=2, scaling="ntk", factor=2.0),
                                dict(rot=64, scaling="yarn", beta_fast=1.0, beta_slow=2.0)])
def test_table_refusals(kw):
    import dsa_sparse_attention_topk_gb300 as dsa
    with pytest.raises(ValueError):
        dsa.rope_turns(device="cpu", **kw)


# ---- refusals of the C entries (no GPU) -----------------------------------------------------

def _rope_call(lib, **kw):
    from ctypes import c_float, c_void_p as P
    a = dict(x=1, out=2, dtype=0, n=2, h=3, d=64, xt=192, xh=64, ot=192, oh=64, pos=3, turns=4, rot=64, offset=0,
             layout=0, amp=1.0, transpose=0, shift=0)
    a.update(kw)
    p = lambda v: None if v is None else P(v * 65536)  # noqa: E731
    x = P(a["x"] * 65536 + a["shift"]) if a["x"] is not None else None
    return lib.dsa_rope(x, p(a["out"]), a["dtype"], a["n"], a["h"], a["d"], a["xt"], a["xh"], a["ot"], a["oh"],
                        p(a["pos"]), p(a["turns"]), a["rot"], a["offset"], a["layout"], c_float(a["amp"]),
                        a["transpose"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(dtype=3), -2), (dict(d=1), -2), (dict(rot=3), -1), (dict(rot=66), -1), (dict(rot=0), -1),
    (dict(offset=2), -1), (dict(offset=-2), -1), (dict(layout=2), -1), (dict(amp=float("nan")), -1),
    (dict(amp=float("inf")), -1), (dict(x=None), -1), (dict(pos=None), -1), (dict(turns=None), -1), (dict(shift=1), -1),
    (dict(ot=128), -1), (dict(oh=63), -1), (dict(xt=-192), -1), (dict(ot=0), -1), (dict(x=2, xt=256), -1),
    (dict(n=1 << 16, h=1 << 15), -2),
])
def test_rope_rejects_bad_arguments(dsa, kw, code):
    assert _rope_call(dsa.lib(), **kw) == code
    assert dsa.lib().dsa_last_error()


def _append_call(lib, **kw):
    from ctypes import c_float, c_void_p as P
    a = dict(k=1, ks=128, kv=2, kvs=576, pos=3, slots=4, n=2, kc=5, kvc=6, num_slots=64, turns=7, amp=1.0, k_offset=0,
             kl=1, kvl=0, shift=0)
    a.update(kw)
    p = lambda v, s=0: None if v is None else P(v * 65536 + s)  # noqa: E731
    return lib.dsa_rope_quant_kv(p(a["k"], a["shift"]), a["ks"], p(a["kv"]), a["kvs"], p(a["pos"]), p(a["slots"]),
                                 a["n"], p(a["kc"]), p(a["kvc"]), a["num_slots"], p(a["turns"]), c_float(a["amp"]),
                                 a["k_offset"], a["kl"], a["kvl"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(k_offset=2), -1), (dict(k_offset=68), -1), (dict(k_offset=-4), -1), (dict(kl=2), -1),
    (dict(kvl=-1), -1), (dict(amp=float("nan")), -1), (dict(k=None, kv=None), -1), (dict(kc=None), -1),
    (dict(kvc=None), -1), (dict(pos=None), -1), (dict(slots=None), -1), (dict(turns=None), -1), (dict(shift=4), -1),
    (dict(ks=130), -1), (dict(kvs=-576), -1), (dict(num_slots=63), -1), (dict(num_slots=0), -1),
    (dict(n=0, k=None, kv=None), 0),
])
def test_rope_quant_kv_rejects_bad_arguments(dsa, kw, code):
    assert _append_call(dsa.lib(), **kw) == code


def test_python_refusals(dsa):
    x, pos, t = torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    for bad in (lambda: dsa.rope(x, pos, t), lambda: dsa.rope(x.double(), pos, t),
                lambda: dsa.rope(x[0], pos, t), lambda: dsa.rope(x, pos, t, out=x[:1]),
                lambda: dsa.rope_quant_kv(None, None, pos, pos.long(), None, None, t),
                lambda: dsa.rope_quant_kv(x.bfloat16(), None, pos, pos.long(), None, None, t)):
        with pytest.raises(ValueError):
            bad()


# ---- rope on the GPU ----------------------------------------------------------------------

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check(got, x, turns, pos, offset, layout, amplitude, sign=1.0):
    ref, m = _ref(x.double().cpu().numpy(), turns, pos.cpu().numpy(), offset, layout, amplitude, sign)
    g = got.double().cpu().numpy()
    half_step = 0.0 if x.dtype == torch.float32 else torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    tol = m * FP32 + half_step * (np.abs(ref) + m * FP32) + tiny * (m > 0)
    assert np.all(np.abs(g - ref) <= tol), np.max(np.abs(g - ref) / (tol + 1e-30))
    rot = 2 * len(turns)
    rest = np.r_[0:offset, offset + rot:x.shape[-1]]
    assert np.array_equal(g[..., rest], x.double().cpu().numpy()[..., rest])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,h,d,rot,offset,pad", [
    (1, 1, 64, 64, 0, 0), (1, 64, 128, 64, 0, 0), (7, 128, 576, 64, 512, 0), (33, 5, 128, 64, 64, 64),
    (3, 3, 100, 50, 50, 0),       # nothing divides 16 bytes: the element-wise path
    (5, 2, 128, 32, 3, 0),        # the rotary part off any vector boundary
    (9, 3, 192, 128, 64, 4),      # row strides that break (bf16) or keep (fp32) 16-byte rows
    (2, 1, 2, 2, 0, 0), (4, 2, 2304, 2048, 256, 0),
    (2000, 63, 128, 64, 64, 0),   # several rows a thread (from 311296 items), rows crossing tokens
    (500, 63, 100, 50, 50, 0), (500, 63, 101, 36, 3, 0), (700, 63, 130, 64, 2, 0), (900, 63, 128, 64, 64, 4),  # and narrow
])
def test_rope_matches_the_formula(dsa, n, h, d, rot, offset, pad, dtype, layout):
    g = torch.Generator().manual_seed(n * 1000 + d + rot)
    base = torch.randn(n, h, d + pad, generator=g).to(DT[dtype]).cuda()
    x = base[..., :d]
    pos = torch.randint(-5, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
    turns = _table(rot)
    t = torch.tensor(turns, dtype=torch.int64).cuda()
    for transpose in (False, True):
        y = dsa.rope(x, pos, t, offset=offset, layout=layout, amplitude=1.25, transpose=transpose)
        _check(y, x, turns, pos, offset, layout, 1.25, -1.0 if transpose else 1.0)
    # in place: the same values, and nothing beside the rotary part is touched
    keep = base.clone()
    y = dsa.rope(x, pos, t, offset=offset, layout=layout, amplitude=1.25, out=x, transpose=True)
    assert y is x and torch.equal(base[..., d:], keep[..., d:])
    assert torch.equal(x, dsa.rope(keep[..., :d], pos, t, offset=offset, layout=layout, amplitude=1.25,
                                   transpose=True))


@pytest.mark.gpu
@pytest.mark.parametrize("pos", [0, 1, 131071, (1 << 31) - 1, -(1 << 31), -1])
def test_far_and_negative_positions(dsa, pos):
    turns = _table(64) + [1 << 62, -(1 << 63), (1 << 63) - 1, 0]  # and quarter, half and no turns a position
    x = torch.randn(1, 2, 72, generator=torch.Generator().manual_seed(1)).cuda()
    p = torch.tensor([pos], dtype=torch.int32).cuda()
    for layout in ("interleaved", "half"):
        y = dsa.rope(x, p, torch.tensor(turns, dtype=torch.int64).cuda(), layout=layout)
        _check(y, x, turns, p, 0, layout, 1.0)


@pytest.mark.gpu
def test_rope_is_its_own_adjoint_and_matches_differences(dsa):
    # <R x, g> = <x, R^T g>, and the difference quotient of <R x, g> along v is <R v, g>
    g = torch.Generator().manual_seed(5)
    x, w, v = (torch.randn(6, 4, 96, generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 65536, (6,), generator=g, dtype=torch.int32).cuda()
    t, amp = dsa.rope_turns(64, scaling="yarn", factor=40.0)
    for layout in ("interleaved", "half"):
        f = lambda a, tr=False: dsa.rope(a, pos, t, offset=16, layout=layout, amplitude=amp,  # noqa: E731
                                         transpose=tr).double()
        grad = f(w, True)
        # 2304 products, each off by at most FP32 of sizes a few units large
        tol = 2304 * FP32 * 8
        assert abs(float((f(x) * w).sum() - (grad * x).sum())) < tol
        # linear, so a step of 1/16 (exact in fp32) has no truncation error
        d = (f(x + v / 16) - f(x - v / 16)) * 8
        assert abs(float((d * w).sum() - (grad * v).sum())) < 16 * 2 * tol


@pytest.mark.gpu
def test_memory_orders_broadcasts_and_two_dims(dsa):
    g = torch.Generator().manual_seed(6)
    turns = _table(64)
    t = torch.tensor(turns, dtype=torch.int64).cuda()
    pos = torch.randint(0, 65536, (5,), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(3, 5, 128, generator=g).to(torch.bfloat16).cuda().transpose(0, 1)  # heads first in memory
    want = dsa.rope(x.contiguous(), pos, t, offset=64)
    assert torch.equal(dsa.rope(x, pos, t, offset=64), want)
    out = torch.empty(3, 5, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(dsa.rope(x, pos, t, offset=64, out=out), want)
    one = x[:, :1].expand(5, 4, 128)             # one head read by four
    assert torch.equal(dsa.rope(one, pos, t, offset=64), want[:, :1].expand(5, 4, 128))
    two = x[:, 1]
    assert torch.equal(dsa.rope(two, pos, t, offset=64), want[:, 1])
    with pytest.raises(dsa.DsaError):
        dsa.rope(one.contiguous(), pos, t, offset=64, out=one)   # four heads written over one
    assert dsa.rope(x[:0], pos[:0], t).shape == (0, 3, 128)


@pytest.mark.gpu
def test_rope_passes_non_finite_values_of_their_own_pair_only(dsa):
    t = torch.tensor(_table(64), dtype=torch.int64).cuda()
    x = torch.ones(1, 1, 128).cuda()
    x[0, 0, 6], x[0, 0, 100] = float("nan"), float("inf")
    y = dsa.rope(x, torch.ones(1, dtype=torch.int32).cuda(), t)
    bad = ~torch.isfinite(y[0, 0])
    assert bad.nonzero().flatten().tolist() == [6, 7, 100]


# ---- rope_quant_kv on the GPU -----------------------------------------------------------

def _tokens(n, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(n, 128 + pad, generator=g).to(torch.bfloat16)
    kv = torch.randn(n, 576 + pad, generator=g).to(torch.bfloat16)
    k[0], kv[0] = 0, 0
    if n > 3:
        k[1] *= 2.0 ** -60
        kv[1] *= 2.0 ** 40
        kv[2, 512:] = 0
        k[2, ::3] = 0
    pos = torch.randint(0, 1 << 18, (n,), generator=g, dtype=torch.int32)
    return k.cuda()[:, :128], kv.cuda()[:, :576], pos.cuda()


def _rows(kc, vc, slots):
    pages = kc.cpu().numpy().reshape(-1, 8448)
    kcodes = pages[:, :8192].reshape(-1, 128)[slots]
    kscale = pages[:, 8192:].reshape(-1, 4)[slots]
    rec = vc.cpu().numpy().reshape(-1, 608)[slots]
    return kcodes, kscale, rec[:, :576], rec[:, 576:596].copy().view(np.float32), rec[:, 596:]


def _quantised_within(value, codes, scale, x, slack):
    """value = decoded code * scale is x rounded to E4M3 at this scale: half a step of 2^-3
    relative (2^-9 of the scale among the subnormals; saturation cuts at 448), around an x known
    to `slack`."""
    v = np.minimum(np.abs(x) / scale, 448.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(v, 1e-30))), -6) - 3)
    over = np.maximum(np.abs(x) - 448.0 * scale, 0)     # cut by saturation
    return np.abs(value - x) <= step / 2 * scale * (1 + 1e-6) + over + slack


@pytest.mark.gpu
@pytest.mark.parametrize("n,pad,k_offset,k_layout,kv_layout", [
    (1, 0, 0, "half", "interleaved"), (64, 0, 64, "interleaved", "half"), (130, 64, 20, "half", "half"),
    (1000, 4, 32, "interleaved", "interleaved"), (30000, 0, 0, "half", "interleaved"),
])
def test_append_matches_the_formula(dsa, n, pad, k_offset, k_layout, kv_layout):
    k, kv, pos = _tokens(n, n, pad)
    t, amp = dsa.rope_turns(64, scaling="yarn", factor=40.0)
    pages = n // 64 + 2
    slots = torch.randperm(pages * 64, generator=torch.Generator().manual_seed(n))[:n]
    skip = torch.zeros(n, dtype=torch.bool)
    skip[3::7] = True
    kc, vc = dsa.alloc_k_cache(pages), dsa.alloc_kv_cache(pages)
    kc.fill_(0xAB)
    vc.fill_(0xAB)
    dsa.rope_quant_kv(k, kv, pos, torch.where(skip, torch.tensor(-1), slots).cuda(), kc, vc, t, amplitude=amp,
                      k_offset=k_offset, k_layout=k_layout, kv_layout=kv_layout)
    assert dsa.device_status() == 0
    take = np.nonzero(~skip.numpy())[0]
    if n > 2000:
        take = take[:: len(take) // 500]
    kcodes, kscale, vcodes, vscale, pad_ = _rows(kc, vc, slots.numpy()[take])
    assert not pad_.any()
    turns, p = t.cpu().tolist(), pos.cpu().numpy()[take]
    # the key: turned dims to the formula; its other groups exactly as the oracle has them
    x = k.double().cpu().numpy()[take]
    y, m = _ref(x[:, None], turns, p, k_offset, k_layout, amp)
    y, m = y[:, 0], m[:, 0]
    ks = np.exp2(kscale.astype(np.float64) - 127)
    value = oracle.mxfp8_dequantize(kcodes, kscale)
    assert np.all(_quantised_within(value, kcodes, np.repeat(ks, 32, 1), y, FP32 * m))
    amax = np.abs(y).reshape(-1, 4, 32).max(-1)
    slack = (FP32 * m).reshape(-1, 4, 32).max(-1)
    low = np.where(amax > slack, np.floor(np.log2(np.maximum(amax - slack, 1e-300))) - 8 + 127, 0)
    high = np.where(amax > 0, np.floor(np.log2(np.maximum(amax + slack, 1e-300))) - 8 + 127, 127)
    assert np.all((kscale >= np.minimum(low, high)) & (kscale <= high))
    c_ref, s_ref = oracle.mxfp8_quantize(x)
    for g in range(4):
        if 32 * g + 32 <= k_offset or 32 * g >= k_offset + 64:
            assert np.array_equal(kcodes[:, 32 * g:32 * g + 32], c_ref[:, 32 * g:32 * g + 32])
            assert np.array_equal(kscale[:, g], s_ref[:, g])
    # the latent row: four tiles exactly, the rope tile to the formula
    x = kv.double().cpu().numpy()[take]
    c_ref, s_ref = oracle.fp8_tile_quantize(x)
    assert np.array_equal(vcodes[:, :512], c_ref[:, :512])
    assert np.array_equal(vscale[:, :4].view(np.uint32), s_ref[:, :4].view(np.uint32))
    y, m = _ref(x[:, None], turns, p, 512, kv_layout, amp)
    y, m = y[:, 0, 512:], m[:, 0, 512:]
    amax = np.abs(y).max(1)
    assert np.all(np.abs(vscale[:, 4] - amax / 448) <= (FP32 * m.max(1) + amax * 2.0 ** -24) / 448)
    value = oracle.codecs.e4m3_decode(vcodes[:, 512:]) * vscale[:, 4:].astype(np.float64)
    safe = np.where(vscale[:, 4:] > 0, vscale[:, 4:], 1).astype(np.float64)
    assert np.all(_quantised_within(value, vcodes, safe, y, FP32 * m))
    # slots of skipped tokens, and every other one, are as they were
    free = np.setdiff1d(np.arange(pages * 64), slots.numpy()[~skip.numpy()])
    kcodes, kscale, vcodes, _, pad_ = _rows(kc, vc, free)
    assert np.all(kcodes == 0xAB) and np.all(kscale == 0xAB) and np.all(vcodes == 0xAB) and np.all(pad_ == 0xAB)


@pytest.mark.gpu
def test_append_at_position_zero_is_the_plain_writer(dsa):
    k, kv, _ = _tokens(200, 9)
    slots = torch.randperm(256)[:200].cuda()
    t, _ = dsa.rope_turns(64)
    a = [dsa.alloc_k_cache(4), dsa.alloc_kv_cache(4)]
    b = [dsa.alloc_k_cache(4), dsa.alloc_kv_cache(4)]
    dsa.rope_quant_kv(k, kv, torch.zeros(200, dtype=torch.int32).cuda(), slots, *a, t)
    dsa.quant_kv(k.contiguous(), kv.contiguous(), slots, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # one cache at a time gives the same bytes
    c = [dsa.alloc_k_cache(4), dsa.alloc_kv_cache(4)]
    p = torch.arange(200, dtype=torch.int32).cuda()
    dsa.rope_quant_kv(k, None, p, slots, c[0], None, t)
    dsa.rope_quant_kv(None, kv, p, slots, None, c[1], t)
    dsa.rope_quant_kv(k, kv, p, slots, *a, t)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@pytest.mark.gpu
def test_append_flags_slots_behind_the_cache(dsa):
    k, kv, pos = _tokens(3, 10)
    t, _ = dsa.rope_turns(64)
    kc, vc = dsa.alloc_k_cache(1), dsa.alloc_kv_cache(2)      # the smaller cache bounds the slots
    vc.fill_(7)
    slots = torch.tensor([64, -1, 1 << 40], dtype=torch.int64).cuda()
    dsa.rope_quant_kv(k, kv, pos, slots, kc, vc, t)
    assert dsa.device_status() & 1
    assert not kc.any() and bool((vc == 7).all())


@pytest.mark.gpu
def test_rotary_calls_on_a_side_stream_and_in_a_graph(dsa):
    k, kv, pos = _tokens(40, 11)
    t, _ = dsa.rope_turns(64)
    slots = torch.arange(40).cuda()
    want = [dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)]
    dsa.rope_quant_kv(k, kv, pos, slots, *want, t)
    q = torch.randn(40, 8, 128).to(torch.bfloat16).cuda()
    wq = dsa.rope(q, pos, t)
    got = [dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)]
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        dsa.rope_quant_kv(k, kv, pos, slots, *got, t)
        dsa.rope(q, pos, t, out=out)
    assert not out.any()
    for step in range(2):   # a replay reads what the tensors hold then
        if step:
            pos.add_(1000)
            dsa.rope_quant_kv(k, kv, pos, slots, *want, t)
            wq = dsa.rope(q, pos, t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wq) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
