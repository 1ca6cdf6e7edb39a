"""The per-head norm with rotation (norm_rope), its gradient and the norming cache writer against the formula
in 64 bits.

Tolerances, in units of 2^-24 (a rounding of fp32).  A lane adds at most 32 elements and a row at most 5 levels of
lanes, so a row's sum is off by at most 37 units of the sum of its terms' sizes; divided by the root mean
square the mean is off by 37 * mean|x - mu + mu| / sigma <= 37 (1 + |mu| / sigma), the factor by
(37 + 4) / 2 + 2 for the sum of squares, the product with 1 / n, eps, and 2 ulp (4 units) of rsqrt, and u takes two more.
With |mu| <= sigma here: |error of u| <= (74 + 27 |u|) units, of z = u w + b two more of |z|'s parts:
    err(z) <= 80 (|w| (1 + |u|) + |b|) =: 80 m.
The turn adds 8 units of |a| + |b| (test_gpu_rope), and both parts' errors.  A result of type T adds
half a step.  For the gradient, with g the gradient turned back (8 units of G = |dy| + |its partner|) and du = g w,
    err(dx) <= r 100 (G |w| + (1 + |u|) mean(G |w| (1 + |u|)) + mean(G |w|)),
each of the three a product of values with the errors above; a sum over rows adds one unit a row that a lane takes in
turn (here below 60) and 15 for the lanes, warps and blocks: err(dw) <= 200 sum G (1 + |u|), err(db) <= 200 sum G.
"""

import ctypes
import math

import pytest
import torch

from dsa_testlib import ensure_built

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


# ---- the formula -------------------------------------------------------------------------

def _phases(turns, pos):
    """cos, sin [n, rot / 2] in float64 from the exact integer phase."""
    frac = [[((int(p) * int(f)) % (1 << 64)) / 2.0 ** 64 for f in turns] for p in pos]
    angle = torch.tensor(frac, dtype=torch.float64).view(len(pos), len(turns)) * (2 * math.pi)
    return angle.cos()[:, None], angle.sin()[:, None]


def _pairs(rot, offset, layout):
    i = torch.arange(rot // 2)
    return (offset + i, offset + rot // 2 + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)


def _turn(y, turns, pos, offset, layout, amp, sign=1.0):
    c, s = _phases(turns, pos)
    i0, i1 = _pairs(2 * len(turns), offset, layout)
    z = y.clone()
    a, b = y[..., i0], y[..., i1]
    z[..., i0], z[..., i1] = amp * (a * c - sign * b * s), amp * (sign * a * s + b * c)
    return z


def _spread(m, turns, offset, layout, amp):
    """sizes m of a row's values: those of a turned pair, added up."""
    i0, i1 = _pairs(2 * len(turns), offset, layout)
    z = m.clone()
    z[..., i0] = z[..., i1] = abs(amp) * (m[..., i0] + m[..., i1])
    return z


def _unit(x, span, center, eps):
    u = x[..., :span]
    if center:
        u = u - u.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(u.square().mean(-1, keepdim=True) + eps)
    return u * r, r


def _ref(x, w, b, turns, pos, span, center, eps, offset, layout, amp):
    """x float64 [n, h, d] -> (y, its bound's size)."""
    u, _ = _unit(x, span, center, eps)
    z, m = torch.cat([u * w + b, x[..., span:]], -1), torch.cat([w.abs() * (1 + u.abs()) + b.abs(), x[..., span:].abs()], -1)
    return _turn(z, turns, pos, offset, layout, amp), _spread(m, turns, offset, layout, amp)


def _ref_grad(dy, x, w, turns, pos, span, center, eps, offset, layout, amp):
    g = _turn(dy, turns, pos, offset, layout, amp, -1.0)
    G = _spread(dy.abs(), turns, offset, layout, amp)
    u, r = _unit(x, span, center, eps)
    du, Gw = g[..., :span] * w, G[..., :span] * w.abs()
    dx = du - u * (du * u).mean(-1, keepdim=True) - (du.mean(-1, keepdim=True) if center else 0)
    bound = 100 * r * (Gw + (1 + u.abs()) * (Gw * (1 + u.abs())).mean(-1, keepdim=True) + Gw.mean(-1, keepdim=True))
    return (torch.cat([dx * r, g[..., span:]], -1), torch.cat([bound, 8 * G[..., span:]], -1),
            (g[..., :span] * u).sum((0, 1)), 200 * (G[..., :span] * (1 + u.abs())).sum((0, 1)),
            g[..., :span].sum((0, 1)), 200 * G[..., :span].sum((0, 1)))


def _inputs(n, h, d, span, rot, dtype, w_dtype, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, h, d + pad, generator=g) * 2 + 0.5).to(dtype)
    w = (1 + 0.3 * torch.randn(span, generator=g)).to(w_dtype)
    b = (0.2 * torch.randn(span, generator=g)).to(w_dtype)
    dy = torch.randn(n, h, d, generator=g).to(dtype)
    pos = torch.randint(-5, 1 << 20, (n,), generator=g, dtype=torch.int32)
    turns = torch.tensor([round(10000.0 ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64) for i in range(rot // 2)])
    return x, w, b, dy, pos, turns


def _close(got, want, bound, dtype):
    got = got.double().cpu()
    tol = HALF_STEP[dtype] * want.abs() + bound * U * (1 + HALF_STEP[dtype])
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half the spacing of subnormal results
    worst = ((got - want).abs() - tol).max()
    assert torch.isfinite(got).all() and worst <= 0, float(worst)


CASES = [
    # n, h, d, span, rot, offset, layout, norm, dtype, w_dtype, pad
    (1, 64, 128, 128, 64, 0, "half", "rms", torch.bfloat16, torch.float32, 0),
    (37, 64, 128, 128, 64, 0, "half", "rms", torch.bfloat16, torch.bfloat16, 0),
    (37, 64, 128, 128, 64, 0, "half", "layer", torch.bfloat16, torch.bfloat16, 0),
    (5, 3, 128, 128, 128, 0, "half", "rms", torch.float16, torch.float16, 0),
    (70, 1, 128, 128, 64, 64, "interleaved", "layer", torch.bfloat16, torch.float32, 0),
    (6, 5, 192, 128, 64, 128, "interleaved", "rms", torch.float32, torch.float32, 64),
    (9, 16, 576, 512, 64, 512, "interleaved", "rms", torch.bfloat16, torch.float32, 0),
    (3, 7, 576, 576, 64, 512, "half", "layer", torch.float32, torch.bfloat16, 0),
    (2, 3, 1024, 1024, 1024, 0, "half", "rms", torch.float32, torch.float32, 0),
    (2, 2, 1024, 1024, 1024, 0, "interleaved", "layer", torch.bfloat16, torch.float32, 0),
    (4, 9, 100, 100, 50, 0, "half", "rms", torch.bfloat16, torch.float32, 0),
    (4, 9, 100, 68, 50, 50, "interleaved", "layer", torch.float16, torch.float32, 4),
    (11, 2, 64, 64, 64, 0, "interleaved", "rms", torch.float32, torch.float16, 0),
    (5, 3, 77, 33, 30, 47, "half", "layer", torch.bfloat16, torch.float32, 3),
    (5, 3, 77, 33, 30, 20, "interleaved", "rms", torch.float32, torch.float32, 0),
    (3, 2, 1023, 1023, 2, 1021, "interleaved", "layer", torch.bfloat16, torch.float32, 0),
    (3, 2, 2, 1, 2, 0, "half", "rms", torch.float32, torch.float32, 0),
    (300, 3, 256, 256, 64, 192, "half", "rms", torch.bfloat16, torch.float32, 0),
    (2, 1, 514, 514, 64, 0, "half", "layer", torch.float16, torch.float32, 0),
    (6, 5, 256, 256, 64, 96, "half", "rms", torch.bfloat16, torch.float32, 0),
    (9, 4, 192, 128, 64, 128, "half", "layer", torch.float16, torch.float32, 8),
    (7, 3, 320, 320, 32, 288, "half", "rms", torch.bfloat16, torch.bfloat16, 0),
]
IDS = ["-".join(str(v).replace("torch.", "") for v in c) for c in CASES]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("how", ["fresh", "in place", "no bias", "no weight"])
def test_norm_rope(dsa, case, how):
    n, h, d, span, rot, offset, layout, norm, dtype, w_dtype, pad = case
    x, w, b, _, pos, turns = _inputs(n, h, d, span, rot, dtype, w_dtype, pad)
    amp, eps = 1.25, 1e-5
    wide = x.cuda()
    xg = wide[..., :d]
    kw = dict(norm=norm, norm_dim=span, eps=eps, offset=offset, layout=layout, amplitude=amp)
    weight, bias = (None if how == "no weight" else w.cuda()), (None if how in ("no bias", "no weight") else b.cuda())
    got = dsa.norm_rope(xg, pos.cuda(), turns.cuda(), weight, bias, out=xg if how == "in place" else None, **kw)
    want, m = _ref(x[..., :d].double(), torch.ones(span).double() if weight is None else w.double(),
                   torch.zeros(span).double() if bias is None else b.double(), turns.tolist(), pos.tolist(), span,
                   norm == "layer", eps, offset, layout, amp)
    _close(got, want, 96 * m, dtype)
    assert torch.equal(wide[..., d:].cpu(), x[..., d:])          # what lies between the rows
    if how != "in place":
        assert torch.equal(xg.cpu(), x[..., :d])


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("into", ["fresh", "dy", "x"])
def test_norm_rope_grad(dsa, case, into):
    n, h, d, span, rot, offset, layout, norm, dtype, w_dtype, pad = case
    x, w, b, dy, pos, turns = _inputs(n, h, d, span, rot, dtype, w_dtype, pad)
    amp, eps = 0.75, 1e-5
    xg, dyg = x.cuda()[..., :d], dy.cuda()
    dx, dw, db = dsa.norm_rope_grad(dyg, xg, pos.cuda(), turns.cuda(), w.cuda(), b.cuda(), norm=norm, norm_dim=span,
                                    eps=eps, offset=offset, layout=layout, amplitude=amp,
                                    dx={"fresh": None, "dy": dyg, "x": xg}[into])
    rdx, bdx, rdw, bdw, rdb, bdb = _ref_grad(dy.double(), x[..., :d].double(), w.double(), turns.tolist(), pos.tolist(),
                                             span, norm == "layer", eps, offset, layout, amp)
    _close(dx, rdx, bdx, dtype)
    _close(dw, rdw, bdw, torch.float32)
    _close(db, rdb, bdb, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_the_gradient_is_that_of_differences(dsa, norm):
    """Central differences of the 64-bit formula: with steps of 1e-4 of a value's size their own error is below 1e-7 of
    the gradient's size, far inside what the kernel's bound gives for the product with a direction."""
    n, h, d, span, rot, offset, layout = 7, 3, 96, 80, 32, 56, "half"
    x, w, b, dy, pos, turns = _inputs(n, h, d, span, rot, torch.float32, torch.float32, seed=3)
    args = (turns.tolist(), pos.tolist(), span, norm == "layer", 1e-6, offset, layout, 1.0)
    dx, dw, db = dsa.norm_rope_grad(dy.cuda(), x.cuda(), pos.cuda(), turns.cuda(), w.cuda(), b.cuda(), norm=norm,
                                    norm_dim=span, offset=offset, layout=layout)
    _, bdx, _, bdw, _, bdb = _ref_grad(dy.double(), x.double(), w.double(), *args)
    g = torch.Generator().manual_seed(4)
    f = lambda xx, ww, bb: (_ref(xx, ww, bb, *args)[0] * dy.double()).sum()  # noqa: E731
    for k, (value, got, bound) in enumerate(((x, dx, bdx), (w, dw, bdw), (b, db, bdb))):
        v = torch.randn(value.shape, generator=g, dtype=torch.float64)
        at = [x.double(), w.double(), b.double()]
        step = 1e-4 * v
        hi, lo = list(at), list(at)
        hi[k], lo[k] = at[k] + step, at[k] - step
        slope = (f(*hi) - f(*lo)) / 2e-4
        mine = (got.double().cpu() * v).sum()
        size = (got.double().cpu().abs() * v.abs()).sum()
        assert abs(mine - slope) <= (bound * U * v.abs()).sum() + 1e-7 * size


@pytest.mark.gpu
def test_equal_inputs_give_equal_gradients(dsa):
    x, w, b, dy, pos, turns = (t.cuda() for t in _inputs(513, 33, 128, 128, 64, torch.bfloat16, torch.float32))
    first = dsa.norm_rope_grad(dy, x, pos, turns, w, b, layout="half")
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, dsa.norm_rope_grad(dy, x, pos, turns, w, b, layout="half")))


@pytest.mark.gpu
def test_broadcast_rows(dsa):
    """Strides of 0: one key for all heads, one gradient for all tokens."""
    x, w, b, dy, pos, turns = _inputs(6, 4, 128, 128, 64, torch.float32, torch.float32)
    xb, dyb = x[:, :1].expand(6, 4, 128), dy[:1].expand(6, 4, 128)
    kw = dict(norm="layer", layout="half")
    got = dsa.norm_rope(x[:, :1].cuda().expand(6, 4, 128), pos.cuda(), turns.cuda(), w.cuda(), b.cuda(), **kw)
    args = (turns.tolist(), pos.tolist(), 128, True, 1e-6, 0, "half", 1.0)
    want, m = _ref(xb.double(), w.double(), b.double(), *args)
    _close(got, want, 96 * m, torch.float32)
    dx, dw, db = dsa.norm_rope_grad(dy[:1].cuda().expand(6, 4, 128), x[:, :1].cuda().expand(6, 4, 128), pos.cuda(),
                                    turns.cuda(), w.cuda(), b.cuda(), **kw)
    ref = _ref_grad(dyb.double(), xb.double(), w.double(), *args)
    for got, want, bound in ((dx, ref[0], ref[1]), (dw, ref[2], ref[3]), (db, ref[4], ref[5])):
        _close(got, want, bound, torch.float32)


@pytest.mark.gpu
def test_heads_before_tokens_and_two_dims(dsa):
    x, w, b, dy, pos, turns = _inputs(6, 4, 128, 128, 64, torch.bfloat16, torch.float32)
    xh = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    out = torch.empty(4, 6, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    a = dsa.norm_rope(x.cuda(), pos.cuda(), turns.cuda(), w.cuda(), b.cuda())
    assert torch.equal(dsa.norm_rope(xh, pos.cuda(), turns.cuda(), w.cuda(), b.cuda(), out=out), a)
    one = dsa.norm_rope(x[:, 2].cuda(), pos.cuda(), turns.cuda(), w.cuda(), b.cuda())
    assert torch.equal(one, a[:, 2])


@pytest.mark.gpu
def test_a_bad_row_stays_alone(dsa):
    x, w, b, dy, pos, turns = _inputs(40, 5, 128, 128, 64, torch.float32, torch.float32)
    run = lambda v: dsa.norm_rope(v.cuda(), pos.cuda(), turns.cuda(), w.cuda(), b.cuda(), layout="half").cpu()  # noqa: E731
    good = run(x)
    y = x.clone()
    y[3, 2, 7], y[8, 0, 100], y[39, 4, 0] = float("nan"), float("inf"), 1e25
    got = run(y)
    bad = torch.zeros(40, 5, dtype=torch.bool)
    bad[3, 2] = bad[8, 0] = bad[39, 4] = True
    assert torch.equal(got[~bad], good[~bad])
    assert torch.isnan(got[3, 2]).all()
    y = torch.zeros_like(x)              # rows of zeros: the bias, turned
    want, _ = _ref(y.double(), w.double(), b.double(), turns.tolist(), pos.tolist(), 128, False, 1e-6, 0, "half", 1.0)
    _close(run(y), want, 96 * (w.double().abs() + b.double().abs()) * 2, torch.float32)


@pytest.mark.gpu
def test_no_rows(dsa):
    x, w, b, dy, pos, turns = (t.cuda() for t in _inputs(4, 3, 64, 64, 64, torch.float32, torch.float32))
    for e in (x[:0], x[:, :0]):
        p = pos[:e.shape[0]]
        assert dsa.norm_rope(e, p, turns, w, b).shape == e.shape
        dx, dw, db = dsa.norm_rope_grad(e, e, p, turns, w, b)
        assert dx.shape == e.shape and not dw.any() and not db.any()


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph(dsa):
    x, w, b, dy, pos, turns = (t.cuda() for t in _inputs(50, 8, 128, 128, 64, torch.bfloat16, torch.float32))
    want = dsa.norm_rope(x, pos, turns, w, b)
    wdx, wdw, wdb = dsa.norm_rope_grad(dy, x, pos, turns, w, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = dsa.norm_rope(x, pos, turns, w, b, stream=side)
    d = dsa.norm_rope_grad(dy, x, pos, turns, w, b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(d, (wdx, wdw, wdb)))
    sx, sdy = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy = dsa.norm_rope(sx, pos, turns, w, b)
        gd = dsa.norm_rope_grad(sdy, sx, pos, turns, w, b)
    for k in (1.0, 2.0):                  # (a power of two: the normed rows are the same but for eps)
        sx.copy_(x * k)
        sdy.copy_(dy * k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, dsa.norm_rope(sx, pos, turns, w, b))
        assert all(torch.equal(p, q) for p, q in zip(gd, dsa.norm_rope_grad(sdy, sx, pos, turns, w, b)))
    assert torch.equal(gy, dsa.norm_rope(x * 2.0, pos, turns, w, b))


class _NormRope(torch.autograd.Function):
    """The two halves that the refusal points to."""

    @staticmethod
    def forward(ctx, dsa, x, w, b, pos, turns):
        ctx.dsa = dsa
        ctx.save_for_backward(x, w, b, pos, turns)
        return dsa.norm_rope(x, pos, turns, w, b, norm="layer")

    @staticmethod
    def backward(ctx, grad):
        x, w, b, pos, turns = ctx.saved_tensors
        dx, dw, db = ctx.dsa.norm_rope_grad(grad.contiguous(), x, pos, turns, w, b, norm="layer")
        return None, dx, dw.to(w.dtype), db.to(b.dtype), None, None


@pytest.mark.gpu
def test_in_the_halves_of_an_autograd_function(dsa):
    x, w, b, dy, pos, turns = (t.cuda() for t in _inputs(5, 3, 64, 64, 32, torch.float32, torch.float32))
    leaves = [t.requires_grad_() for t in (x, w, b)]
    for _ in range(2):                   # (the second backward adds to the first's)
        (_NormRope.apply(dsa, *leaves, pos, turns) * dy).sum().backward()
    ref = _ref_grad(dy.double().cpu(), x.detach().double().cpu(), w.detach().double().cpu(), turns.tolist(), pos.tolist(), 64,
                    True, 1e-6, 0, "interleaved", 1.0)
    for leaf, want, bound in zip(leaves, ref[::2], ref[1::2]):
        _close(leaf.grad, 2 * want, 2 * bound + 2 * want.abs(), torch.float32)


# ---- the writer --------------------------------------------------------------------------

def _e4m3(x):
    step = torch.exp2(((torch.frexp(x)[1] - 1).clamp(min=-6) - 3).double())
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _stored(cache_k, cache_kv, slots):
    pages = cache_k.cpu().view(-1, 8448)
    codes = pages[:, :8192].reshape(-1, 128)[slots].view(torch.float8_e4m3fn).double()
    scales = pages[:, 8192:].reshape(-1, 4)[slots].to(torch.int32)
    rec = cache_kv.cpu().view(-1, 608)[slots]
    return (codes, scales, rec[:, :576].contiguous().view(torch.float8_e4m3fn).double(),
            rec[:, 576:596].contiguous().view(torch.float32).double())


@pytest.mark.gpu
@pytest.mark.parametrize("n,k_norm,k_offset,k_layout,kv_layout,bias", [
    (1, "layer", 0, "half", "interleaved", True), (33, "rms", 64, "interleaved", "half", False),
    (200, "layer", 20, "interleaved", "interleaved", True), (200, "rms", 36, "half", "half", True)])
def test_norm_rope_quant_kv(dsa, n, k_norm, k_offset, k_layout, kv_layout, bias):
    """A code is the nearest of a value within 2^-20 of its own and its pair's size of the formula's, whose sizes are
    those of the bound above: 80 m + 8 units, below 2^-24 * 96 m <= 2^-17 m."""
    g = torch.Generator().manual_seed(n)
    k = (torch.randn(n, 140, generator=g) + 0.5).to(torch.bfloat16)
    kv = (torch.randn(n, 600, generator=g) * 3).to(torch.bfloat16)
    kw, kb, vw = (1 + 0.2 * torch.randn(128, generator=g)), 0.3 * torch.randn(128, generator=g), 1 + 0.2 * torch.randn(512, generator=g)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    turns, amp = dsa.rope_turns(64, scaling="yarn", factor=8.0, device="cpu")
    slots = torch.randperm(320, generator=g)[:n]
    skip = torch.arange(n) % 7 == 3
    kc, vc = dsa.alloc_k_cache(5), dsa.alloc_kv_cache(5)
    dsa.norm_rope_quant_kv(k.cuda()[:, :128], kv.cuda()[:, :576], pos.cuda(), torch.where(skip, -1, slots).cuda(), kc, vc,
                           turns.cuda(), kw.cuda(), kb.cuda() if bias else None, vw.cuda(), k_norm=k_norm, amplitude=amp,
                           k_offset=k_offset, k_layout=k_layout, kv_layout=kv_layout)
    assert dsa.device_status() == 0
    codes, e8, vcodes, vscales = _stored(kc, vc, slots[~skip])
    untouched = torch.ones(320, dtype=torch.bool)
    untouched[slots[~skip]] = False
    assert not vc.cpu().view(-1, 608)[untouched].any()
    pos, k, kv = pos[~skip].tolist(), k[~skip, None, :128].double(), kv[~skip, None, :576].double()
    b = kb.double() if bias else torch.zeros(128).double()
    y, m = _ref(k, kw.double(), b, turns.tolist(), pos, 128, k_norm == "layer", 1e-6, k_offset, k_layout, amp)
    y, d = y[:, 0], 96 * U * m[:, 0]
    grp = lambda t: t.view(len(pos), 4, 32).abs().amax(-1)  # noqa: E731
    top, dt = grp(y), grp(d)
    e_lo, e_hi = (torch.frexp(v)[1] - 9 for v in (top - dt, top + dt))
    e = e8 - 127
    assert ((e >= e_lo) & (e <= e_hi)).all()
    scale = torch.exp2(e.double()).repeat_interleave(32, -1)
    assert ((codes >= _e4m3((y - d) / scale)) & (codes <= _e4m3((y + d) / scale))).all()
    y, m = _ref(kv, vw.double(), torch.zeros(512).double(), turns.tolist(), pos, 512, False, 1e-6, 512, kv_layout, amp)
    y, d = y[:, 0], 96 * U * m[:, 0]
    for t in range(5):
        part = slice(128 * t, min(128 * t + 128, 576))
        top, dt = y[:, part].abs().amax(-1), d[:, part].amax(-1)
        s = vscales[:, t]
        assert ((s - top / 448).abs() <= (dt + U * top) / 448).all()
        yy, dd = y[:, part] / s[:, None], d[:, part] / s[:, None] + 4 * U * y[:, part].abs() / s[:, None]
        assert ((vcodes[:, part] >= _e4m3(yy - dd)) & (vcodes[:, part] <= _e4m3(yy + dd))).all()


@pytest.mark.gpu
def test_writer_rows_that_have_no_norm_and_zeros(dsa):
    g = torch.Generator().manual_seed(5)
    k, kv = torch.randn(4, 128, generator=g).to(torch.bfloat16), torch.randn(4, 576, generator=g).to(torch.bfloat16)
    k[0, 3], kv[0, 100] = float("nan"), float("inf")
    k[1], kv[1] = 0, 0
    kv[2, 513] = float("nan")            # in the part that is not normed
    turns, _ = dsa.rope_turns(64)
    kc, vc = dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)
    zero = torch.zeros(4, dtype=torch.int32).cuda()
    dsa.norm_rope_quant_kv(k.cuda(), kv.cuda(), zero, torch.arange(4).cuda(), kc, vc, turns)
    codes, e8, vcodes, vscales = _stored(kc, vc, torch.arange(4))
    assert torch.isnan(codes[0]).all() and torch.isfinite(codes[1:]).all()
    assert torch.isnan(vscales[0, :4]).all() and torch.isfinite(vscales[0, 4])
    assert not codes[1].any() and not vcodes[1].any() and not vscales[1].any()
    assert torch.isfinite(vcodes[2, :512]).all() and torch.isnan(vcodes[2, 512:]).any()
    # one of the two caches alone, the other half of the call left out
    k2, v2 = dsa.alloc_k_cache(1), dsa.alloc_kv_cache(1)
    dsa.norm_rope_quant_kv(k.cuda(), None, zero, torch.arange(4).cuda(), k2, None, turns)
    dsa.norm_rope_quant_kv(None, kv.cuda(), zero, torch.arange(4).cuda(), None, v2, turns)
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    dsa.norm_rope_quant_kv(k.cuda(), None, zero, torch.arange(61, 65).cuda(), k2, None, turns)
    assert dsa.status_names(dsa.device_status()) == ["BAD_PAGE"]


# ---- refusals (no GPU) -------------------------------------------------------------------

def _call(lib, **kw):
    a = dict(x=1, out=2, dtype=0, n=4, h=3, d=128, xt=384, xh=128, ot=384, oh=128, w=3, b=4, wd=2, span=128, center=0, eps=1e-6,
             pos=5, turns=6, rot=64, offset=0, layout=0, amp=1.0)
    a.update(kw)
    p = {k: None if a[k] is None else ctypes.c_void_p(int(a[k] * (1 << 20))) for k in ("x", "out", "w", "b", "pos", "turns")}
    return lib.dsa_norm_rope(p["x"], p["out"], a["dtype"], a["n"], a["h"], a["d"], a["xt"], a["xh"], a["ot"], a["oh"], p["w"],
                             p["b"], a["wd"], a["span"], a["center"], ctypes.c_float(a["eps"]), p["pos"], p["turns"], a["rot"],
                             a["offset"], a["layout"], ctypes.c_float(a["amp"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(h=-1), -1), (dict(dtype=3), -2), (dict(wd=-1), -2), (dict(d=1, span=1), -2), (dict(d=1025), -2),
    (dict(span=0), -1), (dict(span=129), -1), (dict(rot=0), -1), (dict(rot=63), -1), (dict(rot=130), -1),
    (dict(offset=65), -1), (dict(offset=-1), -1), (dict(layout=2), -1), (dict(center=2), -1), (dict(eps=-1e-6), -1),
    (dict(eps=math.nan), -1), (dict(eps=math.inf), -1), (dict(amp=math.nan), -1), (dict(n=1 << 16, h=1 << 15), -2),
    (dict(x=None), -1), (dict(out=None), -1), (dict(pos=None), -1), (dict(turns=None), -1),
    (dict(x=1 + 2.0 ** -20), -1), (dict(w=3 + 2.0 ** -19), -1), (dict(b=4 + 2.0 ** -20), -1), (dict(pos=5 + 2.0 ** -19), -1),
    (dict(xt=-1), -1), (dict(xt=1 << 40), -1), (dict(oh=100), -1), (dict(ot=256), -1), (dict(ot=0), -1),
    (dict(out=1, ot=512), -1), (dict(n=0), 0), (dict(h=0, x=None), 0)])
def test_norm_rope_refusals(dsa, kw, code):
    assert _call(dsa.lib(), **kw) == code
    if code:
        assert b"norm_rope:" in dsa.lib().dsa_last_error()


def test_norm_rope_grad_refusals(dsa):
    P, f = lambda v: ctypes.c_void_p(v << 20), ctypes.c_float  # noqa: E731
    good = [P(1), P(2), P(3), 0, 4, 3, 128, 384, 128, 384, 128, 384, 128, P(4), 2, 128, 0, f(1e-6), P(5), P(6), 64, 0, 0, f(1.0),
            P(7), P(8), P(9), 1 << 30, None]
    assert dsa.norm_rope_grad_workspace_size(128) > 0 and dsa.norm_rope_grad_workspace_size(0) == 0
    for at, bad in ((0, None), (2, None), (3, 7), (6, 2000), (15, 0), (26, None), (27, 16), (26, ctypes.c_void_p((9 << 20) + 64)),
                    (24, ctypes.c_void_p(2)), (7, -1), (11, 100), (2, P(1))):
        call = list(good)
        call[at] = bad
        if at == 2 and bad is not None:
            call[11] = 512               # in place over dy with other strides
        assert dsa.lib().dsa_norm_rope_grad(*call) < 0


def test_the_binding_refuses(dsa):
    x, pos, turns, w = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.int64), torch.ones(64)
    for bad in (x.double(), x[0, 0], x.to(torch.int32)):
        with pytest.raises(ValueError, match="x must be"):
            dsa.norm_rope(bad, pos, turns)
    for kw in (dict(weight=w[:63]), dict(weight=w.double()), dict(weight=w, bias=w.half()), dict(weight=w, norm_dim=32),
               dict(out=x[:1]), dict(norm="group"), dict(layout="x")):
        with pytest.raises(ValueError):
            dsa.norm_rope(x, pos, turns, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.norm_rope(x, pos, turns, weight=w)
    for leaf in ("x", "weight", "bias"):
        t = dict(x=x, weight=w, bias=w)
        t[leaf] = t[leaf].clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            dsa.norm_rope(t["x"], pos, turns, t["weight"], t["bias"])
        with pytest.raises(ValueError, match="gradient"):
            dsa.norm_rope_grad(x, t["x"], pos, turns, t["weight"], t["bias"])
    with pytest.raises(ValueError, match="dy must"):
        dsa.norm_rope_grad(x.half(), x, pos, turns)
    k, kv, s = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(2, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    kc = torch.zeros(8448, dtype=torch.uint8)
    with pytest.raises(ValueError, match="go together"):
        dsa.norm_rope_quant_kv(k, kv, pos, s, kc, None, turns)
    with pytest.raises(ValueError, match="must be given"):
        dsa.norm_rope_quant_kv(None, None, pos, s, kc, None, turns)
    with pytest.raises(ValueError, match="gradient"):
        dsa.norm_rope_quant_kv(k, None, pos, s, kc, None, turns, k_weight=torch.ones(128, requires_grad=True))
