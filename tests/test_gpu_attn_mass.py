"""Accumulated attention weights (attn_mass, sparse_attn_mass) against the formula in 64 bits.

Tolerance of a weight e^(l - lse).  With S = sm_scale sum |q||kv|: the products are exact (codes of 4 bits, queries of 8);
an accumulator of 128 of them is taken in 8 steps, each adding with an error of 2^-23 of what it holds at most, so below
2^-20 of its products' sizes; the five scales' products and sums add 6 roundings of 2^-24, the factor's 4.  That is 2^-20 S
+ 10 * 2^-24 S <= 2^-19 S on the logit.  l - lse is formed with one rounding, lse's change of base with two: 2^-22 (|l| +
|lse|).  ex2 is good to 2^-22.  Sums of up to 48 columns a chunk and a few hundred chunks: 400 * 2^-24 of their terms.  So
    |error of w| <= w (2^-19 S + 2^-22 (|l| + |lse| + 1) + 400 * 2^-24),
summed over heads and rows, and for accumulated weights half a unit (2^-37) for each part, of which there are no more than
columns.
"""

import ctypes
import math

import pytest
import torch

from dsa_testlib import ensure_built

SM = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _records(n, g, scale=1.0):
    """n FP8 records of normal values, uint8 [n, 608], and their dequantised values [n, 576] in float64."""
    x = torch.randn(n, 640, generator=g) * scale
    x[:, 576:] = 0
    t = x.view(n, 5, 128)
    s = t.abs().amax(-1) / 448.0
    codes = (t / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    rec = torch.zeros(n, 608, dtype=torch.uint8)
    rec[:, :576] = codes.view(n, 640)[:, :576].view(torch.uint8)
    rec[:, 576:596] = s.contiguous().view(torch.uint8).view(n, 20)
    return rec, _values(rec)


def _values(rec):
    codes = rec[:, :576].contiguous().view(torch.float8_e4m3fn).double()
    s = rec[:, 576:596].contiguous().view(torch.float32).double()
    return codes * s.repeat_interleave(128, -1)[:, :576]


class Case:
    """Sequences over a shuffled pool, rows in any order."""

    def __init__(self, rows, lens, h, seed, max_ctx=None, q_scale=1.0, kv_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.h, self.lens, n_seq = h, torch.tensor(lens, dtype=torch.int32), len(lens)
        self.max_ctx = max_ctx or max(max(lens), 1)
        per = (self.max_ctx + 63) // 64
        self.pages = n_seq * per + 1
        self.rec, self.kv = _records(self.pages * 64, g, kv_scale)
        self.table = torch.randperm(self.pages, generator=g)[:n_seq * per].view(n_seq, per).to(torch.int32)
        seq = torch.tensor([b for b, r in enumerate(rows) for _ in range(r)], dtype=torch.int32)
        self.q_seq = seq[torch.randperm(len(seq), generator=g)]
        self.q_pos = (torch.rand(len(seq), generator=g) * (self.lens[self.q_seq.long()] + 2)).to(torch.int32) - 1
        self.q = (torch.randn(len(seq), h, 576, generator=g) * q_scale).to(torch.bfloat16)
        self.g = g

    def row(self, b):
        """Values of sequence b by position."""
        p = torch.arange(int(self.lens[b]))
        return self.kv[self.table[b].long()[p // 64] * 64 + p % 64]

    def terms(self, t, kv):
        """(logits [h, m], sizes S [h, m]) of row t over the values kv [m, 576]."""
        q = self.q[t].double()
        return SM * (q @ kv.T), SM * (q.abs() @ kv.abs().T)

    def lse(self, pick):
        """fp32 log-sum-exps of every row over its positions pick(t)."""
        out = torch.full((len(self.q), self.h), -math.inf)
        for t in range(len(self.q)):
            p = pick(t)
            if len(p):
                out[t] = torch.logsumexp(self.terms(t, self.row(int(self.q_seq[t]))[p])[0], -1).float()
        return out

    def weights(self, t, p, lse):
        """Row t's weights at positions p, and their bounds."""
        if not len(p):
            return torch.zeros(0).double(), torch.zeros(0).double()
        l, size = self.terms(t, self.row(int(self.q_seq[t]))[p])
        base = lse[t].double()[:, None]
        w = torch.exp(l - base)
        w = torch.where(torch.isneginf(base), torch.zeros_like(w), w)
        rel = 2.0 ** -19 * size + 2.0 ** -22 * (l.abs() + base.abs().nan_to_num(0, 0, 0) + 1) + 400 * 2.0 ** -24
        return w.sum(0), (w * rel).sum(0)

    def seen(self, t):
        n = int(self.lens[int(self.q_seq[t])])
        return torch.arange(max(0, min(int(self.q_pos[t]) + 1, n)))

    def dense(self, lse):
        mass = torch.zeros(len(self.lens), self.max_ctx).double()
        tol = torch.zeros_like(mass)
        for t in range(len(self.q)):
            b, p = int(self.q_seq[t]), self.seen(t)
            w, e = self.weights(t, p, lse)
            mass[b, p] += w
            tol[b, p] += e + 2.0 ** -37 * self.h
        return mass, tol

    def cuda(self):
        return {k: getattr(self, k).cuda() for k in ("q", "table", "lens", "q_seq", "q_pos")} | {"cache": self.rec.view(-1).cuda()}


def _dense(dsa, c, lse, **kw):
    d = c.cuda()
    return dsa.attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], d["q_pos"], lse.cuda(), c.max_ctx, SM, **kw)


def _float(mass):
    return mass.cpu().double() * 2.0 ** -36


DENSE = [
    # rows of each sequence, lengths, heads
    ([1], [1], 1),
    ([1], [257], 16),
    ([1, 1, 1], [130, 1, 64], 128),
    ([1, 0, 2, 0], [0, 300, 129, 5], 64),
    ([3, 1, 7], [128, 200, 383], 5),
    ([40], [500], 16),
    ([2, 2, 2], [200, 250, 90], 128),
    ([9], [330], 128),
    ([1] * 20, list(range(1, 200, 10)), 33),
    ([0, 70], [10, 140], 100),
    ([1], [20000], 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,lens,h", DENSE, ids=[f"{sum(r)}x{h}-{max(n)}" for r, n, h in DENSE])
def test_dense(dsa, rows, lens, h):
    c = Case(rows, lens, h, seed=h + sum(lens))
    lse = c.lse(c.seen)
    got = _dense(dsa, c, lse)
    assert dsa.device_status() == 0
    want, tol = c.dense(lse)
    assert ((_float(got) - want).abs() <= tol).all()
    again = _dense(dsa, c, lse, mass=got.clone())     # added once more: the same whole numbers
    assert torch.equal(again, 2 * got)


@pytest.mark.gpu
def test_dense_with_queries_and_values_of_all_sizes(dsa):
    """Queries down to 2^-40 of one another and tiny or large scales; lse shifted so that weights stay in range."""
    for q_scale, kv_scale in ((2.0 ** -60, 2.0 ** 55), (2.0 ** 40, 2.0 ** -42), (1.0, 2.0 ** -20)):
        c = Case([2, 1], [150, 140], 7, seed=3, q_scale=q_scale, kv_scale=kv_scale)
        c.q[..., ::3] *= 2.0 ** -20
        c.q[..., 1::3] *= 2.0 ** -40
        lse = c.lse(c.seen)
        want, tol = c.dense(lse)
        assert ((_float(_dense(dsa, c, lse)) - want).abs() <= tol).all()


@pytest.mark.gpu
def test_dense_wide_rows_of_mass_and_longer_tables(dsa):
    c = Case([2, 3], [100, 180], 16, seed=8, max_ctx=200)
    lse = c.lse(c.seen)
    wide = torch.full((2, 700), 5, dtype=torch.int64).cuda()
    mass = wide[:, 100:350]
    assert _dense(dsa, c, lse, mass=mass) is mass
    want, tol = c.dense(lse)
    assert ((_float(mass[:, :200] - 5) - want).abs() <= tol).all()
    mass[:, :200] = 5
    assert (wide == 5).all()


@pytest.mark.gpu
def test_dense_rows_and_positions_that_do_not_count(dsa):
    c = Case([3, 3, 2], [200, 300, 130], 16, seed=11)
    lse = c.lse(c.seen)
    bad_code, bad_scale, bad_page = 37, 150, 2
    b = 1
    slot = lambda p: int(c.table[b, p // 64]) * 64 + p % 64  # noqa: E731
    c.rec[slot(bad_code), 100] = 0x7F                         # NaN
    c.rec[slot(bad_scale), 580:584] = torch.tensor([math.inf]).view(torch.uint8)
    want, tol = c.dense(lse)                                   # (of the values before)
    want[b, [bad_code, bad_scale]] = 0
    want[b, 64 * bad_page:64 * bad_page + 64] = 0
    lse2, q = lse.clone(), c.q.clone()
    t = int((c.q_pos >= 1).nonzero()[0])
    w, e = c.weights(t, c.seen(t), lse)
    one = Case.weights(c, t, c.seen(t), torch.where(torch.arange(16) == 4, lse, torch.tensor(math.inf)))[0]
    lse2[t, 4] = math.nan
    seq = int(c.q_seq[t])
    p = c.seen(t)
    if seq == b:
        keep = [int(x) not in (bad_code, bad_scale) and int(x) // 64 != bad_page for x in p]
        one = torch.where(torch.tensor(keep), one, 0.0)
    want[seq, p] -= one
    d = c.cuda()
    d["table"][b, bad_page] = c.pages + 7
    q_seq = torch.cat([d["q_seq"], torch.tensor([-1, 3], dtype=torch.int32).cuda()])
    more = torch.cat([d["q"], d["q"][:2]])
    q_pos = torch.cat([d["q_pos"], torch.tensor([50, 50], dtype=torch.int32).cuda()])
    lse2 = torch.cat([lse2, lse2[:2]]).cuda()
    got = dsa.attn_mass(more, d["cache"], d["table"], d["lens"], q_seq, q_pos, lse2, c.max_ctx, SM)
    assert set(dsa.status_names(dsa.device_status())) == {"BAD_PAGE", "BAD_SEQ", "NAN_SCORE"}
    assert ((_float(got) - want).abs() <= tol + 1e-300).all()
    lens = d["lens"].clone()
    lens[2] = c.max_ctx + 1
    got = dsa.attn_mass(d["q"], d["cache"], d["table"], lens, d["q_seq"], d["q_pos"], lse.cuda(), c.max_ctx, SM)
    assert "BAD_LEN" in dsa.status_names(dsa.device_status()) and not got[2].any()


@pytest.mark.gpu
def test_dense_infinite_query_and_lse(dsa):
    c = Case([2], [100], 8, seed=2)
    c.q_pos[:] = torch.tensor([99, 60])
    lse = c.lse(c.seen)
    lse[0, 1], lse[0, 2] = math.inf, -math.inf                 # no weight either way
    c2 = Case([2], [100], 8, seed=2)
    c2.q_pos = c.q_pos
    c2.q[0, 5, 17] = math.inf
    none = lse.clone()
    none[0, 5] = math.inf
    want, tol = c.dense(none)
    assert ((_float(_dense(dsa, c2, lse)) - want).abs() <= tol).all()
    assert dsa.status_names(dsa.device_status()) == ["NAN_SCORE"]


SPARSE = [
    # rows of each sequence, lengths, heads, topk, fewest entries
    ([1], [1], 1, 1, 0),
    ([1], [400], 16, 100, 100),
    ([1, 2, 1], [130, 300, 64], 128, 64, 3),
    ([2, 2], [600, 700], 64, 257, 0),
    ([30], [500], 5, 130, 90),
    ([1] * 9, [150] * 9, 100, 128, 0),
    ([3], [3000], 32, 2048, 2048),
]


def _entries(c, topk, fewest):
    idx = torch.full((len(c.q), topk), -1, dtype=torch.int32)
    for t in range(len(c.q)):
        n = int(c.lens[int(c.q_seq[t])])
        k = min(n, topk)
        k = int(torch.randint(min(fewest, k), k + 1, (1,), generator=c.g))
        at = torch.randperm(topk, generator=c.g)[:k] if t % 2 else torch.arange(k)   # gaps, or none
        idx[t, at] = torch.randperm(n, generator=c.g)[:k].to(torch.int32)
    return idx


def _sparse_want(c, idx, lse):
    w, e = torch.zeros(idx.shape).double(), torch.zeros(idx.shape).double()
    mass, tol = torch.zeros(len(c.lens), c.max_ctx).double(), torch.zeros(len(c.lens), c.max_ctx).double()
    for t in range(len(c.q)):
        at = ((idx[t] >= 0) & (idx[t] < c.lens[int(c.q_seq[t])])).nonzero()[:, 0]
        w[t, at], e[t, at] = c.weights(t, idx[t, at].long(), lse)
        mass.index_put_((c.q_seq[t].long().expand(len(at)), idx[t, at].long()), w[t, at], accumulate=True)
        tol.index_put_((c.q_seq[t].long().expand(len(at)), idx[t, at].long()), e[t, at] + 2.0 ** -37, accumulate=True)
    return w, e, mass, tol


@pytest.mark.gpu
@pytest.mark.parametrize("rows,lens,h,topk,fewest", SPARSE, ids=[f"{sum(c[0])}x{c[2]}-{c[3]}" for c in SPARSE])
def test_sparse(dsa, rows, lens, h, topk, fewest):
    c = Case(rows, lens, h, seed=topk + h)
    idx = _entries(c, topk, fewest)
    lse = c.lse(lambda t: idx[t][idx[t] >= 0].long())
    d = c.cuda()
    args = (d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx.cuda(), lse.cuda(), SM)
    mass = torch.zeros(len(lens), c.max_ctx, dtype=torch.int64).cuda()
    got = dsa.sparse_attn_mass(*args, mass=mass)
    assert dsa.device_status() == 0
    w, e, want, tol = _sparse_want(c, idx, lse)
    assert ((got.cpu().double() - w).abs() <= e).all()
    assert ((_float(mass) - want).abs() <= tol).all()
    out = torch.full(idx.shape, 7.0).cuda()
    assert dsa.sparse_attn_mass(*args, out=out) is out and torch.equal(out, got)      # without mass
    dsa.sparse_attn_mass(*args, mass=mass)
    assert torch.equal(mass, 2 * torch.round(mass.double() / 2).long())               # (every part twice)


@pytest.mark.gpu
def test_sparse_entries_twice_behind_the_end_and_on_bad_pages(dsa):
    c = Case([2, 1], [200, 100], 16, seed=4)
    idx = torch.tensor([[5, 199, 5, 7, -1, 150, 99, 5], [0, 1, 1, 2, 3, 64, 65, -7], [99, 5, 5, 64, 70, 2, 1, 0]], dtype=torch.int32)
    lse = torch.full((3, 16), 4.0)
    w, e, want, tol = _sparse_want(c, idx, lse)
    over = idx.clone()
    long_rows = (c.q_seq == 0).nonzero()[:, 0]
    over[over == -1] = 200                                       # at the end of the longer sequence
    d = c.cuda()
    mass = torch.zeros(2, c.max_ctx, dtype=torch.int64).cuda()
    got = dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], over.cuda(), lse.cuda(), SM, mass=mass)
    assert dsa.status_names(dsa.device_status()) == ["BAD_INDEX"] and len(long_rows) == 2
    assert ((got.cpu().double() - w).abs() <= e).all() and ((_float(mass) - want).abs() <= tol).all()
    d["table"][:, 1] = -1
    got = dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx.cuda(), lse.cuda(), SM).cpu()
    assert dsa.status_names(dsa.device_status())[0] == "BAD_PAGE"
    gone = (idx >= 64) & (idx < 128)
    assert not got[gone].any() and ((got.double() - w).abs() <= e)[~gone].all()


@pytest.mark.gpu
def test_sparse_nan_position_shows_in_the_weights_alone(dsa):
    c = Case([1], [100], 8, seed=6)
    c.rec[int(c.table[0, 0]) * 64 + 9, 3] = 0xFF
    idx = torch.arange(20, dtype=torch.int32)[None]
    lse = torch.full((1, 8), 3.0)
    d = c.cuda()
    mass = torch.zeros(1, 100, dtype=torch.int64).cuda()
    got = dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx.cuda(), lse.cuda(), SM, mass=mass)
    assert torch.isnan(got[0, 9]) and torch.isfinite(got[0, :9]).all() and torch.isfinite(got[0, 10:]).all()
    assert int(mass[0, 9]) == 0 and (mass[0, :9] > 0).all()
    assert dsa.status_names(dsa.device_status()) == ["NAN_SCORE"]


@pytest.mark.gpu
def test_a_cache_beyond_32_bits(dsa):
    """Pages 4.5 GB into the cache."""
    c = Case([1], [130], 16, seed=7)
    far, pages = 115000, 115010
    cache = torch.zeros(pages * 64 * 608, dtype=torch.uint8, device="cuda")
    cache.view(-1, 608)[far * 64:(far + c.pages) * 64] = c.rec.cuda()
    lse = c.lse(c.seen)
    d = c.cuda()
    got = dsa.attn_mass(d["q"], cache, d["table"] + far, d["lens"], d["q_seq"], d["q_pos"], lse.cuda(), c.max_ctx, SM)
    want, tol = c.dense(lse)
    assert ((_float(got) - want).abs() <= tol).all()


@pytest.mark.gpu
def test_streams_and_graphs(dsa):
    """Two streams adding to one accumulator, and a captured call replayed with other inputs."""
    c = Case([3, 5], [300, 280], 16, seed=12)
    lse = c.lse(c.seen)
    one = _dense(dsa, c, lse)
    d = c.cuda()
    args = (d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], d["q_pos"])
    lse = lse.cuda()
    mass = torch.zeros_like(one)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            dsa.attn_mass(*args, lse, c.max_ctx, SM, mass=mass, stream=s)
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(mass, 8 * one)
    fresh = dsa.attn_mass(*args, lse, c.max_ctx, SM, stream=sides[0])
    torch.cuda.current_stream().wait_stream(sides[0])
    assert torch.equal(fresh, one)
    static = lse.clone()
    idx = torch.randint(0, 280, (8, 70), dtype=torch.int32).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gm = dsa.attn_mass(*args, static, c.max_ctx, SM)
        gw = dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx, static, SM)
    for shift in (0.0, 1.5):
        static.copy_(lse + shift)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gm, dsa.attn_mass(*args, static, c.max_ctx, SM))
        assert torch.equal(gw, dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx, static, SM))


@pytest.mark.gpu
def test_the_weights_of_an_attention_that_ran(dsa):
    """Behind prefix_attn and sparse_attn, with their log-sum-exps: every row's weights add up to its heads, but for
    what those hold of their own roundings (sparse_attn: 6e-3 at most, prefix_attn's fp16 operands 1e-3)."""
    c = Case([4, 2], [400, 333], 64, seed=13)
    d = c.cuda()
    lse = torch.empty(6, 64).cuda()
    dsa.prefix_attn(d["q"], d["cache"], None, 0, d["table"], d["lens"], d["q_seq"], d["q_pos"], c.max_ctx, SM, out_lse=lse)
    mass = _float(dsa.attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], d["q_pos"], lse, c.max_ctx, SM))
    for b in range(2):
        rows = int(((c.q_seq == b) & (c.q_pos >= 0)).sum())
        assert abs(float(mass[b].sum()) - 64 * rows) <= 1e-3 * 64 * rows
    idx = torch.stack([torch.randperm(333, generator=c.g)[:100] for _ in range(6)]).to(torch.int32).cuda()
    dsa.sparse_attn(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx, SM, out_lse=lse)
    w = dsa.sparse_attn_mass(d["q"], d["cache"], d["table"], d["lens"], d["q_seq"], idx, lse, SM)
    assert ((w.sum(1) - 64).abs() <= 64 * 6e-3).all()


# ---- refusals (no GPU) -------------------------------------------------------------------

def _p(v):
    return None if v is None else ctypes.c_void_p(int(v * 65536))


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(n_q=-1), -1), (dict(n_seq=-1), -1), (dict(h=0), -2), (dict(h=129), -2), (dict(n_q=65537), -2), (dict(ctx=0), -2),
    (dict(ctx=1 << 21, max_pages=1 << 20), -2), (dict(max_pages=3), -1), (dict(pages=0), -1), (dict(sm=0.0), -1),
    (dict(sm=math.inf), -1), (dict(stride=199), -1), (dict(stride=(1 << 40) + 1), -1), (dict(n_seq=0), -1), (dict(q=None), -1),
    (dict(cache=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(q_seq=None), -1), (dict(lse=None), -1),
    (dict(pick=None), -1), (dict(mass=None, out=None), -1), (dict(ws=None), -1), (dict(ws_bytes=100), -1),
    (dict(ws=9 + 2.0 ** -9), -1), (dict(q=1 + 2.0 ** -13), -1), (dict(mass=7 + 2.0 ** -14), -1), (dict(lse=6 + 2.0 ** -15), -1),
    (dict(n_seq=65537), -2), (dict(n_q=0, q=None), 0)])
def test_refusals(dsa, sparse, kw, code):
    a = dict(q=1, n_q=4, h=16, cache=2, pages=20, table=3, max_pages=4, lens=4, n_seq=2, q_seq=5, pick=10, topk=8, ctx=200, sm=SM,
             lse=6, mass=7, stride=200, out=8, ws=9, ws_bytes=1 << 30)
    a.update(kw)
    head = (_p(a["q"]), a["n_q"], a["h"], _p(a["cache"]), a["pages"], _p(a["table"]), a["max_pages"], _p(a["lens"]), a["n_seq"],
            _p(a["q_seq"]), _p(a["pick"]))
    tail = (_p(a["ws"]), a["ws_bytes"], None)
    if sparse:
        rc = dsa.lib().dsa_sparse_attn_mass(*head, a["topk"], a["ctx"], ctypes.c_float(a["sm"]), _p(a["lse"]), _p(a["mass"]),
                                            a["stride"], _p(a["out"]), *tail)
    else:
        rc = dsa.lib().dsa_attn_mass(*head, a["ctx"], ctypes.c_float(a["sm"]), _p(a["lse"]), _p(a["mass"]), a["stride"], *tail)
    assert rc == code


def test_the_binding_refuses(dsa):
    z = torch.zeros(1, dtype=torch.int32)
    q, cache, lse = torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(608 * 64, dtype=torch.uint8), torch.zeros(1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.attn_mass(q, cache, z[None], z, z, z, lse, 64, SM)
    with pytest.raises(ValueError, match="gradient"):
        dsa.attn_mass(q.clone().requires_grad_(), cache, z[None], z, z, z, lse, 64, SM)
    with pytest.raises(ValueError, match="gradient"):
        dsa.sparse_attn_mass(q, cache, z[None], z, z, z[None], lse.clone().requires_grad_(), SM)
    with pytest.raises(ValueError, match="must be"):
        dsa.sparse_attn_mass(q[0], cache, z[None], z, z, z[None], lse, SM)
    with pytest.raises(ValueError, match="columns"):
        dsa.attn_mass(q, cache, z[None], z, z, z, lse, 64, SM, mass=torch.zeros(1, 63, dtype=torch.int64))
    assert dsa.attn_mass_workspace_size(0, 16, 1) == 0 and dsa.attn_mass_workspace_size(4, 16, 1) > 4 * 16 * 1152
