"""Attention of a batch that shares a prefix (prefix_attn) against the formula in 64 bits.

The reference reads the cache's own bytes.  Gates for o against the float64 attention over the
latent rows, rounded to 11 significant bits for more than 32 heads, as the fp16 operands are then:

* per value: a weight (with up to 32 heads: times its position's scale) is rounded to fp16 (2^-11
  of it, or 2^-25 of the row's largest if subnormal), a split's partial result to fp16 (2^-11),
  the result to bf16 (2^-8); the logits carry the rounding of 576 fp32 additions,
  sm_scale sum|q kv| 576 2^-24 =: D, which moves a weight by up to 2 D of it, and the hardware 2^x
  2^-21 of it.  With S = sum_j p_j |v_j| over n positions
  |o - ref| <= (2^-11 + 2^-11 + 2 D + 2^-20) S + n 2^-25 max|v| + 2^-8 |ref|;
* per call: those roundings are independent of each other, one of at most 2^-8 of a value and so
  2^-8 / sqrt(3) in the mean square, the others far smaller, so the 2-norm of the difference stays
  below 2^-8 of the result's.

On the ordinary inputs the second gate also holds against the unrounded rows: 11 bits move a
logit by some 2^-11.  lse within 1e-4 of the rounded reference (the sparse attention's gate).
"""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from dsa_testlib import ensure_built, LSE_BF16_ATOL

SM = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def round11(x):
    """float64 rounded to 11 significant bits, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 2048.0) / 2048.0, e)


class Batch:
    """Sequences that share the pages of a prefix; lens: each one's length."""

    def __init__(self, dsa, lens, prefix, h, rows=None, seed=0, max_ctx=None, kv=None, q=None, extra_pages=0):
        g = torch.Generator().manual_seed(seed)
        self.prefix, self.h = prefix, h
        self.max_ctx = max_ctx or max(max(lens), prefix, 1)
        per = (self.max_ctx + 63) // 64
        whole, n = prefix // 64, len(lens)
        npg = (prefix + 63) // 64
        pages = npg + n * (per - whole) + extra_pages
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.empty(n, per, dtype=torch.int32)
        self.table[:, :whole] = perm[:whole]
        if per > whole:
            self.table[:, whole:] = perm[npg:npg + n * (per - whole)].view(n, per - whole)
        self.pages = perm[:npg].clone()     # the prefix's partial page is one of its own
        self.num_pages = pages
        vals = torch.randn(pages * 64, 576, generator=g) if kv is None else kv(pages * 64, g)
        self.cache = dsa.alloc_kv_cache(pages)
        dsa.quant_kv_fp8(vals.to(torch.bfloat16).cuda(), torch.arange(pages * 64).cuda(), self.cache)
        if rows is None:
            rows = [(b, L - 1) for b, L in enumerate(lens)]
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.q_seq = torch.tensor([r[0] for r in rows], dtype=torch.int32)
        self.q_pos = torch.tensor([r[1] for r in rows], dtype=torch.int32)
        self.q = (torch.randn(len(rows), h, 576, generator=g) if q is None else q(len(rows), g)).to(torch.bfloat16)

    def call(self, dsa, **kw):
        n = self.q.shape[0]
        ws = torch.full((dsa.prefix_attn_workspace_size(n, self.h, len(self.lens), self.prefix, self.max_ctx),), 0xFF,
                        dtype=torch.uint8, device="cuda")   # NaN everywhere: nothing may come from it
        out = torch.full((n, self.h, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n, self.h), float("nan"), device="cuda")
        table = self.table.cuda() if self.max_ctx > self.prefix else None
        pages = self.pages.cuda() if self.prefix else None
        dsa.prefix_attn(self.q.cuda(), self.cache, pages, self.prefix, table, self.lens.cuda(), self.q_seq.cuda(),
                        self.q_pos.cuda(), self.max_ctx, SM, out=out, out_lse=lse, workspace=ws, **kw)
        return out, lse

    def rows64(self, b):
        """The dequantised latent rows of sequence b as the call sees them, and which of them count."""
        rec = self.cache.cpu().numpy().reshape(-1, 608)
        p = np.arange(self.max_ctx)
        pages = np.where(p < self.prefix, np.r_[self.pages.numpy(), np.zeros(1, np.int32)][np.minimum(
            p // 64, len(self.pages))], self.table.numpy()[b][p // 64])
        ok = (pages >= 0) & (pages < self.num_pages)
        r = rec[np.where(ok, pages, 0).astype(np.int64) * 64 + p % 64]
        return oracle.fp8_tile_dequantize(r[:, :576], r[:, 576:596].copy().view(np.float32)), ok

    def check(self, out, lse, unrounded=False):
        o, e = out.double().cpu().numpy(), lse.double().cpu().numpy()
        err2 = ref2 = raw2 = 0.0
        for t in range(self.q.shape[0]):
            b, pos = int(self.q_seq[t]), int(self.q_pos[t])
            good = 0 <= b < len(self.lens) and 0 <= int(self.lens[b]) <= self.max_ctx
            n = max(0, min(pos + 1, int(self.lens[b]))) if good else 0
            kv, ok = self.rows64(b) if good else (np.zeros((0, 576)), np.zeros(0, bool))
            raw = kv[:n][ok[:n]]
            kv = raw if self.h <= 32 else round11(raw)
            if not len(kv):
                assert not o[t].any() and np.all(np.isneginf(e[t]))
                continue
            q = self.q[t].double().numpy()
            x = SM * (q @ kv.T)
            m = x.max(1, keepdims=True)
            w = np.exp(x - m)
            z = w.sum(1, keepdims=True)
            p = w / z
            ref, size = p @ kv[:, :512], p @ np.abs(kv[:, :512])
            d = SM * (np.abs(q) @ np.abs(kv).T).max() * 576 * 2.0 ** -24
            tol = ((2.0 ** -10 + 2 * d + 2.0 ** -20) * size + len(kv) * 2.0 ** -25 * np.abs(kv[:, :512]).max()
                   + 2.0 ** -8 * np.abs(ref) + 1e-30)
            bad = np.abs(o[t] - ref) / tol
            assert bad.max() <= 1, (t, bad.max())
            assert np.abs(e[t] - (m + np.log(z))[:, 0]).max() <= LSE_BF16_ATOL + d
            err2 += ((o[t] - ref) ** 2).sum()
            ref2 += (ref ** 2).sum()
            if unrounded:
                w = np.exp(SM * (q @ raw.T) - m)
                raw2 += ((o[t] - w @ raw[:, :512] / w.sum(1, keepdims=True)) ** 2).sum()
        assert err2 <= 2.0 ** -16 * ref2, math.sqrt(err2 / ref2)
        assert raw2 <= 2.0 ** -16 * ref2, math.sqrt(raw2 / ref2)


# ---- refusals (no GPU) ------------------------------------------------------------------

def _raw(lib, **kw):
    P = ctypes.c_void_p
    a = dict(q=1, n_q=2, h_s=16, cache=2, pages=8, pp=3, prefix=100, pt=4, max_pages=4, lens=5, n_seq=2, qs=6, qp=7,
             max_ctx=200, scale=0.07, out=8, lse=None, ws=9, ws_bytes=1 << 40, shift=0)
    a.update(kw)
    p = lambda v, s=0: None if v is None else P(v * 65536 + s)  # noqa: E731
    if a["ws_bytes"] < 0:  # one byte too few
        lib.dsa_prefix_attn_workspace_size.restype = ctypes.c_size_t
        a["ws_bytes"] += lib.dsa_prefix_attn_workspace_size(a["n_q"], a["h_s"], a["n_seq"], a["prefix"], a["max_ctx"])
    return lib.dsa_prefix_attn(p(a["q"], a["shift"]), a["n_q"], a["h_s"], p(a["cache"]), a["pages"], p(a["pp"]),
                               a["prefix"], p(a["pt"]), a["max_pages"], p(a["lens"]), a["n_seq"], p(a["qs"]), p(a["qp"]),
                               a["max_ctx"], ctypes.c_float(a["scale"]), p(a["out"]), p(a["lse"]), p(a["ws"]),
                               a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_q=-1), -1), (dict(n_seq=-1), -1), (dict(n_seq=0), -1), (dict(h_s=0), -2), (dict(h_s=129), -2),
    (dict(max_ctx=0, prefix=0), -2), (dict(max_ctx=1048577), -2), (dict(prefix=201), -1), (dict(prefix=-1), -1),
    (dict(pages=0), -1), (dict(max_pages=3), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(q=None), -1), (dict(cache=None), -1), (dict(pp=None), -1),
    (dict(pt=None), -1), (dict(lens=None), -1), (dict(qs=None), -1), (dict(qp=None), -1), (dict(out=None), -1),
    (dict(ws=None), -1), (dict(ws_bytes=-1), -1), (dict(ws_bytes=-1, h_s=128), -1), (dict(shift=8), -1),
    (dict(n_q=0, q=None, out=None, ws=None), 0),
])
def test_refusals(dsa, kw, code):
    assert _raw(dsa.lib(), **kw) == code


def test_workspace_size(dsa):
    f = dsa.prefix_attn_workspace_size
    # at least the expanded rows: 1152 bytes a position
    assert f(32, 128, 32, 32768, 33000) >= 1152 * (32768 + 32 * 232)
    assert f(0, 128, 32, 32768, 33000) == 0 and f(1, 128, 1, 10, 5) == 0 and f(1, 129, 1, 10, 15) == 0


def test_python_refusals(dsa):
    z = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.prefix_attn(q, torch.zeros(608 * 64, dtype=torch.uint8), z, 10, z[None], z, z, z, 20, SM)
    with pytest.raises(ValueError):
        dsa.prefix_attn(q[..., :512], torch.zeros(608 * 64, dtype=torch.uint8), z, 10, z[None], z, z, z, 20, SM)


# ---- parity ---------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("lens,prefix,h", [
    ([1], 1, 1),                      # one position, the whole prefix
    ([1], 0, 16),                     # one position, all tail
    ([65], 64, 3), ([64], 64, 128), ([63], 63, 128), ([128], 128, 128), ([129], 65, 128),
    ([257], 250, 16),                 # a partial last page of the prefix
    ([192], 192, 128), ([200], 0, 128), ([320], 320, 5),
    ([300, 301, 364, 640, 299], 300, 128),
    ([1000] * 9, 900, 16),            # 144 flattened rows: a full tile and a part
    ([700 + 37 * i for i in range(12)], 517, 33),
    ([5000, 4200], 4100, 128),        # several splits
    ([130 + i for i in range(40)], 100, 7),
    ([3000, 2000, 1], 0, 32), ([33, 32, 31, 1], 0, 17), ([2048 + 100 * i for i in range(20)], 2040, 16),
    ([6000 + i for i in range(64)], 5990, 16),   # a prefix on tensor memory, tails beside it
    ([900 + 60 * i for i in range(24)], 700, 48),
])
def test_matches_the_formula(dsa, lens, prefix, h):
    b = Batch(dsa, lens, prefix, h, seed=len(lens) + prefix)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse, unrounded=True)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [8, 64])
def test_every_code_and_scale(dsa, h):
    # random codes (all but the NaN ones, subnormals among them) and scales over 2^16
    b = Batch(dsa, [130, 100], 70, h, seed=11)
    g = torch.Generator().manual_seed(12)
    rec = b.cache.view(-1, 608)
    codes = torch.randint(0, 256, (rec.shape[0], 576), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    scale = torch.exp2(torch.rand(rec.shape[0], 5, generator=g) * 16 - 20)
    rec[:, :576] = codes.cuda()
    rec[:, 576:596] = scale.view(torch.uint8).cuda()
    b.q *= 2.0 ** -4
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,h", [(0, 16), (129, 8), (0, 32)])
def test_many_ragged_rows_of_few_heads(dsa, prefix, h):
    # blocks take equal shares of all rows' positions: rows are cut, several meet in one block, and
    # runs of rows that see nothing lie between them
    g = torch.Generator().manual_seed(h + prefix)
    lens = torch.randint(0, 900, (50,), generator=g).tolist()
    rows = [(b, L - 1 - k) for b, L in enumerate(lens) for k in range(3)]
    for i in list(range(20, 60)) + list(range(0, 150, 4)) + [149]:
        rows[i] = (rows[i][0], -1)
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=8, max_ctx=1000)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)
    again, again_lse = b.call(dsa)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    b.q_pos[:] = -1
    out, lse = b.call(dsa)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.gpu
def test_value_scales_apart_from_the_logits(dsa):
    # the logits come from the last 64 dims alone; the value tiles' scales span 2^120 and do not follow them
    b = Batch(dsa, [700, 650], 80, 16, seed=13)
    b.q[..., :512] = 0
    g = torch.Generator().manual_seed(14)
    rec = b.cache.view(-1, 608)
    scale = torch.exp2(torch.randint(-60, 60, (rec.shape[0], 4), generator=g).float())
    rec[:, 576:592] = scale.view(torch.uint8).cuda()
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [24, 40, 64, 128])
def test_rows_in_any_number_and_order(dsa, h):
    # two-token steps, a chunk of one sequence, rows inside the prefix, rows that see nothing
    lens, prefix = [700, 650, 655, 300], 640
    rows = [(1, 649), (0, 698), (0, 699), (2, 654), (0, 100), (1, 0), (2, -1), (3, 299), (3, 800), (1, 2147483647),
            (0, 639), (0, 640), (2, 63), (2, 64)] + [(0, 660 + i) for i in range(40)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=3, max_ctx=1000)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [48, 64, 128])
def test_adjacent_rows_share_a_tail_behind_a_long_prefix(dsa, h):
    # runs of one to six rows of a sequence, some cut by rows that see no tail or nothing
    lens, prefix = [1500, 1400, 1130], 1100
    rows = [(0, 1200 + 60 * i) for i in range(5)] + [(1, 1399), (0, 1499), (1, 1101), (1, 1100), (1, 1099), (1, -1), (1, 1300),
                                                     (2, 1129), (2, 500), (2, 1128), (0, 1100)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=9, max_ctx=1600)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [16, 48])
def test_bad_pages_sequences_and_lengths_are_skipped_and_flagged(dsa, h):
    lens, prefix = [900, 800, 2000, 850, -3], 700
    rows = [(0, 899), (1, 799), (2, 750), (3, 849), (4, 10), (5, 100), (-1, 100)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=4, max_ctx=1000)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 2 | 4      # BAD_SEQ, BAD_LEN and nothing else
    b.check(out, lse)
    b.lens[2], b.lens[4] = 900, 0
    b.q_seq[5:] = 0
    b.pages[0], b.pages[3] = -1, b.num_pages    # the whole first tile, and one in the middle
    b.table[0, 12], b.table[3, 13] = 1 << 30, -7
    out, lse = b.call(dsa)
    assert dsa.device_status() == 1
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [16, 64])
def test_non_finite_positions_reach_only_the_rows_that_see_them(dsa, h):
    lens, prefix = [400, 410, 390], 320
    rows = [(0, 399), (1, 409), (2, 389), (0, 349), (0, 30), (1, 200)]
    b = Batch(dsa, lens, prefix, h, rows=rows, seed=5)
    clean, clean_lse = b.call(dsa)
    rec = b.cache.view(-1, 608)

    def slot(page, p):
        return int(page[p // 64]) * 64 + p % 64

    saved = rec.clone()
    # a NaN code at position 350 of sequence 0, an infinite scale behind the end of sequence 2
    rec[slot(b.table[0], 350), 520] = 0x7F
    rec[slot(b.table[2], 395), 576:580] = torch.tensor([0, 0, 0x80, 0x7F], dtype=torch.uint8)
    out, lse = b.call(dsa)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(out[1:], clean[1:]) and torch.equal(lse[1:], clean_lse[1:])
    # a NaN inside the prefix at position 40: every row but the one that ends at 30
    rec.copy_(saved)
    rec[slot(b.pages, 40), 0] = 0xFF
    out, lse = b.call(dsa)
    assert torch.equal(out[4], clean[4]) and torch.equal(lse[4], clean_lse[4])
    for t in (0, 1, 2, 3, 5):
        assert torch.isnan(out[t]).all() and torch.isnan(lse[t]).all()
    # a NaN in one head's query stays in that head
    rec.copy_(saved)
    b.q[1, 3, 5] = float("nan")
    out, _ = b.call(dsa)
    assert torch.isnan(out[1, 3]).all()
    keep = torch.ones(6, h, dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(out[keep], clean[keep])
    assert dsa.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h", [16, 64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_far_from_the_first_tile(dsa, sign, h):
    # the logits grow (or fall) by hundreds of powers of two from tile to tile, in half of the
    # heads: the references of the first tile do not serve
    def kv(n, g):
        v = torch.randn(n, 576, generator=g)
        v[:, 0] = 0
        return v

    def q(n, g):
        v = torch.randn(n, h, 576, generator=g)
        v[:, ::2, 0] = 300.0 * sign
        return v

    b = Batch(dsa, [600, 610], 500, h, seed=6, kv=kv, q=q)
    # dim 0 of position p: p / 4 (the FP8 tile scale of 128 dims then is set by it; the bytes rule)
    vals = torch.randn(b.num_pages * 64, 576, generator=torch.Generator().manual_seed(7))
    where = torch.zeros(b.num_pages * 64)
    for s in range(2):
        p = torch.arange(b.max_ctx)
        pages = torch.where(p < 500, b.pages[torch.clamp(p // 64, max=len(b.pages) - 1)], b.table[s][p // 64])
        where[pages.long() * 64 + p % 64] = p / 4.0
    vals[:, 0] = where
    dsa.quant_kv_fp8(vals.to(torch.bfloat16).cuda(), torch.arange(b.num_pages * 64).cuda(), b.cache)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [8, 64])
def test_first_tile_unseen_and_logits_far_below_zero(dsa, h):
    # nothing of the first tile is there to take a reference from, and every logit is some -3000
    def kv(n, g):
        v = torch.randn(n, 576, generator=g)
        v[:, 0] = 40.0
        return v

    def q(n, g):
        v = torch.randn(n, h, 576, generator=g)
        v[:, :, 0] = -1000.0
        return v

    b = Batch(dsa, [300, 310], 256, h, seed=8, kv=kv, q=q)
    b.pages[0] = -1
    out, lse = b.call(dsa)
    assert dsa.device_status() == 1
    b.check(out, lse)


@pytest.mark.gpu
def test_same_bits_every_time_and_in_a_graph_on_another_stream(dsa):
    b = Batch(dsa, [2100 + 50 * i for i in range(6)], 2000, 64, seed=9)
    out, lse = b.call(dsa)
    for _ in range(3):
        o, e = b.call(dsa)
        assert torch.equal(o, out) and torch.equal(e, lse)
    q, pages, table = b.q.cuda(), b.pages.cuda(), b.table.cuda()
    lens, qs, qp = b.lens.cuda(), b.q_seq.cuda(), b.q_pos.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # two graphs with workspaces of their own, replayed at the same time
    runs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
            o, _ = dsa.prefix_attn(q, b.cache, pages, b.prefix, table, lens, qs, qp, b.max_ctx, SM)
        runs.append((graph, o, torch.cuda.Stream()))
    for _ in range(5):
        for graph, _, st in runs:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for _, o, _ in runs:
            assert torch.equal(o, out)
            o.zero_()
    assert dsa.device_status() == 0
    o, _ = dsa.prefix_attn(q, b.cache, pages, b.prefix, table, lens, qs, qp, b.max_ctx, SM, stream=side)
    side.synchronize()
    assert torch.equal(o, out)


@pytest.mark.gpu
def test_agrees_with_the_sparse_attention_over_every_position(dsa):
    # the sparse attention over all positions is the same attention
    b = Batch(dsa, [500, 460], 448, 128, seed=10)
    out, lse = b.call(dsa)
    full = b.table.clone()
    full[:, :7] = b.pages[:7]
    idx = torch.arange(500, dtype=torch.int32).repeat(2, 1)
    idx[1, 460:] = -1
    ref_lse = torch.empty(2, 128, device="cuda")
    ref, _ = dsa.sparse_attn(b.q.cuda(), b.cache, full.cuda(), b.lens.cuda(), b.q_seq.cuda(), idx.cuda(), SM,
                             out_lse=ref_lse)
    # the sparse path's own gates (its latent rows are rounded to bf16: up to sm_scale sum|q kv| 2^-8,
    # at most some 0.1 for these rows, in a logit)
    assert float((out.float() - ref.float()).abs().max()) <= 2e-2
    assert float((out.float() - ref.float()).abs().mean()) <= 2e-3
    assert float((lse - ref_lse).abs().max()) <= 0.1
