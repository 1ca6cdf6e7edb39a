"""A layer that norms and turns what it is given, adds up what its cached positions are worth, gives the least used
ones up and goes on: norm_rope, norm_rope_quant_kv, the decode step, sparse_attn_mass, evict_select, evict_compact and
attn_mass together, as a long conversation over a cache of fixed size uses them.

Each step is checked against the formulas in 64 bits over what the caches hold: selection and output with the bounds of
dsa_testlib, weights with that of test_gpu_attn_mass,
    |error of w| <= w (2^-19 S + 2^-22 (|l| + |lse| + 1) + 400 * 2^-24), half a unit of 2^-36 for each head."""

import math

import numpy as np
import pytest
import torch

import oracle
from dsa_sparse_attention_topk_gb300.layer import DsaDecodeLayer
from dsa_testlib import SFA_MAX_ABS, check_sfa, check_topk, ensure_built
from oracle.indexer import indexer_magnitude_row

SM = 1.0 / math.sqrt(192.0)
H_I, H_S, TOPK, BUDGET, SINKS, RECENT = 8, 16, 64, 96, 4, 16
LENS = [300, 190, 60]
B = len(LENS)


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _turn64(x, pos, turns, amplitude, offset, layout):
    """float64 [n, .., d] rows turned to their positions, from the integer phases."""
    ph = np.array([[((int(p) * int(f) + (1 << 63)) % (1 << 64) - (1 << 63)) / 2.0 ** 64 for f in turns] for p in pos])
    c, s = amplitude * np.cos(2 * math.pi * ph), amplitude * np.sin(2 * math.pi * ph)
    c, s = (v.reshape(v.shape[:1] + (1,) * (x.ndim - 2) + v.shape[1:]) for v in (c, s))
    i = np.arange(32)
    i0, i1 = (offset + i, offset + 32 + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
    y = x.copy()
    y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i0] * s + x[..., i1] * c
    return y


def _normed(x, center, w, b=0.0):
    u = x - x.mean(-1, keepdims=True) if center else x
    return u / np.sqrt((u * u).mean(-1, keepdims=True) + 1e-6) * w + b


class Talk:
    def __init__(self, dsa, seed):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dsa = g, dsa
        self.turns = dsa.rope_turns(64, scaling="yarn", factor=4.0, original_len=128)
        self.per = 6
        self.pages = 3 * B * self.per
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table, self.spare = perm[:B * self.per].view(B, -1).clone(), perm[B * self.per:2 * B * self.per].view(B, -1).clone()
        u = lambda n: 1 + 0.2 * torch.rand(n, generator=g)  # noqa: E731
        self.norm = {"k_weight": u(128), "k_bias": 0.3 * u(128), "kv_weight": u(512), "k_norm": "layer"}
        self.index_norm = {"weight": u(128)}
        cuda = lambda d: {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}  # noqa: E731
        self.layer = DsaDecodeLayer(self.pages, H_I, H_S, TOPK, SM, rope=self.turns, norm=cuda(self.norm),
                                    index_norm=cuda(self.index_norm))
        self.place = list(LENS)             # where each sequence's next token goes
        self.at = list(LENS)                # and the position that it has
        self.k = [self.r(n, 128) + 0.5 for n in LENS]
        self.kv = [self.r(n, 576) * 2 for n in LENS]
        for b in range(B):
            pos = torch.arange(LENS[b])
            self.layer.write(self.k[b].cuda(), self.kv[b].cuda(), self.slot(b, pos).cuda(), pos.int().cuda())
        self.mass = torch.zeros(B, self.per * 64, dtype=torch.int64).cuda()

    def r(self, *s):
        return torch.randn(*s, generator=self.g).to(torch.bfloat16)

    def slot(self, b, p):
        return self.table[b, p // 64].long() * 64 + p % 64

    def inputs(self):
        """The next token of every sequence, behind what its cache holds."""
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        x = {"k_new": self.r(B, 128) + 0.5, "kv_new": self.r(B, 576) * 2,
             "slots_new": torch.stack([self.slot(b, torch.tensor(self.place[b])) for b in range(B)]),
             "q_idx": self.r(B, H_I, 128) * 3, "w": torch.randn(B, H_I, generator=self.g), "q_sfa": self.r(B, H_S, 576) * 0.5,
             "page_table": self.table, "seq_lens": i32([n + 1 for n in self.place]), "q_seq": i32(list(range(B))),
             "q_pos": i32(self.place)}
        return x, i32(self.at)

    def took(self):
        self.place = [n + 1 for n in self.place]
        self.at = [n + 1 for n in self.at]

    def records(self, b, n):
        """The bytes of sequence b's first n places: key codes and scales, latent records."""
        p = np.arange(n)
        pg = self.table.numpy()[b][p // 64].astype(np.int64)
        kc = self.layer.k_cache.cpu().numpy().reshape(-1, 8448)[pg]
        return (kc[:, :8192].reshape(-1, 64, 128)[p, p % 64], kc[:, 8192:].reshape(-1, 64, 4)[p, p % 64],
                self.layer.kv_cache.cpu().numpy().reshape(-1, 608)[pg * 64 + p % 64])

    def values(self, b, n):
        codes, scales, rec = self.records(b, n)
        return (oracle.mxfp8_dequantize(codes, scales),
                oracle.fp8_tile_dequantize(rec[:, :576], rec[:, 576:596].copy().view(np.float32)))

    def weights(self, q, kv, lse):
        """(sum over heads of the weights, their bound) of one row over the values kv, in units of 1."""
        l, size, lse = SM * q @ kv.T, SM * np.abs(q) @ np.abs(kv).T, lse[:, None]
        w = np.exp(l - lse)
        tol = w * (2.0 ** -19 * size + 2.0 ** -22 * (np.abs(l) + np.abs(lse) + 1) + 400 * 2.0 ** -24) + 2.0 ** -37
        return w.sum(0), tol.sum(0)

    def check_step(self, x, rope_pos, before, out, lse, idx):
        """A step's queries, selection, output and what it added to the mass."""
        turns, amp = self.turns[0].cpu().tolist(), self.turns[1]
        pos = rope_pos.cuda()
        q_idx = self.dsa.norm_rope(x["q_idx"].cuda(), pos, self.turns[0], weight=self.index_norm["weight"].cuda(),
                                   amplitude=amp, layout="half").double().cpu().numpy()
        want = _turn64(_normed(x["q_idx"].double().numpy(), False, self.index_norm["weight"].double().numpy()),
                       rope_pos.numpy(), turns, amp, 0, "half")
        assert np.all(np.abs(q_idx - want) <= 2.0 ** -8 * np.abs(want) + 1e-4)  # (arithmetic: 2^-17 (|u| + 2) at most)
        q_sfa = self.dsa.rope(x["q_sfa"].cuda(), pos, self.turns[0], amplitude=amp, offset=512).double().cpu().numpy()
        gained = (self.mass.cpu() - before).double().numpy() * 2.0 ** -36
        for b in range(B):
            n = self.place[b] + 1
            k_hat, kv_hat = self.values(b, n)
            qc, qs = oracle.mxfp8_quantize(q_idx[b])
            q_hat, w = oracle.mxfp8_dequantize(qc, qs), x["w"][b].double().numpy()
            got = idx[b].cpu().numpy()
            check_topk(got, None, oracle.indexer_scores_row(q_hat, w, k_hat), indexer_magnitude_row(q_hat, w, k_hat), TOPK)
            ref, _ = oracle.sparse_attention_row(q_sfa[b], kv_hat, got, SM)
            check_sfa(out[b].float().cpu().numpy(), ref)
            got = got[got >= 0]
            add, tol = self.weights(q_sfa[b], kv_hat[got], lse[b].double().cpu().numpy())
            want, bound = np.zeros(self.mass.shape[1]), np.zeros(self.mass.shape[1])
            want[got], bound[got] = add, tol
            assert np.all(np.abs(gained[b] - want) <= bound)


@pytest.mark.gpu
def test_what_a_norming_layer_caches(dsa):
    """Codes of the normed and turned values: half a step of 2^-3 relative (a key's may be 448 where its value is up to
    512: an eighth), or of a tile's smallest step, below 2^-18 of its largest; arithmetic, 2^-16.4 (|u w| + |w|) with
    |w| < 2 and |u w| at most the tile's largest, turned by 1.14 at most: 2^-15 (largest + 1) together."""
    t = Talk(dsa, 0)
    turns, amp = t.turns[0].cpu().tolist(), t.turns[1]
    for b in range(B):
        n = LENS[b]
        k_hat, kv_hat = t.values(b, n)
        k = _turn64(_normed(t.k[b].double().numpy(), True, t.norm["k_weight"].double().numpy(), t.norm["k_bias"].double().numpy()),
                    np.arange(n), turns, amp, 0, "half")
        kv = t.kv[b].double().numpy()
        kv = np.concatenate([_normed(kv[:, :512], False, t.norm["kv_weight"].double().numpy()), kv[:, 512:]], 1)
        kv = _turn64(kv, np.arange(n), turns, amp, 512, "interleaved")
        assert np.all(np.abs(k_hat - k) <= 2.0 ** -3 * np.abs(k) + 2.0 ** -15 * (np.abs(k).max(1, keepdims=True) + 1))
        for i in range(0, 576, 128):
            want, got = kv[:, i:i + 128], kv_hat[:, i:i + 128]
            assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -15 * (np.abs(want).max(1, keepdims=True) + 1))


@pytest.mark.gpu
@pytest.mark.parametrize("graph,apart", [(False, False), (True, False), (False, True)])
def test_a_talk_that_outgrows_its_cache(dsa, graph, apart):
    t = Talk(dsa, 1 + graph + 2 * apart)
    max_ctx, static, replay = t.per * 64, None, None
    for turn in range(2):                   # six steps, an eviction, six more, another
        for step in range(6):
            x, rope_pos = t.inputs()
            before = t.mass.cpu()
            if graph and replay is None:
                static = {k: v.cuda() for k, v in x.items()} | {"rope_pos": rope_pos.cuda(), "mass": t.mass}
                replay = t.layer.capture_step(static, max_ctx)
                assert torch.equal(t.mass.cpu(), before)
            if graph:
                for k, v in x.items():
                    static[k].copy_(v)
                static["rope_pos"].copy_(rope_pos)
                replay()
                out, lse, idx = replay.out, replay.lse, replay.idx
            else:
                out, lse, idx = t.layer.step(*(v.cuda() for v in x.values()), max_ctx, rope_pos=rope_pos.cuda(), mass=t.mass)
            torch.cuda.synchronize()
            assert dsa.device_status() == 0
            t.check_step(x, rope_pos, before, out, lse, idx)
            t.took()
        mass, held = t.mass.cpu().numpy(), [t.records(b, t.place[b]) for b in range(B)]
        table = t.table.cuda()
        kept, lens = t.layer.evict(t.mass, table, torch.tensor(t.place, dtype=torch.int32).cuda(), BUDGET, sinks=SINKS,
                                   recent=RECENT, dst_table=t.spare.cuda() if apart else None)
        assert dsa.device_status() == 0
        if apart:
            t.table, t.spare = t.spare, t.table
        for b in range(B):
            n = t.place[b]
            stay = np.arange(n)
            if n > BUDGET:
                between = np.arange(SINKS, n - RECENT)
                order = np.lexsort((between, -mass[b, between]))[:BUDGET - SINKS - RECENT]
                stay = np.sort(np.concatenate([np.arange(SINKS), between[order], np.arange(n - RECENT, n)]))
            m = len(stay)
            assert int(lens[b]) == m
            row = kept[b].cpu().numpy()
            assert np.array_equal(row[:m], stay) and np.all(row[m:] == -1)
            for now, then in zip(t.records(b, m), held[b]):
                assert np.array_equal(now, then[stay])
            now = t.mass[b].cpu().numpy()
            assert np.array_equal(now[:m], mass[b, stay]) and not now[m:].any()
            t.place[b] = m


@pytest.mark.gpu
def test_dense_attention_adds_up_too(dsa):
    """attend_prefix over an evicted cache, its rows turned to their own positions, and decode with mass."""
    t = Talk(dsa, 9)
    x, rope_pos = t.inputs()
    t.layer.step(*(v.cuda() for v in x.values()), t.per * 64, rope_pos=rope_pos.cuda(), mass=t.mass)
    t.took()
    lens = torch.tensor(t.place, dtype=torch.int32).cuda()
    _, lens = t.layer.evict(t.mass, t.table.cuda(), lens, BUDGET, sinks=SINKS, recent=RECENT)
    t.place = lens.tolist()
    q = t.r(B, H_S, 576) * 0.5
    pos = torch.tensor(t.at, dtype=torch.int32).cuda() - 1
    mass = torch.zeros(B, BUDGET, dtype=torch.int64).cuda()
    seq = torch.arange(B, dtype=torch.int32).cuda()
    out, lse = t.layer.attend_prefix(q.cuda(), None, 0, t.table.cuda(), lens, seq, lens - 1, BUDGET, rope_pos=pos, mass=mass)
    assert dsa.device_status() == 0
    turned = dsa.rope(q.cuda(), pos, t.turns[0], amplitude=t.turns[1], offset=512).double().cpu().numpy()
    for b in range(B):
        n = t.place[b]
        _, kv_hat = t.values(b, n)
        ref, _ = oracle.sparse_attention_row(turned[b], kv_hat, np.arange(n), SM)
        assert np.abs(out[b].double().cpu().numpy() - ref).max() <= SFA_MAX_ABS
        want, tol = t.weights(turned[b], kv_hat, lse[b].double().cpu().numpy())
        got = mass[b].cpu().double().numpy() * 2.0 ** -36
        assert np.all(np.abs(got[:n] - want) <= tol) and not got[n:].any()
    # decode, given the same, adds what its step adds
    x, rope_pos = t.inputs()
    args = [v.cuda() for v in x.values()]
    one, two = torch.zeros_like(t.mass), torch.zeros_like(t.mass)
    a = [v.clone() for v in t.layer.step(*args, t.per * 64, rope_pos=rope_pos.cuda(), mass=one)]
    b = t.layer.decode(*args[3:], t.per * 64, rope_pos=rope_pos.cuda(), mass=two)
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and torch.equal(one, two) and bool(one.any())


def test_refusals():
    turns = (torch.zeros(32, dtype=torch.int64), 1.0)
    for kw in (dict(norm={}), dict(index_norm={}), dict(rope=turns, norm={"weight": None}),
               dict(rope=turns, index_norm={"k_weight": None})):
        with pytest.raises(ValueError):
            DsaDecodeLayer(1, H_I, H_S, TOPK, SM, device="cpu", **kw)
    with pytest.raises(ValueError):
        DsaDecodeLayer(1, H_I, H_S, TOPK, SM, device="cpu").attend_prefix(
            torch.zeros(1, H_S, 576), torch.zeros(1, dtype=torch.int32), 5, None, None, None, None, 5, mass=torch.zeros(1, 5))
