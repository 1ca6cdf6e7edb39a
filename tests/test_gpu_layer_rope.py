"""A layer that turns its own queries, keys and latent rows: the rotary calls, the rotating
writers, the decode step and the shared-prefix attention together, as a serving loop uses
them -- a shared prompt is written once, every sequence adds its own tokens, and each step
decodes over the sparse selection or densely behind the prompt."""

import math

import numpy as np
import pytest
import torch

import oracle
from dsa_sparse_attention_topk_gb300.layer import DsaDecodeLayer
from dsa_testlib import check_sfa, check_topk, ensure_built, SFA_MAX_ABS
from oracle.indexer import indexer_magnitude_row

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(192.0)
B, H_I, H_S, TOPK, PROMPT, OWN = 3, 8, 16, 64, 200, 40


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _turn64(x, pos, turns, amplitude, offset, layout):
    """float64 [.., d] rows turned to their positions, from the integer phases."""
    ph = np.array([[((int(p) * int(f) + (1 << 63)) % (1 << 64) - (1 << 63)) / 2.0 ** 64 for f in turns] for p in pos])
    c, s = amplitude * np.cos(2 * math.pi * ph), amplitude * np.sin(2 * math.pi * ph)
    c, s = (v.reshape(v.shape[:1] + (1,) * (x.ndim - 2) + v.shape[1:]) for v in (c, s))
    i = np.arange(32)
    i0, i1 = (offset + i, offset + 32 + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
    y = x.copy()
    y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i0] * s + x[..., i1] * c
    return y


class Serving:
    """B sequences behind one prompt: inputs, pages and a layer that has written everything but
    the last token of each."""

    def __init__(self, dsa, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.turns = dsa.rope_turns(64, scaling="yarn", factor=4.0, original_len=128)
        n = PROMPT + OWN
        per, whole = (n + 63) // 64, PROMPT // 64
        pages = whole + B * (per - whole)
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.empty(B, per, dtype=torch.int32)
        self.table[:, :whole] = perm[:whole]
        self.table[:, whole:] = perm[whole:].view(B, -1)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
        prompt_k, prompt_kv = r(PROMPT, 128), r(PROMPT, 576)
        self.k = torch.stack([torch.cat([prompt_k, r(OWN, 128)]) for _ in range(B)])
        self.kv = torch.stack([torch.cat([prompt_kv, r(OWN, 576)]) for _ in range(B)])
        self.layer = DsaDecodeLayer(pages, H_I, H_S, TOPK, SM, rope=self.turns)
        pos = torch.arange(n)
        slot = lambda b, p: (self.table[b, p // 64].long() * 64 + p % 64).cuda()  # noqa: E731
        # the prompt's whole pages once, the rest of it and the own tokens per sequence
        w = pos[:whole * 64]
        self.layer.write(self.k[0, w].cuda(), self.kv[0, w].cuda(), slot(0, w), w.int().cuda())
        for b in range(B):
            w = pos[whole * 64:n - 1]
            self.layer.write(self.k[b, w].cuda(), self.kv[b, w].cuda(), slot(b, w), w.int().cuda())
        self.inputs = {
            "k_new": self.k[:, -1].contiguous().cuda(), "kv_new": self.kv[:, -1].contiguous().cuda(),
            "slots_new": torch.cat([slot(b, pos[-1:]) for b in range(B)]),
            "q_idx": r(B, H_I, 128).cuda(), "w": torch.randn(B, H_I, generator=g).cuda(),
            "q_sfa": r(B, H_S, 576).cuda(), "page_table": self.table.cuda(),
            "seq_lens": torch.full((B,), n, dtype=torch.int32).cuda(),
            "q_seq": torch.arange(B, dtype=torch.int32).cuda(),
            "q_pos": torch.full((B,), n - 1, dtype=torch.int32).cuda()}
        self.n = n

    def cached(self, b):
        """Sequence b's keys and latent rows, dequantised from the caches' bytes."""
        p = np.arange(self.n)
        pg = self.table.numpy()[b][p // 64]
        kc = self.layer.k_cache.cpu().numpy().reshape(-1, 8448)[pg]
        rows = np.arange(self.n)
        codes = kc[:, :8192].reshape(-1, 64, 128)[rows, p % 64]
        scales = kc[:, 8192:].reshape(-1, 64, 4)[rows, p % 64]
        rec = self.layer.kv_cache.cpu().numpy().reshape(-1, 608)[pg.astype(np.int64) * 64 + p % 64]
        return (oracle.mxfp8_dequantize(codes, scales),
                oracle.fp8_tile_dequantize(rec[:, :576], rec[:, 576:596].copy().view(np.float32)))


@pytest.mark.parametrize("graph", [False, True])
def test_a_turning_layers_step(dsa, graph):
    s = Serving(dsa)
    if graph:
        replay = s.layer.capture_step(s.inputs, s.n)
        replay.out.zero_()
        replay()
        out, idx = replay.out, replay.idx
    else:
        out, _, idx = s.layer.step(*s.inputs.values(), s.n)
    torch.cuda.synchronize()
    assert dsa.device_status() == 0
    turns, amp = s.turns[0].cpu().tolist(), s.turns[1]
    pos = s.inputs["q_pos"].cpu().numpy()
    # the indexer and the attention get the turned queries rounded to bf16, as rope returns them
    q_idx = dsa.rope(s.inputs["q_idx"], s.inputs["q_pos"], s.turns[0], amplitude=amp, layout="half").double().cpu().numpy()
    q_sfa = dsa.rope(s.inputs["q_sfa"], s.inputs["q_pos"], s.turns[0], amplitude=amp, offset=512).double().cpu().numpy()
    for got, raw, off, layout in ((q_idx, s.inputs["q_idx"], 0, "half"), (q_sfa, s.inputs["q_sfa"], 512, "interleaved")):
        ref = _turn64(raw.double().cpu().numpy(), pos, turns, amp, off, layout)
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5)
    for b in range(B):
        k_hat, kv_hat = s.cached(b)
        # what the caches hold is the turned rows to a code's rounding: half a step of 2^-3
        # relative, or of a code's smallest step, amax 2^-9 / 448 < amax 2^-17, and the scale's share
        want = _turn64(s.kv[b].double().numpy(), np.arange(s.n), turns, amp, 512, "interleaved")
        tile = np.abs(want[:, 512:]).max(1, keepdims=True)
        assert np.all(np.abs(kv_hat[:, 512:] - want[:, 512:]) <= 2.0 ** -4 * np.abs(want[:, 512:]) + 2.0 ** -17 * tile)
        qc, qs = oracle.mxfp8_quantize(q_idx[b])
        q_hat, w = oracle.mxfp8_dequantize(qc, qs), s.inputs["w"][b].double().cpu().numpy()
        scores = oracle.indexer_scores_row(q_hat, w, k_hat)
        check_topk(idx[b].cpu().numpy(), None, scores, indexer_magnitude_row(q_hat, w, k_hat), TOPK)
        ref, _ = oracle.sparse_attention_row(q_sfa[b], kv_hat, idx[b].cpu().numpy(), SM)
        check_sfa(out[b].float().cpu().numpy(), ref)


def test_dense_attention_behind_the_prompt(dsa):
    s = Serving(dsa, seed=1)
    s.layer.step(*s.inputs.values(), s.n)
    i = s.inputs
    out, lse = s.layer.attend_prefix(i["q_sfa"], s.table[0, :(PROMPT + 63) // 64].contiguous().cuda(), PROMPT,
                                     i["page_table"], i["seq_lens"], i["q_seq"], i["q_pos"], s.n)
    assert dsa.device_status() == 0
    q = dsa.rope(i["q_sfa"], i["q_pos"], s.turns[0], amplitude=s.turns[1], offset=512).double().cpu().numpy()
    for b in range(B):
        _, kv_hat = s.cached(b)
        ref, ref_lse = oracle.sparse_attention_row(q[b], kv_hat, np.arange(s.n), SM)
        assert np.abs(out[b].double().cpu().numpy() - ref).max() <= SFA_MAX_ABS
        assert np.abs(lse[b].double().cpu().numpy() - ref_lse).max() <= 5e-3


def test_refusals(dsa):
    layer = DsaDecodeLayer(1, H_I, H_S, TOPK, SM, rope=dsa.rope_turns(64))
    z = torch.zeros(1, 576, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        layer.write(z[:, :128].contiguous(), z, torch.zeros(1, dtype=torch.int64, device="cuda"))
    q = torch.zeros(2, H_I, 128, dtype=torch.bfloat16, device="cuda")
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):  # one new token, two query rows, no positions
        layer.step(z[:, :128].contiguous(), z, torch.zeros(1, dtype=torch.int64, device="cuda"), q,
                   torch.zeros(2, H_I, device="cuda"), torch.zeros(2, H_S, 576, dtype=torch.bfloat16, device="cuda"),
                   i32[:1, None], i32[:1], i32, i32, 64)
