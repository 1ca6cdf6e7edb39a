"""attend_prefix with mass on two streams at once, and beside a recorded step of the same sizes."""

import math

import pytest
import torch

from dsa_sparse_attention_topk_gb300.layer import DsaDecodeLayer
from dsa_testlib import ensure_built

SM, B, H_I, H_S, TOPK, PER = 1.0 / math.sqrt(192.0), 6, 8, 16, 64, 8


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


@pytest.mark.gpu
def test_calls_at_once(dsa):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    lay = DsaDecodeLayer(B * PER, H_I, H_S, TOPK, SM)
    table = torch.randperm(B * PER, generator=g).view(B, PER).to(torch.int32).cuda()
    every = torch.arange(B * PER * 64).cuda()
    lay.write(r(B * PER * 64, 128), r(B * PER * 64, 576), every)
    lens, seq, ctx = i32([500, 400, 512, 300, 450, 129]), i32(list(range(B))), PER * 64
    qs = [r(B, H_S, 576) * s for s in (0.3, 0.6)]

    def attend(q, mass):
        lay.attend_prefix(q, None, 0, table, lens, seq, lens - 1, ctx, mass=mass)

    new = lambda: torch.zeros(B, ctx, dtype=torch.int64).cuda()  # noqa: E731
    want = []
    for q in qs:
        want.append(new())
        attend(q, want[-1])
    empty = torch.zeros(0, dtype=torch.int64).cuda()
    inputs = {"k_new": r(0, 128), "kv_new": r(0, 576), "slots_new": empty, "q_idx": r(B, H_I, 128), "w": torch.rand(B, H_I).cuda(),
              "q_sfa": r(B, H_S, 576), "page_table": table, "seq_lens": lens, "q_seq": seq, "q_pos": lens - 1, "mass": new()}
    replay = lay.capture_step(inputs, ctx)
    replay()
    torch.cuda.synchronize()
    step = inputs["mass"].clone()
    assert bool(step.any()) and dsa.device_status() == 0
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [new(), new()]
    inputs["mass"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, mass in zip(sides, qs, got):
            with torch.cuda.stream(s):
                attend(q, mass)
        with torch.cuda.stream(sides[2]):
            replay()
    torch.cuda.synchronize()
    assert dsa.device_status() == 0
    assert all(torch.equal(a, 20 * b) for a, b in zip(got, want)) and torch.equal(inputs["mass"], 20 * step)
