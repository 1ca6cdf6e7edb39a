"""prefix_attn where one item holds many tiles: references that rise, fall and alternate between
the tiles of the two parities, in a part of the rows, for both forms of the tensor-memory kernel.

A call's plan says which form and how many tiles an item has; each shape here pins what it
needs, so that a plan that goes another way is seen.  Tolerances are those of test_gpu_prefix."""

import copy

import numpy as np
import pytest
import torch

from dsa_testlib import ensure_built
from test_gpu_prefix import Batch, SM

POWERS = SM * 1.4426950408889634   # a logit's powers of two per unit of q . kv

# rows, heads, lengths, prefix, bound of the lengths; CTAs an MMA, tiles and splits that hold the rows
SHAPES = {
    "pair_tails": (54, 64, [700, 650, 800, 1000], 640, 1000, dict(group=2, tail_first=0, tiles_tail=16, splits_tail=1)),
    "pair_tails_split": (54, 40, [700, 650, 990, 1000], 640, 1000, dict(group=2, tail_first=0, tiles_tail=16, splits_tail=2)),
    "pair_prefix": (100, 64, [1280, 1281], 1280, 1281, dict(group=2, tiles_prefix=20, splits_prefix=1)),
    "single_tails": (48, 40, [700 - 9 * i for i in range(48)], 0, 700, dict(group=1, tiles_tail=11, splits_tail=1)),
    "single_tails_split": (24, 48, [900 - 7 * i for i in range(24)], 600, 900,
                           dict(group=1, tail_first=0, tiles_tail=15, splits_tail=2)),
}

# powers of two of tile j's logits above the rest (some rows see them, some their negative)
MOVES = {
    "rise": lambda j, n: 17.0 * j,
    "fall": lambda j, n: -17.0 * j,
    "odd_high": lambda j, n: 40.0 * (j % 2),
    "even_rise": lambda j, n: -30.0 if j % 2 else 11.0 * j,
    "odd_rise": lambda j, n: 11.0 * j if j % 2 else -30.0,
    "one_late": lambda j, n: 50.0 if j == n - 2 else 0.0,
    "one_early": lambda j, n: 35.0 if j == 1 else 0.0,
    "mixed": lambda j, n: float((j * 37) % 11 - 5) * 12.0,
}


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


class Tiles(Batch):
    def __init__(self, dsa, shape, move=None, seed=0):
        n, h, lens, prefix, max_ctx, plan = SHAPES[shape]
        rows = [(i * len(lens) // n, 0) for i in range(n)]
        rows = [(b, lens[b] - 1 - 7 * (i % 8)) for i, (b, _) in enumerate(rows)]
        got = dsa.test_prefix_plan(n, h, len(lens), prefix, max_ctx)
        assert {k: got[k] for k in plan} == plan and got["few_parts"] == 0
        self._rows = {}
        super().__init__(dsa, lens, prefix, h, rows=rows, seed=seed, max_ctx=max_ctx)
        self.n_tiles = (max_ctx + 63) // 64
        if move is not None:
            # the last 64 dims: the first holds tile j's height / 16 powers of two, the others nothing
            vals = torch.randn(self.num_pages * 64, 576, generator=torch.Generator().manual_seed(seed + 1))
            vals[:, 512:] = 0
            height = torch.tensor([MOVES[move](j, self.n_tiles) for j in range(self.n_tiles)])
            for b in range(len(lens)):
                p = torch.arange(max_ctx)
                pages = torch.where(p < prefix, torch.cat([self.pages, self.pages.new_zeros(1)])[(p // 64).clamp(
                    max=len(self.pages))], self.table[b][p // 64])
                vals[pages.long() * 64 + p % 64, 512] = height[p // 64] / 16
            dsa.quant_kv_fp8(vals.to(torch.bfloat16).cuda(), torch.arange(self.num_pages * 64).cuda(), self.cache)
            sign = torch.tensor([1.0, 0.0, -1.0, 1.0, 1.0])[torch.arange(n * h) % 5].view(n, h)
            sign[: n // 4] = 1.0         # whole warps that agree
            self.q[..., 512:] = 0
            self.q[..., 512] = (sign * 16 / POWERS).to(torch.bfloat16)

    def rows64(self, b):
        if b not in self._rows:
            self._rows[b] = super().rows64(b)
        return self._rows[b]

    def check(self, out, lse, step=5):
        """Every step-th row and the last ones."""
        some = copy.copy(self)
        some._rows = {}
        n = self.q.shape[0]
        i = torch.tensor(sorted({*range(0, n, step), n - 2, n - 1}))
        some.q, some.q_seq, some.q_pos = self.q[i], self.q_seq[i], self.q_pos[i]
        Batch.check(some, out[i], lse[i])


@pytest.mark.gpu
@pytest.mark.parametrize("move", sorted(MOVES))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_references_move_between_an_items_tiles(dsa, shape, move):
    b = Tiles(dsa, shape, move, seed=len(shape) + len(move))
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)
    again, again_lse = b.call(dsa)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_first_reference_behind_tiles_that_are_not_there(dsa, shape):
    b = Tiles(dsa, shape, "fall", seed=3)
    if b.prefix:
        b.pages[:3], b.pages[5] = -1, b.num_pages
    else:
        b.table[:, :3], b.table[::3, 4] = -1, 1 << 30
    out, lse = b.call(dsa)
    assert dsa.device_status() == 1
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_every_code_and_scale_in_long_items(dsa, shape):
    b = Tiles(dsa, shape, seed=4)
    g = torch.Generator().manual_seed(5)
    rec = b.cache.view(-1, 608)
    codes = torch.randint(0, 256, (rec.shape[0], 576), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38
    rec[:, :576] = codes.cuda()
    rec[:, 576:596] = torch.exp2(torch.rand(rec.shape[0], 5, generator=g) * 16 - 20).view(torch.uint8).cuda()
    b.q *= 2.0 ** -4
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_non_finite_positions_in_long_items(dsa, shape):
    b = Tiles(dsa, shape, "mixed", seed=6)
    clean, clean_lse = b.call(dsa)
    rec = b.cache.view(-1, 608)
    # a NaN code at position 200 of the last sequence; with a prefix the page may be everyone's
    page = int(b.pages[200 // 64]) if b.prefix > 200 else int(b.table[-1, 200 // 64])
    rec[page * 64 + 200 % 64, 200] = 0x7F
    # and an infinite scale behind every row's end
    rec[int(b.table[0, -1]) * 64 + 63, 576:580] = torch.tensor([0, 0, 0x80, 0x7F], dtype=torch.uint8)
    out, lse = b.call(dsa)
    assert dsa.device_status() == 0
    hit = torch.ones_like(b.q_seq, dtype=torch.bool) if b.prefix > 200 else b.q_seq == len(b.lens) - 1
    hit &= b.q_pos >= 200
    assert hit.any()
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", ["pair_tails_split", "pair_prefix"])
def test_long_items_in_two_graphs_at_once(dsa, shape):
    b = Tiles(dsa, shape, "mixed", seed=7)
    want, _ = b.call(dsa)
    q, pages, table = b.q.cuda(), b.pages.cuda(), b.table.cuda()
    lens, qs, qp = b.lens.cuda(), b.q_seq.cuda(), b.q_pos.cuda()
    torch.cuda.synchronize()
    side, runs = torch.cuda.Stream(), []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
            o, _ = dsa.prefix_attn(q, b.cache, pages, b.prefix, table, lens, qs, qp, b.max_ctx, SM)
        runs.append((graph, o, torch.cuda.Stream()))
    for _ in range(4):
        for graph, _, st in runs:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for _, o, _ in runs:
            assert torch.equal(o, want)
            o.zero_()
    assert dsa.device_status() == 0


@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_the_plans_of_these_shapes(dsa, shape):
    n, h, lens, prefix, max_ctx, plan = SHAPES[shape]
    got = dsa.test_prefix_plan(n, h, len(lens), prefix, max_ctx)
    assert {k: got[k] for k in plan} == plan
    with pytest.raises(dsa.DsaError):
        dsa.test_prefix_plan(n, 129, len(lens), prefix, max_ctx)
