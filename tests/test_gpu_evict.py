"""Eviction by accumulated weight: which positions stay (evict_select), and their records moved (evict_compact).
Whole numbers and copies throughout: everything is compared exactly with a plain implementation."""

import ctypes

import pytest
import torch

from dsa_testlib import ensure_built

BIG = (1 << 63) - 1


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _select(mass, lens, budget, sinks, recent):
    """The definition: one sequence at a time, Python's sort."""
    kept, new, weights = [], [], []
    for m, n in zip(mass.tolist(), lens.tolist()):
        n = n if 0 <= n <= mass.shape[1] else 0
        if n <= budget:
            stay = list(range(n))
        else:
            between = sorted(range(sinks, n - recent), key=lambda p: (-m[p], p))[:budget - sinks - recent]
            stay = sorted(list(range(sinks)) + between + list(range(n - recent, n)))
        kept.append(stay + [-1] * (budget - len(stay)))
        new.append(len(stay))
        weights.append([m[p] for p in stay] + [0] * (budget - len(stay)))
    return torch.tensor(kept, dtype=torch.int32), torch.tensor(new, dtype=torch.int32), torch.tensor(weights)


def _mass(kind, n_seq, ctx, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "steps":            # heavy-tailed, and nothing where no step selected
        m = (torch.exp(1.7 * torch.randn(n_seq, ctx, generator=g) - 6).double() * 2.0 ** 36).long()
        return m * (torch.rand(n_seq, ctx, generator=g) < 0.6)
    if kind == "zeros":
        return torch.zeros(n_seq, ctx, dtype=torch.int64)
    if kind == "few values":       # many ties
        return torch.randint(0, 4, (n_seq, ctx), generator=g) * 1000
    if kind == "any bits":         # every bit of 64, both signs
        return torch.randint(-(1 << 62), 1 << 62, (n_seq, ctx), generator=g) * 2 + 1
    if kind == "ends":             # the type's lowest and highest values
        return torch.tensor([-BIG - 1, BIG, 0, -1])[torch.randint(0, 4, (n_seq, ctx), generator=g)]
    return torch.arange(ctx).expand(n_seq, ctx) + (1 << 40)  # "rising": only the low bits differ


KINDS = ["steps", "zeros", "few values", "any bits", "ends", "rising"]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_seq,ctx,budget,sinks,recent", [
    (1, 1, 1, 0, 0), (3, 2, 1, 0, 0), (5, 700, 100, 4, 32), (4, 700, 700, 0, 0), (2, 700, 1000, 1, 1), (7, 4097, 64, 0, 64),
    (7, 4097, 64, 64, 0), (3, 4097, 65, 32, 32), (2, 20000, 2048, 4, 257), (1, 50000, 49999, 1, 0), (160, 300, 17, 2, 3),
    (40, 5000, 1000, 0, 0)])
def test_select(dsa, kind, n_seq, ctx, budget, sinks, recent):
    mass = _mass(kind, n_seq, ctx, ctx + budget)
    g = torch.Generator().manual_seed(n_seq)
    lens = torch.randint(0, ctx + 1, (n_seq,), generator=g, dtype=torch.int32)
    lens[0] = ctx
    if n_seq > 2:
        lens[1], lens[2] = 0, min(ctx, budget + 1)
    got = dsa.evict_select(mass.cuda(), lens.cuda(), budget, sinks, recent)
    assert dsa.device_status() == 0
    for have, want in zip(got, _select(mass, lens, budget, sinks, recent)):
        assert torch.equal(have.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_seq,ctx", [(2, 300000), (9, 300000), (1, 500000), (9, 20000), (7, 20000)])
def test_select_of_long_contexts(dsa, kind, n_seq, ctx):
    """Few sequences have sixteen CTAs each, more of them eight; a CTA holds 24 K keys in shared memory, so 300,000
    positions are beyond that with eight, 500,000 with sixteen."""
    mass = _mass(kind, n_seq, ctx, 9)
    lens = torch.tensor([ctx, ctx - ctx // 6 + 1] * 5, dtype=torch.int32)[:n_seq]
    got = dsa.evict_select(mass.cuda(), lens.cuda(), ctx // 3, 4, 64)
    for have, want in zip(got, _select(mass, lens, ctx // 3, 4, 64)):
        assert torch.equal(have.cpu(), want)


@pytest.mark.gpu
def test_select_rows_apart_bad_lengths_and_given_results(dsa):
    wide = _mass("steps", 4, 900, 1).cuda()
    mass = wide[:, 100:600]
    lens = torch.tensor([500, -1, 501, 300], dtype=torch.int32)
    kept = torch.full((4, 50), 7, dtype=torch.int32).cuda()
    new = torch.full((4,), 7, dtype=torch.int32).cuda()
    weights = torch.full((4, 50), 7, dtype=torch.int64).cuda()
    got = dsa.evict_select(mass, lens.cuda(), 50, 3, 5, kept=kept, new_lens=new, kept_mass=weights)
    assert got[0] is kept and got[1] is new and got[2] is weights
    assert dsa.status_names(dsa.device_status()) == ["BAD_LEN"]
    for have, want in zip(got, _select(mass.cpu(), lens, 50, 3, 5)):
        assert torch.equal(have.cpu(), want)
    none = dsa.evict_select(mass[:0], lens[:0].cuda(), 50)
    assert none[0].shape == (0, 50) and none[1].shape == (0,)


# ---- moving ------------------------------------------------------------------------------

def _pool(pages, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 256, (pages * 8448,), generator=g, dtype=torch.uint8),
            torch.randint(0, 256, (pages * 64 * 608,), generator=g, dtype=torch.uint8))


def _compact(kept, table, k, kv, dst_table, pages):
    """The definition: every record read before any is written."""
    k, kv = k.clone().view(-1, 8448), kv.clone().view(-1, 608)
    moves = []
    for b in range(kept.shape[0]):
        for i, p in enumerate(kept[b].tolist()):
            if not 0 <= p < table.shape[1] * 64:
                continue
            s, d = int(table[b, p // 64]), int(dst_table[b, i // 64])
            if 0 <= s < pages and 0 <= d < pages:
                moves.append((s, p % 64, d, i % 64))
    new_k, new_kv = k.clone(), kv.clone()
    for s, r, d, q in moves:
        new_kv[d * 64 + q] = kv[s * 64 + r]
        new_k[d, q * 128:q * 128 + 128] = k[s, r * 128:r * 128 + 128]
        new_k[d, 8192 + 4 * q:8196 + 4 * q] = k[s, 8192 + 4 * r:8196 + 4 * r]
    return new_k.view(-1), new_kv.view(-1)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n_seq,per,budget,kind", [
    (1, 1, 1, "steps"), (3, 5, 63, "steps"), (4, 6, 129, "few values"), (2, 4, 256, "steps"), (5, 3, 100, "any order")])
def test_compact(dsa, in_place, n_seq, per, budget, kind):
    g = torch.Generator().manual_seed(budget)
    per_new = (budget + 63) // 64
    pages = n_seq * (per + per_new) + 2
    k, kv = _pool(pages, budget)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table, fresh = perm[:n_seq * per].view(n_seq, per), perm[n_seq * per:n_seq * (per + per_new)].view(n_seq, per_new)
    dst = table if in_place else fresh
    if kind == "any order":              # the same position twice, and gaps
        kept = torch.randint(-1, per * 64, (n_seq, budget), generator=g, dtype=torch.int32)
    else:
        lens = torch.randint(0, per * 64 + 1, (n_seq,), generator=g, dtype=torch.int32)
        lens[0] = per * 64
        kept = _select(_mass(kind, n_seq, per * 64, 3), lens, budget, 0, 0)[0]
    want = _compact(kept, table, k, kv, dst, pages)
    kg, kvg = k.cuda(), kv.cuda()
    dsa.evict_compact(kept.cuda(), table.cuda(), kg, kvg, dst_table=None if in_place else dst.cuda())
    assert dsa.device_status() == 0
    assert torch.equal(kg.cpu(), want[0]) and torch.equal(kvg.cpu(), want[1])
    for which in (0, 1):                 # one cache alone; the other stays
        kg, kvg = k.cuda(), kv.cuda()
        args = (kg, None) if which == 0 else (None, kvg)
        dsa.evict_compact(kept.cuda(), table.cuda(), *args, dst_table=None if in_place else dst.cuda())
        assert torch.equal(kg.cpu(), want[0] if which == 0 else k) and torch.equal(kvg.cpu(), want[1] if which else kv)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_bad_pages_and_positions_are_left_out(dsa, in_place):
    k, kv = _pool(12, 1)
    table = torch.tensor([[3, 12, 5], [1, 2, 0]], dtype=torch.int32)
    fresh = torch.tensor([[6, -1], [8, 9]], dtype=torch.int32)
    kept = torch.tensor([[0, 5, 70, 140], [1, 192, -2, 100]], dtype=torch.int32).repeat(1, 17)[:, :66].contiguous()
    dst = table if in_place else fresh
    want = _compact(kept, table, k, kv, dst, 12)
    kg, kvg = k.cuda(), kv.cuda()
    dsa.evict_compact(kept.cuda(), table.cuda(), kg, kvg, dst_table=None if in_place else dst.cuda())
    assert set(dsa.status_names(dsa.device_status())) == {"BAD_PAGE", "BAD_INDEX"}
    assert torch.equal(kg.cpu(), want[0]) and torch.equal(kvg.cpu(), want[1])


@pytest.mark.gpu
def test_graph_and_stream(dsa):
    mass, lens = _mass("steps", 6, 640, 2).cuda(), torch.full((6,), 640, dtype=torch.int32).cuda()
    k, kv = (t.cuda() for t in _pool(60, 3))
    table = torch.randperm(60).to(torch.int32).view(6, 10).cuda()
    side = torch.cuda.Stream()
    kk, vv = k.clone(), kv.clone()
    side.wait_stream(torch.cuda.current_stream())
    kept, new, weights = dsa.evict_select(mass, lens, 100, 2, 8, stream=side)
    dsa.evict_compact(kept, table, kk, vv, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = _compact(kept.cpu(), table.cpu(), k.cpu(), kv.cpu(), table.cpu(), 60)
    assert torch.equal(kk.cpu(), want[0]) and torch.equal(vv.cpu(), want[1])
    graph = torch.cuda.CUDAGraph()
    static = mass.clone()
    with torch.cuda.graph(graph):
        gk, gn, gw = dsa.evict_select(static, lens, 100, 2, 8)
        dsa.evict_compact(gk, table, kk, vv)
    for seed in (5, 6):
        static.copy_(_mass("steps", 6, 640, seed))
        kk.copy_(k)
        vv.copy_(kv)
        graph.replay()
        torch.cuda.synchronize()
        ref = _select(static.cpu(), lens.cpu(), 100, 2, 8)
        assert torch.equal(gk.cpu(), ref[0]) and torch.equal(gw.cpu(), ref[2])
        want = _compact(ref[0], table.cpu(), k.cpu(), kv.cpu(), table.cpu(), 60)
        assert torch.equal(kk.cpu(), want[0]) and torch.equal(vv.cpu(), want[1])


# ---- refusals (no GPU) -------------------------------------------------------------------

def _p(v):
    return None if v is None else ctypes.c_void_p(int(v * 65536))


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(ctx=0), -2), (dict(ctx=1 << 21), -2), (dict(budget=0), -2), (dict(budget=1 << 21), -2),
    (dict(sinks=-1), -1), (dict(recent=-1), -1), (dict(sinks=5, recent=6), -1), (dict(stride=99), -1), (dict(stride=1 << 40), -1),
    (dict(mass=None), -1), (dict(lens=None), -1), (dict(kept=None), -1), (dict(new=None), -1), (dict(mass=1 + 2.0 ** -14), -1),
    (dict(weights=5 + 2.0 ** -14), -1), (dict(kept=3 + 2.0 ** -15), -1), (dict(n=1 << 28), -2), (dict(new=2), -1), (dict(n=0, mass=None), 0)])
def test_select_refusals(dsa, kw, code):
    a = dict(mass=1, stride=100, lens=2, n=3, ctx=100, budget=10, sinks=2, recent=3, kept=3, new=4, weights=5)
    a.update(kw)
    assert dsa.lib().dsa_evict_select(_p(a["mass"]), a["stride"], _p(a["lens"]), a["n"], a["ctx"], a["budget"], a["sinks"],
                                      a["recent"], _p(a["kept"]), _p(a["new"]), _p(a["weights"]), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(budget=0), -2), (dict(max_pages=0), -1), (dict(pages=0), -1), (dict(kept=None), -1),
    (dict(table=None), -1), (dict(k=None, kv=None), -1), (dict(dst=2, dst_pages=9), -1), (dict(dst=3, dst_pages=1), -1),
    (dict(max_pages=1), -1), (dict(kept=1 + 2.0 ** -15), -1), (dict(kv=5 + 2.0 ** -13), -1), (dict(ws=None), -1),
    (dict(ws_bytes=1000), -1), (dict(ws=6 + 2.0 ** -9), -1), (dict(n=1 << 26, budget=1024, max_pages=64), -2), (dict(n=0, kept=None), 0)])
def test_compact_refusals(dsa, kw, code):
    a = dict(kept=1, n=3, budget=100, table=2, max_pages=8, dst=None, dst_pages=0, k=4, kv=5, pages=20, ws=6, ws_bytes=1 << 30)
    a.update(kw)
    assert dsa.lib().dsa_evict_compact(_p(a["kept"]), a["n"], a["budget"], _p(a["table"]), a["max_pages"], _p(a["dst"]),
                                       a["dst_pages"], _p(a["k"]), _p(a["kv"]), a["pages"], _p(a["ws"]), a["ws_bytes"],
                                       None) == code


def test_the_binding_refuses(dsa):
    mass, lens = torch.zeros(2, 10, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    for bad in (mass.int(), mass[0], mass.t()):
        with pytest.raises(ValueError, match="mass must"):
            dsa.evict_select(bad, lens, 4)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.evict_select(mass, lens, 4)
    with pytest.raises(ValueError, match="kept must"):
        dsa.evict_compact(lens, lens[None])
    assert dsa.evict_compact_workspace_size(0, 5) == 0 and dsa.evict_compact_workspace_size(2, 100) == 2 * 100 * 752
