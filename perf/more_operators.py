"""Cases of the per-head norm with the rotation, its gradient, the norming cache writer, the accumulated attention weights
and the eviction that goes by them, each with its plain form.

``run`` computes a case in elementary torch operations (32 bits; angles in 64) where ``own`` is false, and through the
package's entry points where it is true.  ``exact`` is the operators' definition in 64 bits, written apart from both.

The sizes are those of the package's own workloads (indexer heads of 128, latent rows of 576 = 512 + 64 rotary, 64-token
pages, Top-2048, contexts of 32K and 128K, chunks of 4096 rows) and odd ones around them."""

import math

import torch

own = False

PAGE, D_K, D_KV, D_V, ROT = 64, 128, 576, 512, 64
K_PAGE_BYTES, KV_TOKEN_BYTES = 8448, 608
SM_SCALE = 1.0 / math.sqrt(192.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
EPS = 1e-6
MASS_UNIT = 2.0 ** -36  # accumulated weights are whole numbers of this


# ---- cases -----------------------------------------------------------------------------

def _norm(op, name, n, h, d, span, rot, offset, kind, bias, layout, dtype, weights, pad):
    return {"name": name, "op": op, "n": n, "h": h, "d": d, "span": span, "rot": rot, "offset": offset, "kind": kind,
            "bias": bias, "layout": layout, "dtype": dtype, "weights": weights, "pad": pad}


def _append(name, n, pages, pos_max, kind, bias, k_offset, k_layout, kv_layout):
    return {"name": name, "op": "append", "n": n, "pages": pages, "pos_max": pos_max, "kind": kind, "bias": bias,
            "k_offset": k_offset, "k_layout": k_layout, "kv_layout": kv_layout}


def _mass(name, seqs, per_seq, h, lo, hi):
    return {"name": name, "op": "mass", "seqs": seqs, "per_seq": per_seq, "h": h, "lo": lo, "hi": hi}


def _picked(name, seqs, per_seq, h, ctx, topk, fewest):
    return {"name": name, "op": "picked", "seqs": seqs, "per_seq": per_seq, "h": h, "ctx": ctx, "topk": topk,
            "fewest": fewest}


def _evict(name, seqs, lo, hi, budget, sinks, recent, in_place):
    return {"name": name, "op": "evict", "seqs": seqs, "lo": lo, "hi": hi, "budget": budget, "sinks": sinks,
            "recent": recent, "in_place": in_place}


def listed():
    return [
        # one row's indexer query: latency alone
        _norm("norm", "norm_one_row", 1, 64, 128, 128, 64, 0, "rms", False, "half", "bf16", "fp32", 0),
        # the indexer queries of a chunk of 4096 prompt rows
        _norm("norm", "norm_chunk_4k", 4096, 64, 128, 128, 64, 0, "rms", False, "half", "bf16", "bf16", 0),
        # the gradient of that chunk's norm and rotation, and of its weight
        _norm("grad", "norm_grad_chunk_4k", 4096, 64, 128, 128, 64, 0, "rms", False, "half", "bf16", "bf16", 0),
        # the gradient in fp32 with a mean and a bias: odd counts, rows inside a wider projection, the rotary part not normed
        _norm("grad", "norm_grad_fp32", 2047, 63, 192, 128, 64, 128, "layer", True, "interleaved", "fp32", "fp32", 64),
        # the new tokens of a decode batch of 32
        _append("append_decode_b32", 32, 64, 32768, "layer", True, 0, "half", "interleaved"),
        # a whole 64K prompt
        _append("append_prompt_64k", 65536, 1024, 65536, "layer", True, 64, "interleaved", "half"),
        # a decode batch's dense step, every cached position weighed: contexts of 16K to 32K
        _mass("mass_decode_b32_32k", 32, 1, 128, 16384, 32768),
        # the last 64 rows of a 32K prompt as the observation window of an eviction
        _mass("mass_window_64_32k", 1, 64, 128, 32768, 32768),
        # a sparse decode step of 32 rows with the heads of one of eight shards
        _picked("picked_decode_b32", 32, 1, 16, 32768, 2048, 2048),
        # 512 causal rows behind a 16K prompt, each over its selection; the first ones with padding behind it
        _picked("picked_chunk_512", 1, 512, 128, 16384, 2048, 1800),
        # a decode batch cut down to 2048 positions each, into pages of their own
        _evict("evict_decode_b32_32k", 32, 16384, 32768, 2048, 4, 64, False),
        # one document of 128K positions halved in place
        _evict("evict_long_128k", 1, 131072, 131072, 65536, 4, 1024, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "grad", "append", "mass", "picked", "evict"])
    if op in ("norm", "grad"):
        d = rng.choice([64, 100, 128, 128, 192, 256, 576])
        span = rng.choice([d, d, d - 32, 64])
        rot = rng.choice([r for r in (32, 64, 64, 96, 50) if r <= d])
        h = rng.choice([1, 3, 8, 16, 63, 64, 128])
        n = _log(rng, 1, max(1, min(65536, 33_000_000 // (h * d))))
        kind = rng.choice(["rms", "rms", "layer"])
        return _norm(op, "", n, h, d, span, rot, rng.choice([0, d - rot]), kind, kind == "layer" and rng.random() < 0.7,
                     rng.choice(["half", "interleaved"]), rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     rng.choice(["fp32", "same"]), rng.choice([0, 0, 64, 4]))
    if op == "append":
        n = _log(rng, 1, 65536)
        kind = rng.choice(["rms", "layer"])
        return _append("", n, (n + PAGE - 1) // PAGE + rng.randrange(1, 40), _log(rng, 65536, 1 << 20), kind,
                       kind == "layer", 4 * rng.randrange(0, 17), rng.choice(["half", "interleaved"]),
                       rng.choice(["half", "interleaved"]))
    while op == "mass":
        seqs, per_seq, h = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 32, 64]), rng.choice([1, 5, 16, 32, 64, 128])
        hi = _log(rng, 1, 131072)
        if seqs * per_seq * h * hi <= 134_000_000 and seqs * hi <= 1_048_576 and hi >= per_seq:
            return _mass("", seqs, per_seq, h, rng.randrange(max(per_seq, hi // 3), hi + 1), hi)
    while op == "picked":
        seqs, per_seq, h = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 64]), rng.choice([1, 5, 16, 32, 64, 128])
        ctx, topk = _log(rng, 1, 65536), rng.choice([1, 33, 100, 256, 1024, 2000, 2048])
        if seqs * per_seq * h * topk <= 134_000_000 and seqs * ctx <= 1_048_576 and seqs * per_seq * ctx <= 16_777_216:
            return _picked("", seqs, per_seq, h, ctx, topk, rng.randrange(0, min(ctx, topk) + 1))
    while True:
        seqs, hi = _log(rng, 1, 64), _log(rng, 1, 200000)
        budget, sinks = _log(rng, 1, hi), rng.choice([0, 0, 1, 4])
        recent = rng.choice([0, 0, 1, 32, 257])
        if seqs * hi <= 262144 and sinks + recent <= budget:
            return _evict("", seqs, rng.randrange(hi // 3, hi + 1), hi, budget, sinks, recent, rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------------------

def _angles(rot):
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    # the package takes turns a position in 64-bit fixed point
    turns = [round(v / (2 * math.pi) * 2.0 ** 64) for v in f]
    return {"freq": torch.tensor(f, dtype=torch.float64, device="cuda"),
            "turns": torch.tensor(turns, dtype=torch.int64, device="cuda")}


def _latent_cache(g, tokens):
    """FP8 records of normal values: codes, and the scale amax / 448 of each tile of 128."""
    cache = torch.zeros(tokens, KV_TOKEN_BYTES, dtype=torch.uint8, device="cuda")
    for a in range(0, tokens, 131072):
        rows = torch.randn(min(131072, tokens - a), 640, generator=g, device="cuda")
        rows[:, D_KV:] = 0
        tiles = rows.view(-1, 5, 128)
        scales = tiles.abs().amax(-1) / E4M3_MAX
        codes = (tiles / scales[..., None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache[a:a + len(rows), :D_KV] = codes.view(-1, 640)[:, :D_KV].view(torch.uint8)
        cache[a:a + len(rows), D_KV:D_KV + 20] = scales.contiguous().view(torch.uint8)
    return cache.view(-1)


def _pages(g, seqs, per):
    """A page table over a pool of just these pages, in any order."""
    return torch.randperm(seqs * per, generator=g, device="cuda").to(torch.int32).view(seqs, per)


def _lens(g, case, lo, hi):
    u = torch.rand(case["seqs"], generator=g, device="cuda")
    lens = (lo + (u * (hi - lo + 1)).long()).clamp(max=hi).to(torch.int32)
    lens[0] = hi
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    if op in ("norm", "grad"):
        n, h, d, span, dtype = case["n"], case["h"], case["d"], case["span"], DTYPES[case["dtype"]]
        w_dtype = dtype if case["weights"] == "same" else DTYPES[case["weights"]]
        x = (randn(n, h, d + case["pad"]) * 2 + 0.3).to(dtype)[..., :d]
        # a chunk's consecutive positions, or rows of a batch at any position
        pos = torch.randint(0, 65536, (n,), generator=g, device="cuda", dtype=torch.int32)
        if n > 512:
            pos = torch.arange(n, device="cuda", dtype=torch.int32) + pos[0]
        return {"case": case, "x": x, "pos": pos, "weight": (1 + 0.2 * randn(span)).to(w_dtype),
                "bias": (0.1 * randn(span)).to(w_dtype) if case["bias"] else None,
                "dy": randn(n, h, d).to(dtype) if op == "grad" else None, **_angles(case["rot"])}
    if op == "append":
        n, pages = case["n"], case["pages"]
        k = randn(n, D_K)
        k[:, torch.randperm(D_K, generator=g, device="cuda")[:4]] *= 8  # outlier channels
        kv = randn(n, D_KV) * 3
        pos = torch.randint(0, case["pos_max"], (n,), generator=g, device="cuda", dtype=torch.int32)
        perm = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        if n > 512:  # a prompt fills its pages in order
            slots = perm[i // PAGE] * PAGE + i % PAGE
            pos = (i % case["pos_max"]).to(torch.int32)
        else:        # one token of each sequence, anywhere in the pool
            slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n]
        slots[5::37] = -1  # padded rows of the batch
        return {"case": case, "k": k.to(torch.bfloat16), "kv": kv.to(torch.bfloat16), "pos": pos, "slots": slots,
                "k_weight": 1 + 0.2 * randn(D_K), "k_bias": 0.1 * randn(D_K) if case["bias"] else None,
                "kv_weight": 1 + 0.2 * randn(D_V),
                "k_cache": torch.zeros(pages * K_PAGE_BYTES, dtype=torch.uint8, device="cuda"),
                "kv_cache": torch.zeros(pages * PAGE * KV_TOKEN_BYTES, dtype=torch.uint8, device="cuda"),
                **_angles(ROT)}
    if op == "evict":
        seqs, hi, budget = case["seqs"], case["hi"], case["budget"]
        table = _pages(g, seqs, (hi + PAGE - 1) // PAGE)
        old = table.numel()
        dst, pages = None, old
        if not case["in_place"]:  # fresh pages of the same pool, behind the old ones
            dst = _pages(g, seqs, (budget + PAGE - 1) // PAGE) + old
            pages = old + dst.numel()
        # accumulated weights: heavy-tailed, and nothing at the positions that no step selected
        weight = torch.exp(1.7 * randn(seqs, hi) - 6) * (torch.rand(seqs, hi, generator=g, device="cuda") < 0.6)
        k = randn(pages, K_PAGE_BYTES).mul_(100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        k[:, PAGE * D_K:] = torch.randint(110, 130, (pages, PAGE * 4), generator=g, device="cuda", dtype=torch.uint8)
        return {"case": case, "mass": (weight.double() / MASS_UNIT).long(), "table": table, "dst": dst, "old": old,
                "seq_lens": _lens(g, case, case["lo"], hi), "k_cache": k.view(-1),
                "kv_cache": _latent_cache(g, pages * PAGE)}
    seqs, per_seq, h = case["seqs"], case["per_seq"], case["h"]
    rows = seqs * per_seq
    hi = case["hi"] if op == "mass" else case["ctx"]
    table = _pages(g, seqs, (hi + PAGE - 1) // PAGE)
    s = {"case": case, "kv_cache": _latent_cache(g, table.numel() * PAGE), "table": table, "max_ctx": hi,
         "q": randn(rows, h, D_KV).to(torch.bfloat16),
         "q_seq": torch.arange(seqs, device="cuda", dtype=torch.int32).repeat_interleave(per_seq)}
    if op == "mass":
        s["seq_lens"] = _lens(g, case, case["lo"], hi)
        s["q_pos"] = (s["seq_lens"].repeat_interleave(per_seq) - per_seq
                      + torch.arange(per_seq, device="cuda", dtype=torch.int32).repeat(seqs)).to(torch.int32)
        # what the attention over the same positions returned
        s["lse"] = torch.logsumexp(_logits(s), -1).view(rows, h)
        return s
    topk = case["topk"]
    s["seq_lens"] = torch.full((seqs,), hi, dtype=torch.int32, device="cuda")
    s["idx"] = torch.full((rows, topk), -1, dtype=torch.int32, device="cuda")
    k = min(topk, hi)
    for a in range(0, rows, 64):
        r = torch.rand(min(64, rows - a), hi, generator=g, device="cuda")
        s["idx"][a:a + 64, :k] = r.topk(k, -1).indices.to(torch.int32)
    # rows that found fewer positions than Top-K
    found = case["fewest"] + torch.randint(0, k - case["fewest"] + 1, (rows,), generator=g, device="cuda")
    s["idx"].masked_fill_(torch.arange(topk, device="cuda") >= found[:, None], -1)
    s["lse"] = torch.empty(rows, h, device="cuda")
    for a in range(0, rows, 64):
        s["lse"][a:a + 64] = torch.logsumexp(_picked_logits(s, slice(a, a + 64)), -1)
    return s


# ---- the plain forms ---------------------------------------------------------------------

def _turn(x, s, offset, layout, transpose=False):
    """x [n, h, d] fp32: the rotary part of each head turned to its row's position."""
    angle = s["pos"].double()[:, None] * s["freq"]
    c = angle.cos().float()[:, None]
    z = (-angle.sin() if transpose else angle.sin()).float()[:, None]
    rot = 2 * s["freq"].numel()
    part = x[..., offset:offset + rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * c - b * z, a * z + b * c], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * c - b * z, a * z + b * c], -1).flatten(-2)
    return torch.cat([x[..., :offset], part, x[..., offset + rot:]], -1)


def _normed(x, kind):
    """(x - mean) / sqrt(mean square + eps), the mean only with "layer"; and that factor."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_norm(s):
    c = s["case"]
    x, span = s["x"].float(), c["span"]
    y = _normed(x[..., :span], c["kind"])[0] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return _turn(torch.cat([y, x[..., span:]], -1), s, c["offset"], c["layout"]).to(s["x"].dtype)


def _plain_grad(s):
    c = s["case"]
    x, span = s["x"].float(), c["span"]
    g = _turn(s["dy"].float(), s, c["offset"], c["layout"], True)
    u, r = _normed(x[..., :span], c["kind"])
    du = g[..., :span] * s["weight"].float()
    dx = du - u * (du * u).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - du.mean(-1, keepdim=True)
    out = {"dx": torch.cat([dx * r, g[..., span:]], -1).to(s["x"].dtype),
           "dweight": (g[..., :span] * u).sum((0, 1))}
    if s["bias"] is not None:
        out["dbias"] = g[..., :span].sum((0, 1))
    return out


def _k_views(cache):
    p = cache.view(-1, K_PAGE_BYTES)
    return p[:, :PAGE * D_K].view(torch.float8_e4m3fn), p[:, PAGE * D_K:].view(torch.float8_e8m0fnu)


def _kv_views(cache):
    r = cache.view(-1, KV_TOKEN_BYTES)
    return r[:, :D_KV].view(torch.float8_e4m3fn), r[:, D_KV:D_KV + 20].view(torch.float32)


def _caches(k_cache, kv_cache):
    k, ks = _k_views(k_cache)
    v, vs = _kv_views(kv_cache)
    return {"k_codes": k, "k_scales": ks, "kv_codes": v, "kv_scales": vs}


def _plain_append(s):
    c = s["case"]
    k = _normed(s["k"].float(), c["kind"])[0] * s["k_weight"]
    if s["k_bias"] is not None:
        k = k + s["k_bias"]
    k = _turn(k[:, None], s, c["k_offset"], c["k_layout"])[:, 0]
    kv = s["kv"].float()
    kv = torch.cat([_normed(kv[:, :D_V], "rms")[0] * s["kv_weight"], kv[:, D_V:]], -1)
    kv = _turn(kv[:, None], s, D_V, c["kv_layout"])[:, 0]
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    at, row = (slots // PAGE)[:, None], (slots % PAGE)[:, None]
    # keys: one power of two a group of 32
    g = k[keep].view(-1, 4, 32)
    e = torch.frexp(g.abs().amax(-1))[1] - 9
    codes = (g * torch.exp2(-e.float())[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    page = s["k_cache"].view(-1, K_PAGE_BYTES)
    page[at, row * D_K + torch.arange(D_K, device="cuda")] = codes.view(-1, D_K).view(torch.uint8)
    page[at, PAGE * D_K + row * 4 + torch.arange(4, device="cuda")] = (e + 127).to(torch.uint8)
    # latent rows: amax / 448 of each 128, the last tile 64 wide
    t = torch.nn.functional.pad(kv[keep], (0, 64)).view(-1, 5, 128)
    scales = t.abs().amax(-1) / E4M3_MAX
    codes = (t / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1, 640)[:, :D_KV]
    record = s["kv_cache"].view(-1, KV_TOKEN_BYTES)
    record[slots, :D_KV] = codes.contiguous().view(torch.uint8)
    record[slots, D_KV:D_KV + 20] = scales.contiguous().view(torch.uint8)
    return _caches(s["k_cache"], s["kv_cache"])


def _rows_of(cache, slots, dtype):
    """The dequantised latent rows at the cache slots, any shape."""
    rec = cache.view(-1, KV_TOKEN_BYTES)[slots]
    codes = rec[..., :D_KV].contiguous().view(torch.float8_e4m3fn).to(dtype)
    scales = rec[..., D_KV:D_KV + 20].contiguous().view(torch.float32).to(dtype)
    return codes * scales.repeat_interleave(128, -1)[..., :D_KV]


def _slots(table, pos):
    return table.long().gather(-1, pos // PAGE) * PAGE + pos % PAGE


def _logits(s):
    """Every row over its sequence's positions [seqs, per_seq, h, max_ctx] fp32; -inf where it does not see one."""
    c = s["case"]
    p = torch.arange(s["max_ctx"], device="cuda")
    kv = _rows_of(s["kv_cache"], _slots(s["table"], p.expand(c["seqs"], -1)), torch.float32)
    a = torch.bmm(s["q"].float().view(c["seqs"], -1, D_KV) * SM_SCALE, kv.transpose(1, 2))
    a = a.view(c["seqs"], c["per_seq"], c["h"], -1)
    seen = torch.minimum(s["q_pos"].view(c["seqs"], -1) + 1, s["seq_lens"][:, None])
    return a.masked_fill_((p >= seen[..., None])[:, :, None], float("-inf"))


def _plain_mass(s):
    c = s["case"]
    a = _logits(s).sub_(s["lse"].view(c["seqs"], c["per_seq"], c["h"], 1)).exp_()
    return a.sum((1, 2))


def _picked_logits(s, rows):
    """Rows over their selected entries [rows, h, topk] fp32; -inf at empty entries."""
    idx = s["idx"][rows].long()
    kv = _rows_of(s["kv_cache"], _slots(s["table"][s["q_seq"][rows].long()], idx.clamp(min=0)), torch.float32)
    a = torch.bmm(s["q"][rows].float() * SM_SCALE, kv.transpose(1, 2))
    return a.masked_fill_((idx < 0)[:, None], float("-inf"))


def _plain_picked(s):
    # (a row without entries has an lse of -inf, and logits of -inf)
    lse = s["lse"].masked_fill(s["lse"] == float("-inf"), 0.0)
    weights = _picked_logits(s, slice(None)).sub_(lse[..., None]).exp_().sum(1)
    mass = torch.zeros(s["case"]["seqs"], s["max_ctx"], device="cuda", dtype=torch.float64)
    idx = s["idx"].long()
    at = s["q_seq"].long()[:, None] * s["max_ctx"] + idx.clamp(min=0)
    mass.view(-1).index_add_(0, at.view(-1), weights.double().view(-1))
    return {"weights": weights, "mass": mass.float()}


def _plain_select(s):
    """The positions that stay, in order, -1 behind them; how many; their accumulated weights."""
    c = s["case"]
    p, lens = torch.arange(c["hi"], device="cuda"), s["seq_lens"].long()[:, None]
    most = torch.iinfo(torch.int64).max
    m = s["mass"].masked_fill((p < c["sinks"]) | (p >= lens - c["recent"]), most).masked_fill(p >= lens, -1)
    best = torch.sort(m, dim=1, descending=True, stable=True).indices[:, :c["budget"]]
    kept = torch.sort(best.masked_fill(best >= lens, most), dim=1).values
    kept = torch.nn.functional.pad(kept, (0, c["budget"] - kept.shape[1]), value=most)
    mass = s["mass"].gather(1, kept.clamp(max=c["hi"] - 1)).masked_fill(kept == most, 0)
    return kept.masked_fill(kept == most, -1).to(torch.int32), s["seq_lens"].clamp(max=c["budget"]), mass


def _plain_evict(s):
    c = s["case"]
    kept, lens, mass = _plain_select(s)
    table = s["table"] if s["dst"] is None else s["dst"]
    there = kept >= 0
    i = torch.arange(c["budget"], device="cuda").expand_as(kept)
    src = _slots(s["table"], kept.long().clamp(min=0))[there]
    dst = _slots(table, i.clamp(max=table.shape[1] * PAGE - 1))[there]
    record = s["kv_cache"].view(-1, KV_TOKEN_BYTES)
    record[dst] = record[src]
    page = s["k_cache"].view(-1, K_PAGE_BYTES)
    codes, scales = page[:, :PAGE * D_K].view(-1, PAGE, D_K), page[:, PAGE * D_K:].view(-1, PAGE, 4)
    codes[dst // PAGE, dst % PAGE] = codes[src // PAGE, src % PAGE]
    scales[dst // PAGE, dst % PAGE] = scales[src // PAGE, src % PAGE]
    return kept, lens, mass


def _evicted(s, kept, lens, mass):
    first = 0 if s["dst"] is None else s["old"]
    return {"kept": kept, "lens": lens, "mass": mass,
            **_caches(s["k_cache"][first * K_PAGE_BYTES:], s["kv_cache"][first * PAGE * KV_TOKEN_BYTES:])}


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import dsa_sparse_attention_topk_gb300 as dsa
        if op == "norm":
            return dsa.norm_rope(s["x"], s["pos"], s["turns"], weight=s["weight"], bias=s["bias"], norm=c["kind"],
                                 norm_dim=c["span"], eps=EPS, offset=c["offset"], layout=c["layout"])
        if op == "grad":
            dx, dweight, dbias = dsa.norm_rope_grad(s["dy"], s["x"], s["pos"], s["turns"], weight=s["weight"],
                                                    bias=s["bias"], norm=c["kind"], norm_dim=c["span"], eps=EPS,
                                                    offset=c["offset"], layout=c["layout"])
            return {"dx": dx, "dweight": dweight, **({} if dbias is None else {"dbias": dbias})}
        if op == "append":
            dsa.norm_rope_quant_kv(s["k"], s["kv"], s["pos"], s["slots"], s["k_cache"], s["kv_cache"], s["turns"],
                                   k_weight=s["k_weight"], k_bias=s["k_bias"], kv_weight=s["kv_weight"],
                                   k_norm=c["kind"], eps=EPS, k_offset=c["k_offset"], k_layout=c["k_layout"],
                                   kv_layout=c["kv_layout"])
            return _caches(s["k_cache"], s["kv_cache"])
        if op == "mass":
            mass = dsa.attn_mass(s["q"], s["kv_cache"], s["table"], s["seq_lens"], s["q_seq"], s["q_pos"], s["lse"],
                                 s["max_ctx"], SM_SCALE)
            return mass.float().mul_(MASS_UNIT)
        if op == "picked":
            mass = torch.zeros(c["seqs"], s["max_ctx"], dtype=torch.int64, device="cuda")
            weights = dsa.sparse_attn_mass(s["q"], s["kv_cache"], s["table"], s["seq_lens"], s["q_seq"], s["idx"],
                                           s["lse"], SM_SCALE, mass=mass)
            return {"weights": weights, "mass": mass.float().mul_(MASS_UNIT)}
        kept, lens, mass = dsa.evict_select(s["mass"], s["seq_lens"], c["budget"], sinks=c["sinks"], recent=c["recent"])
        dsa.evict_compact(kept, s["table"], s["k_cache"], s["kv_cache"], dst_table=s["dst"])
        return _evicted(s, kept, lens, mass)
    if op == "evict":
        return _evicted(s, *_plain_evict(s))
    return {"norm": _plain_norm, "grad": _plain_grad, "append": _plain_append, "mass": _plain_mass,
            "picked": _plain_picked}[op](s)


def work(case):
    op = case["op"]
    if op in ("norm", "grad"):
        rows, size = case["n"] * case["h"], 4 if case["dtype"] == "fp32" else 2
        moved = (3 if op == "grad" else 2) * rows * case["d"] * size
        return {"bytes": moved + 4 * case["n"] + 8 * case["span"],
                "flops": rows * ((9 if op == "grad" else 4) * case["span"] + 3 * case["rot"])}
    if op == "append":
        # bf16 rows, positions and slots read; codes and scales written
        return {"bytes": case["n"] * (2 * (D_K + D_KV) + 12 + D_K + 4 + KV_TOKEN_BYTES),
                "flops": case["n"] * (3 * 2 * ROT + 7 * (D_K + D_KV))}
    if op == "evict":
        mid = (case["lo"] + case["hi"]) / 2
        kept = case["seqs"] * min(mid, case["budget"])
        return {"bytes": 8 * case["seqs"] * mid + 12 * kept + 2 * kept * (KV_TOKEN_BYTES + D_K + 4), "flops": 0}
    rows = case["seqs"] * case["per_seq"]
    if op == "mass":
        mid = (case["lo"] + case["hi"]) / 2
        seen = mid - (case["per_seq"] - 1) / 2
        return {"bytes": 596 * case["seqs"] * mid + rows * case["h"] * (2 * D_KV + 4) + 4 * case["seqs"] * case["hi"],
                "flops": 2.0 * (D_KV + 1) * rows * case["h"] * seen}
    # the entries of all rows of a sequence lie among its positions, each of which need be read once
    entries = rows * (case["fewest"] + min(case["topk"], case["ctx"])) / 2
    return {"bytes": 596 * min(entries, case["seqs"] * case["ctx"]) + rows * case["h"] * (2 * D_KV + 4)
            + 8 * rows * case["topk"] + 4 * case["seqs"] * case["ctx"],
            "flops": 2.0 * (D_KV + 1) * entries * case["h"]}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _turned64(x, pos, rot, offset, layout, sign):
    freq = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    angle = pos.double().view(-1, 1, 1) * freq
    z = torch.polar(torch.ones_like(angle), sign * angle)
    y = x.double().clone()
    i = torch.arange(rot // 2, device="cuda")
    first, second = (offset + i, offset + rot // 2 + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _norm64(x, weight, bias, kind):
    """The norm of the last dim in 64 bits, differentiable."""
    mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS) * weight.double()
    return y if bias is None else y + bias.double()


def _e4m3_64(x):
    """The nearest E4M3 value, ties to even, saturating."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)   # x = m 2^(e+1), m in [1/2, 1)
    step = torch.exp2((e - 3).double())
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _weights64(q, kv, lse, seen):
    """sum over rows and heads of exp(q . kv - lse): q [rows, h, 576], kv [m, 576], seen [rows, m]."""
    total = torch.zeros(len(kv), dtype=torch.float64, device="cuda")
    for r in range(len(q)):
        a = torch.exp(q[r].double() @ kv.T * SM_SCALE - lse[r].double()[:, None]).sum(0)
        total += torch.where(seen[r], a, 0.0)
    return total


def _evicted64(s):
    """One sequence after another, in the order of (weight, position) pairs; values as 64-bit numbers."""
    c, n = s["case"], s["case"]["budget"]
    old_k = {name: v.double() for name, v in zip(("codes", "scales"), _k_views(s["k_cache"]))}
    old_v = {name: v.double() for name, v in zip(("codes", "scales"), _kv_views(s["kv_cache"]))}
    k = {"codes": old_k["codes"].view(-1, D_K), "scales": old_k["scales"].view(-1, 4)}
    new_k, new_v = {x: v.clone() for x, v in k.items()}, {x: v.clone() for x, v in old_v.items()}
    kept = torch.full((c["seqs"], n), -1, dtype=torch.int32, device="cuda")
    mass = torch.zeros(c["seqs"], n, dtype=torch.int64, device="cuda")
    to = s["table"] if s["dst"] is None else s["dst"]
    lens = s["seq_lens"].tolist()
    for b, length in enumerate(lens):
        first, last = min(c["sinks"], length), max(length - c["recent"], 0)
        always = [p for p in range(length) if p < first or p >= last]
        m = s["mass"][b, :length].cpu()
        others = torch.ones(length, dtype=torch.bool)
        others[always] = False
        free = others.nonzero()[:, 0]
        at = torch.argsort(m[free], descending=True, stable=True)[:n - len(always)]
        stay = torch.sort(torch.cat([torch.tensor(always, dtype=torch.int64), free[at]])).values.to("cuda")
        i = torch.arange(len(stay), device="cuda")
        kept[b, :len(stay)], mass[b, :len(stay)] = stay.int(), s["mass"][b][stay]
        src = s["table"][b].long()[stay // PAGE] * PAGE + stay % PAGE
        dst = to[b].long()[i // PAGE] * PAGE + i % PAGE
        for old, new in ((k, new_k), (old_v, new_v)):
            for x in old:
                new[x][dst] = old[x][src]
    first = 0 if s["dst"] is None else s["old"]
    return {"kept": kept, "lens": torch.tensor([min(x, n) for x in lens], dtype=torch.int32, device="cuda"), "mass": mass,
            "k_codes": new_k["codes"].view(-1, PAGE * D_K)[first:], "k_scales": new_k["scales"].view(-1, PAGE * 4)[first:],
            "kv_codes": new_v["codes"][first * PAGE:], "kv_scales": new_v["scales"][first * PAGE:]}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "grad"):
        span, sizes = case["span"], case["n"] * case["h"] * case["d"]
        if sizes > 200_000_000:
            return None
        x = s["x"].double()
        u, rest = x[..., :span], x[..., span:]
        if op == "norm":
            y = torch.cat([_norm64(u, s["weight"], s["bias"], case["kind"]), rest], -1)
            return _turned64(y, s["pos"], case["rot"], case["offset"], case["layout"], 1.0)
        g = _turned64(s["dy"], s["pos"], case["rot"], case["offset"], case["layout"], -1.0)
        with torch.enable_grad():
            leaves = [u.detach().requires_grad_(), s["weight"].double().requires_grad_()]
            if s["bias"] is not None:
                leaves.append(s["bias"].double().requires_grad_())
            y = _norm64(leaves[0], leaves[1], leaves[2] if len(leaves) > 2 else None, case["kind"])
            du, dw, *db = torch.autograd.grad(y, leaves, g[..., :span].contiguous())
        return {"dx": torch.cat([du, g[..., span:]], -1), "dweight": dw, **({"dbias": db[0]} if db else {})}
    if op == "append":
        pages = case["pages"]
        k = _norm64(s["k"].double(), s["k_weight"], s["k_bias"], case["kind"])
        k = _turned64(k[:, None], s["pos"], ROT, case["k_offset"], case["k_layout"], 1.0)[:, 0]
        kv = torch.cat([_norm64(s["kv"][:, :D_V].double(), s["kv_weight"], None, "rms"), s["kv"][:, D_V:].double()], -1)
        kv = _turned64(kv[:, None], s["pos"], ROT, D_V, case["kv_layout"], 1.0)[:, 0]
        keep = s["slots"] >= 0
        slots, k, kv = s["slots"][keep], k[keep].view(-1, 4, 32), kv[keep]
        power = torch.exp2((torch.frexp(k.abs().amax(-1, True))[1] - 9).double())
        out = {"k_codes": torch.zeros(pages * PAGE, D_K, dtype=torch.float64, device="cuda"),
               "k_scales": torch.full((pages * PAGE, 4), 2.0 ** -127, dtype=torch.float64, device="cuda"),
               "kv_codes": torch.zeros(pages * PAGE, D_KV, dtype=torch.float64, device="cuda"),
               "kv_scales": torch.zeros(pages * PAGE, 5, dtype=torch.float64, device="cuda")}
        out["k_codes"][slots] = _e4m3_64(k / power).view(-1, D_K)
        out["k_scales"][slots] = power[..., 0]
        for t, (a, b) in enumerate([(0, 128), (128, 256), (256, 384), (384, 512), (512, 576)]):
            scale = kv[:, a:b].abs().amax(-1, True) / E4M3_MAX
            out["kv_scales"][slots, t] = scale[:, 0]
            out["kv_codes"][slots, a:b] = _e4m3_64(kv[:, a:b] / scale.float().double())
        out["k_codes"] = out["k_codes"].view(pages, -1)
        out["k_scales"] = out["k_scales"].view(pages, -1)
        return out
    if op == "evict":
        return _evicted64(s)
    table, lens, seqs = s["table"].long(), s["seq_lens"].tolist(), s["q_seq"].tolist()
    if op == "mass":
        out = torch.zeros(case["seqs"], case["hi"], dtype=torch.float64, device="cuda")
        for b in range(case["seqs"]):
            j = torch.arange(lens[b], device="cuda")
            kv = _rows_of(s["kv_cache"], table[b][j // PAGE] * PAGE + j % PAGE, torch.float64)
            r = [t for t, x in enumerate(seqs) if x == b]
            seen = j <= s["q_pos"][r].long()[:, None]
            out[b, :lens[b]] = _weights64(s["q"][r], kv, s["lse"][r], seen)
        return out
    weights = torch.zeros(len(seqs), case["topk"], dtype=torch.float64, device="cuda")
    mass = torch.zeros(case["seqs"], case["ctx"], dtype=torch.float64, device="cuda")
    for t, b in enumerate(seqs):
        entry = (s["idx"][t] >= 0).nonzero()[:, 0]
        j = s["idx"][t][entry].long()
        if len(j) == 0:
            continue
        kv = _rows_of(s["kv_cache"], table[b][j // PAGE] * PAGE + j % PAGE, torch.float64)
        w = _weights64(s["q"][t:t + 1], kv, s["lse"][t:t + 1], torch.ones(1, len(j), dtype=torch.bool, device="cuda"))
        weights[t, entry] = w
        mass[b, j] += w
    return {"weights": weights, "mass": mass}
