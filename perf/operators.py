"""Cases of the rotary, rotated-append and shared-prefix operators, each with its plain form.

``run`` computes a case in elementary torch operations (32 bits; angles in 64) where ``own`` is false, and through the
package's entry points where it is true.  ``exact`` is the operators' definition in 64 bits, written apart from both.

The sizes are those of the package's own workloads (indexer heads of 128, latent rows of 576 = 512 + 64 rotary, 64-token
pages, contexts of 32K and 128K, chunks of 4096 rows) and odd ones around them."""

import math

import torch

own = False

PAGE, D_K, D_KV, D_V, ROT = 64, 128, 576, 512, 64
K_PAGE_BYTES, KV_TOKEN_BYTES = 8448, 608
SM_SCALE = 1.0 / math.sqrt(192.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------------

def _rope(name, n, h, d, offset, rot, layout, transpose, dtype, pos_max, factor, pad):
    return {"name": name, "op": "rope", "n": n, "h": h, "d": d, "offset": offset, "rot": rot, "layout": layout,
            "transpose": transpose, "dtype": dtype, "pos_max": pos_max, "factor": factor, "pad": pad}


def _append(name, n, pages, pos_max, k_offset, k_layout, kv_layout, factor):
    return {"name": name, "op": "append", "n": n, "pages": pages, "pos_max": pos_max, "k_offset": k_offset,
            "k_layout": k_layout, "kv_layout": kv_layout, "factor": factor}


def _prefix(name, seqs, per_seq, h, prefix, tail_lo, tail_hi):
    return {"name": name, "op": "prefix", "seqs": seqs, "per_seq": per_seq, "h": h, "prefix": prefix,
            "tail_lo": tail_lo, "tail_hi": tail_hi}


def listed():
    return [
        # one row's indexer query at the end of a 128K context: latency alone
        _rope("rope_one_row", 1, 64, 128, 0, 64, "half", False, "bf16", 131072, 1.0, 0),
        # the attention queries of a decode batch of 32, rotary part behind the 512 others, long-context frequencies
        _rope("rope_decode_b32", 32, 128, 576, 512, 64, "interleaved", False, "bf16", 32768, 40.0, 0),
        # the attention queries of a chunk of 4096 prompt rows
        _rope("rope_chunk_4k", 4096, 128, 576, 512, 64, "interleaved", False, "bf16", 65536, 40.0, 0),
        # the gradient of such a rotation in fp32, odd token and head counts, rows inside a wider projection
        _rope("rope_grad_fp32", 2047, 63, 128, 64, 64, "half", True, "fp32", 65536, 1.0, 64),
        # the new tokens of a decode batch of 32
        _append("append_decode_b32", 32, 64, 32768, 0, "half", "interleaved", 40.0),
        # a chunk of 4096 prompt tokens (an odd number of them)
        _append("append_chunk_4k", 4095, 64, 65536, 0, "half", "interleaved", 40.0),
        # a whole 64K prompt, rotary part of the key at the end of the head
        _append("append_prompt_64k", 65536, 1024, 65536, 64, "interleaved", "half", 1.0),
        # one row with the heads of one of eight shards over a short prompt: latency alone
        _prefix("prefix_one_row", 1, 1, 16, 250, 7, 7),
        # a decode batch of 32 over one 32K system prompt, own tails of a chat's length
        _prefix("prefix_decode_b32_32k", 32, 1, 128, 32768, 64, 1024),
        # two-token steps of 4 sequences that share a 128K document
        _prefix("prefix_mtp_b4_128k", 4, 2, 128, 131000, 3, 300),
        # 128 rows with the heads of one of eight shards, ragged tails as long as the prefix
        _prefix("prefix_shard_b128_2k", 128, 1, 16, 2048, 1, 2048),
        # a chunk of 512 prompt rows (causal among themselves) behind a 16K prefix
        _prefix("prefix_chunk_512", 1, 512, 128, 16384, 512, 512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix", "prefix"])
    if op == "rope":
        d = rng.choice([64, 128, 192, 576, 100])
        rot = rng.choice([r for r in (32, 64, 64, 96, 128, 50) if r <= d])
        offset = rng.choice([0, d - rot])
        h = rng.choice([1, 3, 8, 16, 63, 64, 128])
        n = _log(rng, 1, max(1, min(65536, 150_000_000 // (h * d))))
        return _rope("", n, h, d, offset, rot, rng.choice(["half", "interleaved"]), rng.random() < 0.4,
                     rng.choice(["bf16", "bf16", "fp16", "fp32"]), _log(rng, 4096, 1 << 20),
                     rng.choice([1.0, 8.0, 40.0]), rng.choice([0, 0, 64, 4]))
    if op == "append":
        n = _log(rng, 1, 65536)
        return _append("", n, (n + PAGE - 1) // PAGE + rng.randrange(1, 40), _log(rng, 65536, 1 << 20),
                       rng.choice([0, 64, 32, 4 * rng.randrange(0, 17)]), rng.choice(["half", "interleaved"]),
                       rng.choice(["half", "interleaved"]), rng.choice([1.0, 40.0]))
    while True:
        seqs, per_seq, h = _log(rng, 1, 128), rng.choice([1, 1, 2, 3, 64]), rng.choice([1, 5, 16, 32, 64, 128, 128])
        prefix, hi = _log(rng, 1, 131072), _log(rng, 1, 2048)
        c = _prefix("", seqs, per_seq, h, prefix, rng.randrange(1, hi + 1), hi)
        rows = seqs * per_seq
        # (a tail shorter than per_seq puts a sequence's first rows inside the prefix)
        if prefix + c["tail_lo"] >= per_seq and rows * (prefix + hi) * h <= 600_000_000 and rows * hi <= 262144:
            return c


# ---- inputs ----------------------------------------------------------------------------

def _inv_freq(rot, factor, base=10000.0, trained=4096):
    """Rotary frequencies (radians a position); factor > 1: interpolated by parts (yarn), with its amplitude."""
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if factor == 1.0:
        return theta, 1.0
    at = lambda turns: rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
    return [t * (1 - r) + t / factor * r for t, r in zip(theta, ramp)], 0.1 * math.log(factor) + 1.0


def _angles(rot, factor):
    f, amplitude = _inv_freq(rot, factor)
    # the package takes turns a position in 64-bit fixed point
    turns = [round(v / (2 * math.pi) * 2.0 ** 64) for v in f]
    return {"freq": torch.tensor(f, dtype=torch.float64, device="cuda"),
            "turns": torch.tensor(turns, dtype=torch.int64, device="cuda"), "amplitude": amplitude}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "rope":
        n, h, d = case["n"], case["h"], case["d"]
        x = randn(n, h, d + case["pad"]).to(DTYPES[case["dtype"]])[..., :d]
        # rows of a batch at any position, or a chunk's consecutive ones
        pos = torch.randint(0, case["pos_max"], (n,), generator=g, device="cuda", dtype=torch.int32)
        if n > 512:
            pos = (torch.arange(n, device="cuda", dtype=torch.int32) + pos[0]).clamp_(max=case["pos_max"])
        return {"case": case, "x": x, "pos": pos, **_angles(case["rot"], case["factor"])}
    if case["op"] == "append":
        n, pages = case["n"], case["pages"]
        k = randn(n, D_K)
        k[:, torch.randperm(D_K, generator=g, device="cuda")[:4]] *= 8  # outlier channels
        kv = randn(n, D_KV)
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
                "k_cache": torch.zeros(pages * K_PAGE_BYTES, dtype=torch.uint8, device="cuda"),
                "kv_cache": torch.zeros(pages * PAGE * KV_TOKEN_BYTES, dtype=torch.uint8, device="cuda"),
                **_angles(ROT, case["factor"])}
    seqs, per_seq, h, prefix = case["seqs"], case["per_seq"], case["h"], case["prefix"]
    u = torch.rand(seqs, generator=g, device="cuda")
    lo, hi = case["tail_lo"], case["tail_hi"]
    tails = (lo + (u * (hi - lo + 1)).long()).clamp(max=hi)
    tails[0] = hi
    seq_lens = (prefix + tails).to(torch.int32)
    shared = prefix // PAGE                       # whole pages are shared; the last, partial one is each sequence's copy
    per = (prefix + hi + PAGE - 1) // PAGE
    mine = per - shared
    pages = shared + seqs * mine
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.empty(seqs, per, dtype=torch.int32, device="cuda")
    table[:, :shared] = perm[:shared]
    table[:, shared:] = perm[shared:].view(seqs, mine)
    cache = torch.zeros(pages * PAGE, KV_TOKEN_BYTES, dtype=torch.uint8, device="cuda")
    for a in range(0, pages * PAGE, 65536):
        rows = randn(min(65536, pages * PAGE - a), D_KV).to(torch.bfloat16).float()
        codes, scales = _fp8_tiles(rows)
        cache[a:a + len(rows), :D_KV] = codes.view(torch.uint8)
        cache[a:a + len(rows), D_KV:D_KV + 20] = scales.contiguous().view(torch.uint8)
    rows = seqs * per_seq
    q_seq = torch.arange(seqs, device="cuda", dtype=torch.int32).repeat_interleave(per_seq)
    q_pos = seq_lens[q_seq.long()] - per_seq + torch.arange(per_seq, device="cuda", dtype=torch.int32).repeat(seqs)
    return {"case": case, "q": randn(rows, h, D_KV).to(torch.bfloat16), "kv_cache": cache.view(-1),
            "prefix_pages": table[0, :(prefix + PAGE - 1) // PAGE].contiguous(), "table": table, "seq_lens": seq_lens,
            "q_seq": q_seq, "q_pos": q_pos.to(torch.int32), "max_ctx": prefix + hi}


# ---- the plain forms ---------------------------------------------------------------------

def _rotate(x, pos, freq, amplitude, offset, layout, transpose):
    """x [n, h, d] fp32: the rotary part of each head turned by pos * freq, times the amplitude."""
    rot = 2 * freq.numel()
    angle = pos.double()[:, None] * freq
    c = (angle.cos() * amplitude).float()[:, None, :]
    s = (angle.sin() * (-amplitude if transpose else amplitude)).float()[:, None, :]
    part = x[..., offset:offset + rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([x[..., :offset], part, x[..., offset + rot:]], -1)


def _mxfp8(x):
    """x [n, 128] fp32 -> E4M3 codes [n, 128], E8M0 scales [n, 4]: one power of two a group of 32."""
    g = x.view(-1, D_K // 32, 32)
    amax = g.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 9).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    inverse = ((127 - e) << 23).to(torch.int32).view(torch.float32)
    codes = (g * inverse[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(-1, D_K), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _to_e4m3(x):
    """64-bit values within +-448 -> the nearest E4M3 codes, ties to even."""
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).to(torch.float8_e4m3fn)


def _fp8_tiles(x):
    """x [n, 576] fp32 -> E4M3 codes [n, 576], fp32 scales [n, 5]: amax / 448 of each 128 (the last tile 64 wide)."""
    t = torch.nn.functional.pad(x, (0, 64)).view(-1, 5, 128)
    scales = (t.abs().amax(-1).double() / E4M3_MAX).float()
    # (the quotient in 64 bits: of bf16 values it often lies next to a border between two codes)
    q = t.double() / torch.where(scales > 0, scales, torch.ones_like(scales))[..., None].double()
    codes = _to_e4m3(q.clamp(-E4M3_MAX, E4M3_MAX).view(-1, 640)[:, :D_KV])
    return codes, scales


def _k_views(cache):
    p = cache.view(-1, K_PAGE_BYTES)
    return p[:, :PAGE * D_K].view(torch.float8_e4m3fn), p[:, PAGE * D_K:].view(torch.float8_e8m0fnu)


def _kv_views(cache):
    r = cache.view(-1, KV_TOKEN_BYTES)
    return r[:, :D_KV].view(torch.float8_e4m3fn), r[:, D_KV:D_KV + 20].view(torch.float32)


def _caches(s):
    k, ks = _k_views(s["k_cache"])
    v, vs = _kv_views(s["kv_cache"])
    return {"k_codes": k, "k_scales": ks, "kv_codes": v, "kv_scales": vs}


def _plain_append(s):
    c = s["case"]
    k = _rotate(s["k"].float()[:, None], s["pos"], s["freq"], s["amplitude"], c["k_offset"], c["k_layout"], False)[:, 0]
    kv = _rotate(s["kv"].float()[:, None], s["pos"], s["freq"], s["amplitude"], D_V, c["kv_layout"], False)[:, 0]
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    codes, scales = _mxfp8(k[keep])
    page = s["k_cache"].view(-1, K_PAGE_BYTES)
    at, row = (slots // PAGE)[:, None], (slots % PAGE)[:, None]
    page[at, row * D_K + torch.arange(D_K, device="cuda")] = codes.view(torch.uint8)
    page[at, PAGE * D_K + row * 4 + torch.arange(4, device="cuda")] = scales.view(torch.uint8)
    codes, scales = _fp8_tiles(kv[keep])
    record = s["kv_cache"].view(-1, KV_TOKEN_BYTES)
    record[slots, :D_KV] = codes.view(torch.uint8)
    record[slots, D_KV:D_KV + 20] = scales.contiguous().view(torch.uint8)
    return _caches(s)


def _rows_of(cache, slots, dtype):
    """The dequantised latent rows at the cache slots, any shape."""
    rec = cache.view(-1, KV_TOKEN_BYTES)[slots]
    codes = rec[..., :D_KV].contiguous().view(torch.float8_e4m3fn).to(dtype)
    scales = rec[..., D_KV:D_KV + 20].contiguous().view(torch.float32).to(dtype)
    return codes * scales.repeat_interleave(128, -1)[..., :D_KV]


def _slots(table, pos):
    return table.long().gather(-1, pos // PAGE) * PAGE + pos % PAGE


def _plain_prefix(s):
    c = s["case"]
    prefix, rows, h = c["prefix"], s["q"].shape[0], c["h"]
    p = torch.arange(prefix, device="cuda")
    shared = _rows_of(s["kv_cache"], _slots(s["prefix_pages"], p), torch.float32)
    t = torch.arange(prefix, s["max_ctx"], device="cuda")
    seq = s["q_seq"].long()
    limit = torch.minimum(s["q_pos"] + 1, s["seq_lens"][seq]).long()
    tail = _rows_of(s["kv_cache"], _slots(s["table"], t.expand(c["seqs"], -1)), torch.float32)[seq]
    q = s["q"].float() * SM_SCALE
    a = (q.view(rows * h, D_KV) @ shared.T).view(rows, h, prefix)
    a.masked_fill_((p >= limit[:, None])[:, None], float("-inf"))
    b = torch.bmm(q, tail.transpose(1, 2))
    b.masked_fill_((t >= limit[:, None])[:, None], float("-inf"))
    top = torch.maximum(a.amax(-1, True), b.amax(-1, True))
    a, b = a.sub_(top).exp_(), b.sub_(top).exp_()
    total = a.sum(-1, True) + b.sum(-1, True)
    o = (a.view(rows * h, prefix) @ shared[:, :D_V]).view(rows, h, D_V) + torch.bmm(b, tail[..., :D_V])
    return (o / total).to(torch.bfloat16)


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        import dsa_sparse_attention_topk_gb300 as dsa
        if c["op"] == "rope":
            return dsa.rope(s["x"], s["pos"], s["turns"], offset=c["offset"], layout=c["layout"],
                            amplitude=s["amplitude"], transpose=c["transpose"])
        if c["op"] == "append":
            dsa.rope_quant_kv(s["k"], s["kv"], s["pos"], s["slots"], s["k_cache"], s["kv_cache"], s["turns"],
                              amplitude=s["amplitude"], k_offset=c["k_offset"], k_layout=c["k_layout"],
                              kv_layout=c["kv_layout"])
            return _caches(s)
        return dsa.prefix_attn(s["q"], s["kv_cache"], s["prefix_pages"], c["prefix"], s["table"], s["seq_lens"],
                               s["q_seq"], s["q_pos"], s["max_ctx"], SM_SCALE)[0]
    if c["op"] == "rope":
        return _rotate(s["x"].float(), s["pos"], s["freq"], s["amplitude"], c["offset"], c["layout"],
                       c["transpose"]).to(s["x"].dtype)
    return _plain_append(s) if c["op"] == "append" else _plain_prefix(s)


def work(case):
    if case["op"] == "rope":
        values = case["n"] * case["h"] * case["d"]
        size = 4 if case["dtype"] == "fp32" else 2
        turned = case["n"] * case["h"] * case["rot"]
        return {"bytes": 2 * values * size + 4 * case["n"] + 8 * (case["rot"] // 2), "flops": 3 * turned}
    if case["op"] == "append":
        # bf16 rows, positions and slots read; codes and scales written
        return {"bytes": case["n"] * (2 * (D_K + D_KV) + 12 + D_K + 4 + KV_TOKEN_BYTES),
                "flops": case["n"] * (3 * 2 * ROT + 2 * (D_K + D_KV))}
    rows = case["seqs"] * case["per_seq"]
    tail = (case["tail_lo"] + case["tail_hi"]) / 2
    seen = case["prefix"] + tail - (case["per_seq"] - 1) / 2
    return {"bytes": 596 * (case["prefix"] + case["seqs"] * tail) + rows * case["h"] * 2 * (D_KV + D_V),
            "flops": 2.0 * (D_KV + D_V) * rows * case["h"] * seen}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _turned64(x, pos, rot, factor, offset, layout, sign):
    freq, amplitude = _inv_freq(rot, factor)
    angle = pos.double().view(-1, 1, 1) * torch.tensor(freq, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(angle, amplitude), sign * angle)
    y = x.double().clone()
    half = rot // 2
    i = torch.arange(half, device="cuda")
    first, second = (offset + i, offset + half + i) if layout == "half" else (offset + 2 * i, offset + 2 * i + 1)
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _e4m3_64(x):
    """The nearest E4M3 value, ties to even, saturating."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)   # x = m 2^(e+1), m in [1/2, 1)
    step = torch.exp2((e - 3).double())
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned64(s["x"], s["pos"], case["rot"], case["factor"], case["offset"], case["layout"],
                         -1.0 if case["transpose"] else 1.0)
    if case["op"] == "append":
        pages = case["pages"]
        k = _turned64(s["k"][:, None], s["pos"], ROT, case["factor"], case["k_offset"], case["k_layout"], 1.0)[:, 0]
        kv = _turned64(s["kv"][:, None], s["pos"], ROT, case["factor"], D_V, case["kv_layout"], 1.0)[:, 0]
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
    out = torch.empty(*s["q"].shape[:2], D_V, dtype=torch.float64, device="cuda")
    prefix, h = case["prefix"], case["h"]
    i = torch.arange(prefix, device="cuda")
    shared = _rows_of(s["kv_cache"], s["prefix_pages"].long()[i // PAGE] * PAGE + i % PAGE, torch.float64)
    lens, seqs, at = s["seq_lens"].tolist(), s["q_seq"].tolist(), s["q_pos"].tolist()
    for b in range(case["seqs"]):
        j = torch.arange(prefix, lens[b], device="cuda")
        kv = torch.cat([shared, _rows_of(s["kv_cache"], s["table"][b].long()[j // PAGE] * PAGE + j % PAGE,
                                         torch.float64)])
        mine = [r for r, x in enumerate(seqs) if x == b]
        for r0 in range(0, len(mine), 64):
            r = torch.tensor(mine[r0:r0 + 64], device="cuda")
            n = torch.tensor([min(at[x] + 1, lens[b]) for x in mine[r0:r0 + 64]], device="cuda")
            logits = (s["q"][r].double().view(-1, D_KV) @ kv.T).view(len(r), h, -1) * SM_SCALE
            logits = torch.where((torch.arange(len(kv), device="cuda") < n[:, None])[:, None], logits, float("-inf"))
            out[r] = (torch.softmax(logits, -1).view(len(r) * h, -1) @ kv[:, :D_V]).view(len(r), h, D_V)
    return out
