"""A call on a stream that is not the current one: what it allocates belongs to that stream.

A workspace is dropped when the call returns, while its kernels have yet to run.  The allocator
gives a block back to the stream that it was allocated on, at once: taken from the current stream,
the next allocation there would get the memory that the kernels on the other stream still use."""

import contextlib
import math

import pytest
import torch

import dsa_sparse_attention_topk_gb300 as pkg
from dsa_testlib import ensure_built

SM = 1.0 / math.sqrt(192.0)


class _Library:
    """Entry points that do nothing, and workspace sizes of 512 bytes."""

    def __getattr__(self, name):
        return lambda *a: 512 if name.endswith("_workspace_size") else 0


class _Stream:
    cuda_stream = 77


@pytest.fixture
def traced(monkeypatch):
    """The binding on CPU tensors; yields the list of (bytes, on the call's stream, recorded on the caller's)."""
    here, seen = [], []
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        here.append(s)
        yield
        here.pop()

    def traced_empty(*a, **kw):
        t = empty(*a, **kw)
        seen.append([t.numel() * t.element_size(), list(here), False, t.data_ptr()])
        return t

    def record(t, s):
        assert s == "current"
        for e in seen:
            if e[3] == t.data_ptr():
                e[2] = True

    monkeypatch.setattr(pkg, "lib", _Library)
    monkeypatch.setattr(pkg, "_same_device", lambda what, *t: 0)
    monkeypatch.setattr(torch, "empty", traced_empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    monkeypatch.setattr(pkg, "_need", lambda t, dtype, name: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    yield seen


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


K_CACHE = torch.zeros(pkg.KCACHE_PAGE_BYTES, dtype=torch.uint8)
KV_CACHE = torch.zeros(pkg.PAGE_SIZE * pkg.KVCACHE_TOKEN_BYTES, dtype=torch.uint8)

CALLS = {
    "rope": lambda s: pkg.rope(torch.zeros(3, 64), _i32(3), torch.zeros(32, dtype=torch.int64), stream=s),
    "prefix_attn": lambda s: pkg.prefix_attn(_bf16(1, 16, 576), KV_CACHE, _i32(1), 10, _i32(1, 1), _i32(1), _i32(1),
                                             _i32(1), 20, SM, stream=s),
    "sparse_attn": lambda s: pkg.sparse_attn(_bf16(1, 16, 576), KV_CACHE, _i32(1, 1), _i32(1), _i32(1), _i32(1, 8), SM,
                                             stream=s),
    "sparse_attn_noalloc": lambda s: pkg.sparse_attn_noalloc(_bf16(1, 16, 576), KV_CACHE, _i32(1, 1), _i32(1), _i32(1),
                                                             _i32(1, 8), SM, stream=s),
    "decode_step": lambda s: pkg.decode_step(_bf16(0, 128), _bf16(0, 576), torch.zeros(0, dtype=torch.int64), K_CACHE,
                                             KV_CACHE, _bf16(1, 8, 128), torch.zeros(1, 8), _bf16(1, 16, 576), _i32(1, 1),
                                             _i32(1), _i32(1), _i32(1), 8, 20, SM, stream=s),
    "indexer_topk": lambda s: pkg.indexer_topk(_bf16(1, 8, 128), torch.zeros(1, 8), K_CACHE, _i32(1, 1), _i32(1), _i32(1),
                                               _i32(1), 8, 20, stream=s),
    "indexer_scores": lambda s: pkg.indexer_scores(_bf16(1, 8, 128), torch.zeros(1, 8), K_CACHE, _i32(1, 1), _i32(1),
                                                   _i32(1), _i32(1), 20, stream=s),
    "topk_merge": lambda s: pkg.topk_merge(_i32(2, 1, 8), torch.zeros(2, 1, 8), 8, local_lo=_i32(1), local_hi=_i32(1),
                                           stream=s),
    "lse_combine": lambda s: pkg.lse_combine(_bf16(2, 1, 16, 512), torch.zeros(2, 1, 16), stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_belong_to_the_calls_stream(traced, name):
    s = _Stream()
    call = CALLS[name]
    traced.clear()
    call(s)
    assert traced and all(e[1] == [s] for e in traced)
    # what is returned is read on the caller's stream; a workspace (512 bytes here) is not
    assert all(e[2] == (e[0] != 512) for e in traced)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [16, 128])
def test_memory_taken_right_after_a_call_on_another_stream(h):
    """A long call on a side stream, then allocations of its workspace's size on the current one."""
    dsa = ensure_built()
    g = torch.Generator().manual_seed(h)
    n_seq, prefix, max_ctx = 8, 4000, 5000
    per = (max_ctx + 63) // 64
    pages = n_seq * per
    cache = dsa.alloc_kv_cache(pages)
    dsa.quant_kv_fp8(torch.randn(pages * 64, 576, generator=g).to(torch.bfloat16).cuda(), torch.arange(pages * 64).cuda(),
                     cache)
    table = torch.randperm(pages, generator=g).to(torch.int32).view(n_seq, per).cuda()
    q = torch.randn(n_seq, h, 576, generator=g).to(torch.bfloat16).cuda()
    lens = torch.full((n_seq,), max_ctx, dtype=torch.int32).cuda()
    args = (q, cache, table[0, :(prefix + 63) // 64].contiguous(), prefix, table, lens,
            torch.arange(n_seq, dtype=torch.int32).cuda(), lens - 1, max_ctx, SM)
    want, _ = dsa.prefix_attn(*args)
    size = dsa.prefix_attn_workspace_size(n_seq, h, n_seq, prefix, max_ctx)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)   # about a millisecond: the call's kernels start behind it
        got, _ = dsa.prefix_attn(*args, stream=side)
        taken = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(bool((t == 0xFF).all()) for t in taken)
        assert torch.equal(got, want)
    assert dsa.device_status() == 0


@pytest.mark.gpu
def test_a_captured_call_on_a_stream_forked_from_the_capture():
    dsa = ensure_built()
    g = torch.Generator().manual_seed(3)
    cache = dsa.alloc_kv_cache(40)
    dsa.quant_kv_fp8(torch.randn(40 * 64, 576, generator=g).to(torch.bfloat16).cuda(), torch.arange(40 * 64).cuda(), cache)
    table = torch.arange(40, dtype=torch.int32).view(2, 20).cuda()
    q = torch.randn(2, 64, 576, generator=g).to(torch.bfloat16).cuda()
    lens = torch.full((2,), 1200, dtype=torch.int32).cuda()
    pos = torch.arange(2, dtype=torch.int32).cuda()
    turns, _ = dsa.rope_turns(64)

    def step(stream):
        turned = dsa.rope(q, pos, turns, offset=512, stream=stream)
        return dsa.prefix_attn(turned, cache, None, 0, table, lens, pos, lens - 1, 1280, SM, stream=stream)[0]

    want = step(None)
    torch.cuda.synchronize()
    main, fork = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main, capture_error_mode="relaxed"):
        fork.wait_stream(main)
        got = step(fork)
        main.wait_stream(fork)
        same = got + 0
        del got
    for _ in range(3):
        same.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(same, want)
    assert dsa.device_status() == 0
