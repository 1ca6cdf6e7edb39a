"""What the norming, weighing and evicting calls allocate when they are given a stream: on that stream, and what is
returned recorded on the caller's."""

import pytest
import torch

import dsa_sparse_attention_topk_gb300 as pkg
from test_call_streams import KV_CACHE, SM, _Stream, _bf16, _i32, traced  # noqa: F401

ROWS = dict(weight=torch.ones(64), bias=torch.ones(64))
CALLS = {
    "norm_rope": lambda s: pkg.norm_rope(torch.zeros(3, 64), _i32(3), torch.zeros(32, dtype=torch.int64), **ROWS, stream=s),
    "norm_rope_grad": lambda s: pkg.norm_rope_grad(torch.zeros(3, 64), torch.zeros(3, 64), _i32(3),
                                                   torch.zeros(32, dtype=torch.int64), **ROWS, stream=s),
    "sparse_attn_mass": lambda s: pkg.sparse_attn_mass(_bf16(1, 16, 576), KV_CACHE, _i32(1, 1), _i32(1), _i32(1), _i32(1, 8),
                                                       torch.zeros(1, 16), SM, stream=s),
    "evict_select": lambda s: pkg.evict_select(torch.zeros(2, 100, dtype=torch.int64), _i32(2), 10, stream=s),
    "evict_compact": lambda s: pkg.evict_compact(_i32(1, 8), _i32(1, 1), kv_cache=KV_CACHE, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_belong_to_the_calls_stream(traced, name):  # noqa: F811
    s = _Stream()
    call = CALLS[name]
    traced.clear()
    call(s)
    assert traced and all(e[1] == [s] for e in traced)
    assert all(e[2] == (e[0] != 512) for e in traced)


def test_new_mass_is_zeroed_on_the_calls_stream(traced, monkeypatch):  # noqa: F811
    s, where = _Stream(), []
    zero = torch.Tensor.zero_

    def zeroed(t):
        where.append(list(traced[-1][1]))
        return zero(t)

    traced.clear()
    monkeypatch.setattr(torch.Tensor, "zero_", zeroed)
    mass = pkg.attn_mass(_bf16(1, 16, 576), KV_CACHE, _i32(1, 1), _i32(1), _i32(1), _i32(1), torch.zeros(1, 16), 20, SM,
                         stream=s)
    assert where == [[s]] and all(e[1] == [s] for e in traced) and mass.shape == (1, 20)
