"""What rope and prefix_attn refuse on the host."""

import ctypes
import math

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import dsa_sparse_attention_topk_gb300 as pkg
from dsa_testlib import ensure_built
from test_gpu_rope import _append_call, _rope_call

SM = 1.0 / math.sqrt(192.0)


def _rope(x, **kw):
    return pkg.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.int64), **kw)


def _prefix(q, **kw):
    z = torch.zeros(1, dtype=torch.int32)
    return pkg.prefix_attn(q, torch.zeros(608 * 64, dtype=torch.uint8), z, 10, z[None], z, z, z, 20, SM, **kw)


CALLS = {
    "rope": (_rope, (2, 64), torch.float32, dict(out=torch.zeros(2, 64))),
    "prefix_attn": (_prefix, (1, 16, 576), torch.bfloat16, dict(out_lse=torch.zeros(1, 16))),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_gradient_is_not_lost_in_silence(name):
    call, shape, dtype, outs = CALLS[name]
    x = torch.zeros(shape, dtype=dtype, requires_grad=True)
    for bad in (x, x * 1):
        with pytest.raises(ValueError, match="gradient"):
            call(bad)
    (key, out), = outs.items()
    with pytest.raises(ValueError, match="gradient"):
        call(x.detach(), **{key: out.clone().requires_grad_()})
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="gradient"):
            call(forward_ad.make_dual(x.detach(), torch.ones_like(x)))
        with pytest.raises(ValueError, match="CUDA"):     # the next check: these are CPU tensors
            call(x.detach())
    for quiet in (torch.no_grad, torch.inference_mode):
        with quiet(), pytest.raises(ValueError, match="CUDA"):
            call(x)


@pytest.mark.parametrize("kw", [
    dict(xt=1 << 40, n=3), dict(xh=1 << 40, ot=1 << 30), dict(n=1 << 24, h=1, xt=1 << 39, ot=64),
    dict(n=1 << 24, h=1, xt=64, ot=1 << 39),
    dict(n=2, h=1 << 24, xh=64, xt=1 << 30, oh=1 << 40, ot=64),      # (h - 1) oh wraps in 64 bits
])
def test_rope_refuses_axes_whose_offsets_overflow(kw):
    assert _rope_call(ensure_built().lib(), **kw) == -1


@pytest.mark.parametrize("kw", [dict(n=3, ks=1 << 40), dict(n=1 << 24, kvs=1 << 39), dict(n=1 << 30, ks=1 << 12)])
def test_rope_quant_kv_refuses_rows_whose_offsets_overflow(kw):
    assert _append_call(ensure_built().lib(), **kw) == -1


@pytest.mark.parametrize("which", ["pages", "table", "lens", "q_seq", "q_pos", "out_lse"])
def test_prefix_attn_refuses_misaligned_tables(which):
    names = ["q", "cache", "pages", "table", "lens", "q_seq", "q_pos", "out", "out_lse", "ws"]
    p = {n: ctypes.c_void_p((i + 1) * 65536 + (2 if n == which else 0)) for i, n in enumerate(names)}
    assert ensure_built().lib().dsa_prefix_attn(
        p["q"], 2, 16, p["cache"], 8, p["pages"], 100, p["table"], 4, p["lens"], 2, p["q_seq"], p["q_pos"], 200,
        ctypes.c_float(0.07), p["out"], p["out_lse"], p["ws"], 1 << 40, None) == -1


class _Library:
    """Records the workspace size that an entry point is given."""
    given = []

    def __getattr__(self, name):
        return (lambda *a: 512) if name.endswith("_workspace_size") else (lambda *a: self.given.append(a[-2]) or 0)


def test_a_workspace_is_measured_in_bytes_of_its_own(monkeypatch):
    monkeypatch.setattr(pkg, "lib", _Library)
    monkeypatch.setattr(pkg, "_same_device", lambda what, *t: 0)
    monkeypatch.setattr(pkg, "_call_on", lambda dev, stream, fn, *a: fn(*a, None))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    q = torch.zeros(1, 16, 576, dtype=torch.bfloat16)
    # 512 elements that are one byte
    with pytest.raises(ValueError, match="workspace"):
        _prefix(q, workspace=torch.zeros(1, dtype=torch.uint8).expand(512))
    with pytest.raises(ValueError, match="workspace"):
        _prefix(q, workspace=torch.zeros(2048, dtype=torch.uint8)[::2])
    _prefix(q, workspace=torch.zeros(512, dtype=torch.uint8))
    _prefix(q, workspace=torch.zeros(128))
    assert _Library.given == [512, 512]


class _Rotary(torch.autograd.Function):
    """The two halves that the refusal points to."""

    @staticmethod
    def forward(ctx, x, pos, turns):
        ctx.save_for_backward(pos, turns)
        return pkg.rope(x, pos, turns)

    @staticmethod
    def backward(ctx, grad):
        return pkg.rope(grad, *ctx.saved_tensors, transpose=True), None, None


@pytest.mark.gpu
def test_rope_in_the_halves_of_an_autograd_function():
    ensure_built()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 3, 64, generator=g).cuda().requires_grad_()
    w = torch.randn(5, 3, 64, generator=g).cuda()
    pos = torch.arange(5, dtype=torch.int32).cuda() * 1000
    turns, _ = pkg.rope_turns(64)
    (_Rotary.apply(x, pos, turns) * w).sum().backward()
    assert torch.equal(x.grad, pkg.rope(w, pos, turns, transpose=True))
    # a rotation keeps the product of two tensors turned alike: each of 64 terms off by 4e-7 of some units
    with torch.no_grad():
        same = (pkg.rope(x, pos, turns) * pkg.rope(w, pos, turns)).sum(-1) - (x * w).sum(-1)
    assert float(same.abs().max()) < 64 * 4e-7 * 16
