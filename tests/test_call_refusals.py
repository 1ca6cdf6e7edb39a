"""What rope and prefix_attn refuse on the host."""

import math

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import dsa_sparse_attention_topk_gb300 as pkg

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
