"""evict_select refuses new lengths that lie partly in the old ones: another sequence's are still to be read there."""

import ctypes

import pytest
import torch

from dsa_testlib import ensure_built


@pytest.mark.parametrize("lens,new,code", [(8, 8, -1), (8, 12, -1), (12, 8, -1), (8, 16, -1), (16, 8, -1)])
def test_the_call_refuses(lens, new, code):
    dsa, p = ensure_built(), lambda v: ctypes.c_void_p((1 << 20) + v)  # noqa: E731
    rc = dsa.lib().dsa_evict_select(p(1 << 21), 100, p(lens), 3, 100, 10, 2, 3, p(1 << 22), p(new), p(1 << 23), None)
    assert rc == code and b"share memory" in dsa.lib().dsa_last_error()


def test_lengths_next_to_one_another_get_past_it():
    """(To the next check: there is no device here, or the pointers are none of its.)"""
    dsa, p = ensure_built(), lambda v: ctypes.c_void_p((1 << 20) + v)  # noqa: E731
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are for machines without a device")
    for lens, new in ((8, 20), (20, 8)):
        rc = dsa.lib().dsa_evict_select(p(1 << 21), 100, p(lens), 3, 100, 10, 2, 3, p(1 << 22), p(new), p(1 << 23), None)
        assert rc != 0 and b"share memory" not in dsa.lib().dsa_last_error()


@pytest.mark.gpu
def test_the_binding_refuses():
    dsa = ensure_built()
    both = torch.full((4,), 20, dtype=torch.int32).cuda()
    mass = torch.zeros(3, 30, dtype=torch.int64).cuda()
    for a, b in ((both[:3], both[:3]), (both[:3], both[1:]), (both[1:], both[:3])):
        with pytest.raises(ValueError, match="share memory"):
            dsa.evict_select(mass, a, 10, new_lens=b)
    six = torch.full((6,), 20, dtype=torch.int32).cuda()
    assert dsa.evict_select(mass, six[:3], 10, new_lens=six[3:])[1].tolist() == [10, 10, 10]
