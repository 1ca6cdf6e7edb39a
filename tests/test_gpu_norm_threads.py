"""Host threads that call norm_rope and its gradient with other sizes at the same time: what one call asks of a kernel
must not take away what another's launch needs."""

import threading

import pytest
import torch

from dsa_testlib import ensure_built


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


@pytest.mark.gpu
@pytest.mark.parametrize("grad", [False, True])
def test_two_sizes_of_one_kernel(dsa, grad):
    """Sizes that the same kernel serves with 50 to 75 KB of shared memory each."""
    jobs, errors = [], []
    for d, rot in ((1024, 64), (896, 64)) if grad else ((1023, 1022), (701, 700)):
        x = torch.randn(9, 1, d, device="cuda", dtype=torch.bfloat16)
        turns = (torch.arange(1, rot // 2 + 1, dtype=torch.int64) << 50).cuda()
        pos, w = torch.arange(9, dtype=torch.int32).cuda(), torch.ones(d).cuda()
        call = (lambda s, x=x, p=pos, t=turns, w=w: dsa.norm_rope_grad(x, x, p, t, w, w, stream=s)) if grad else (
            lambda s, x=x, p=pos, t=turns, w=w: (dsa.norm_rope(x, p, t, w, w, layout="half", stream=s),))
        jobs.append((call, call(None)))
    torch.cuda.synchronize()

    def work(call, want):
        s = torch.cuda.Stream()
        try:
            for _ in range(1500):
                got = call(s)
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:  # noqa: BLE001  (a thread's failure has to reach the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=jobs[i % 2]) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
