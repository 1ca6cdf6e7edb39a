"""Host threads that call the indexer and the merge with other sizes at the same time: what one call asks of a kernel must
not take away what another's launch needs."""

import threading

import pytest
import torch

from dsa_sparse_attention_topk_gb300 import workloads as W
from dsa_testlib import DeviceWorkload, ensure_built


@pytest.fixture(scope="module")
def dsa():
    return ensure_built()


def _merges(dsa):
    jobs = []
    for parts, k_in in ((8, 2048), (2, 500)):
        g = torch.Generator().manual_seed(k_in)
        idx = torch.randperm(parts * k_in, generator=g).to(torch.int32).view(parts, 1, k_in).cuda()
        scores = torch.randn(parts, 1, k_in, generator=g).cuda()
        jobs.append(lambda s, idx=idx, scores=scores: dsa.topk_merge(idx, scores, 256, stream=s)[:2])
    return jobs


def _selections(dsa):
    jobs = []
    for ctx in (30000, 2000):
        d = DeviceWorkload(W.custom([ctx] * 4, h_i=64, topk=256, seed=ctx), with_kv=False)

        def call(s, d=d, wl=d.wl):
            with torch.cuda.stream(s):  # (None: the current one)
                scores = torch.empty(wl.n_q, wl.topk, device="cuda")
            return dsa.indexer_topk(d.q_idx, d.w, d.k_cache, d.page_table, d.seq_lens, d.q_seq, d.q_pos, wl.topk, wl.max_ctx,
                                    out_scores=scores, stream=s)

        jobs.append(call)
    return jobs


@pytest.mark.gpu
@pytest.mark.parametrize("make", [_merges, _selections])
def test_two_sizes_of_one_kernel(dsa, make):
    jobs, errors = make(dsa), []
    want = [call(None) for call in jobs]
    torch.cuda.synchronize()

    def work(call, want):
        s = torch.cuda.Stream()
        try:
            for _ in range(500):
                got = call(s)
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:  # noqa: BLE001  (a thread's failure has to reach the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(jobs[i % 2], want[i % 2])) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    assert dsa.device_status() == 0
