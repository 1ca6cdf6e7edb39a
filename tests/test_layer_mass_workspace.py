"""The workspace of attend_prefix's accumulated weights is one that no other call could be using."""

import pytest
import torch

import dsa_sparse_attention_topk_gb300.layer as layer
from dsa_testlib import ensure_built

H_S = 4


@pytest.fixture
def calls(monkeypatch):
    ensure_built()
    seen = []
    for name in ("attn_mass", "sparse_attn_mass"):
        monkeypatch.setattr(layer, name, lambda *a, _n=name, workspace=None, **k: seen.append((_n, workspace)))
    for name in ("prefix_attn", "sparse_attn", "indexer_topk"):
        monkeypatch.setattr(layer, name, lambda *a, **k: None)
    return seen


def _layer():
    return layer.DsaDecodeLayer(1, 2, H_S, 8, 1.0, device="cpu")


def _decode(lay, n_q, n_seq):
    z = torch.zeros(n_q, dtype=torch.int32)
    lay.decode(torch.zeros(n_q, 2, 128), torch.zeros(n_q, 2), torch.zeros(n_q, H_S, 576), torch.zeros(n_seq, 1, dtype=torch.int32),
               torch.zeros(n_seq, dtype=torch.int32), z, z, 64, mass=torch.zeros(n_seq, 64, dtype=torch.int64))


def test_attend_prefix_shares_no_workspace(calls):
    lay = _layer()
    _decode(lay, 3, 3)
    kept = calls.pop()[1]
    for _ in range(2):
        z = torch.zeros(3, dtype=torch.int32)
        lay.attend_prefix(torch.zeros(3, H_S, 576), None, 0, torch.zeros(3, 1, dtype=torch.int32), z, z, z, 64,
                          mass=torch.zeros(3, 64, dtype=torch.int64))
    used = [w for name, w in calls if name == "attn_mass"]
    assert kept is not None and len(used) == 2 and all(w is None for w in used)
