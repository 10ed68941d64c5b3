"""Handles that the binding keeps beside their owner's, without a GPU."""

import types

import pytest
import torch


@pytest.fixture()
def sffn(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    from activation_sparse_ffn_gb300 import sffn
    monkeypatch.setattr(sffn, "_stream", lambda stream: None)
    return sffn


def test_reordering_refuses_caches_that_are_closed(sffn, monkeypatch):
    calls = []
    monkeypatch.setattr(sffn, "_lib", types.SimpleNamespace(sffn_kv_reorder=lambda *a: calls.append(a) or 0))
    caches = [types.SimpleNamespace(handle=4096), types.SimpleNamespace(handle=8192)]
    held = sffn.KvCaches(caches)
    batch = sffn.KvBatch(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    parents = torch.zeros(4, dtype=torch.int32)
    sffn.sffn_kv_reorder(held, batch, parents, 2)
    assert len(calls) == 1 and list(calls[0][0]) == [4096, 8192]
    caches[1].handle = None                                     # as KvCache.close leaves it
    with pytest.raises(ValueError, match="closed"):
        sffn.sffn_kv_reorder(held, batch, parents, 2)
    assert len(calls) == 1
