"""The example's cache knows its end without a GPU: a token more than it (or the table of positions) has room for is
refused, where it would be written outside the arrays or get a position of zeros."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import sequence_encoder as S  # noqa: E402


@pytest.mark.parametrize("capacity,max_len", [(3, 10), (10, 3)])
def test_a_full_cache_is_refused(monkeypatch, capacity, max_len):
    model = S.Encoder(20, dim=16, heads=2, kv_heads=1, max_len=max_len, dtype=torch.float32, device="cpu")
    monkeypatch.setattr(S.ops, "embedding", lambda ids, table, scale=1.0: scale * table[ids.long()])
    monkeypatch.setattr(S.ops, "layer_norm", lambda x, w, b: x)
    monkeypatch.setattr(S.ops, "cached_attention", lambda q, k, v, lens: q)
    monkeypatch.setattr(S.ops, "topk", lambda h, e, k: (None, torch.zeros(h.shape[0], k, dtype=torch.int32), None))
    cache, ids = model.new_cache(2, capacity), torch.tensor([1, 2], dtype=torch.int32)
    for _ in range(3):
        hidden, _ = model.serve(ids, cache)
        assert hidden.shape == (2, 16)
    with pytest.raises(ValueError, match="full"):
        model.serve(ids, cache)
