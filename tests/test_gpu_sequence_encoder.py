"""The example's model: training lowers the loss, the item table's gradient is the lookup's and the loss's together,
and serving one token at a time gives the packed encoder's hidden states."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import sequence_encoder as S  # noqa: E402

from vocabulary_label_bce_amd import ops  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kv_heads", [(torch.bfloat16, 2), (torch.float32, 1)])
def test_training_lowers_the_loss(dtype, kv_heads):
    model = S.Encoder(3000, dim=128, heads=2, kv_heads=kv_heads, dtype=dtype)
    batch, _ = S.histories(16, 3000, 1, 200, seed=2)
    first = model.train_step(*batch).item()
    for _ in range(8):
        last = model.train_step(*batch).item()
    assert last < 0.9 * first


def test_table_gradient_is_both_parts():
    """One step's change of the item table against autograd through the differentiable calls (float32: the two
    accumulate in different orders)."""
    model = S.Encoder(500, dim=64, heads=2, kv_heads=2, dtype=torch.float32)
    batch, _ = S.histories(5, 500, 1, 40, seed=3)
    ids, places, cu, ro, pos = batch
    table = model.items.clone().requires_grad_()
    H = model.hidden(ops.embedding(ids, table, model.scale), places, cu)
    mask = torch.ones(H.shape[0], dtype=torch.uint8, device="cuda")
    ops.cut_bce(H, table, ro, pos, mask).backward()
    for t in model.p.values():
        t.grad = None
    before = model.items.clone()
    model.train_step(*batch, lr=1.0 / 500)
    got = before - model.items
    assert float((got - table.grad).norm()) <= 1e-4 * float(table.grad.norm())


@pytest.mark.parametrize("kv_heads", [2, 1])
def test_serving_matches_the_packed_encoder(kv_heads):
    model = S.Encoder(400, dim=64, heads=2, kv_heads=kv_heads, max_len=64, dtype=torch.float32, seed=4)
    (ids, places, cu, _, _), lens = S.histories(6, 400, 30, 30, seed=5)
    with torch.no_grad():
        want = model.hidden(ops.embedding(ids, model.items, model.scale), places, cu).view(6, 30, -1)
        cache = model.new_cache(6, 64)
        for t in range(30):
            got, best = model.serve(ids.view(6, 30)[:, t].contiguous(), cache)
            assert float((got - want[:, t]).abs().max()) <= 1e-4 * float(want.abs().max())
    assert best.shape == (6, 8)
