"""Two backwards through one forward of ``cut_bce``."""
import pytest
import torch

from vocabulary_label_bce_amd import workloads as W
from vocabulary_label_bce_amd.ops import cut_bce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 256), ("f32", 64)])
def test_a_kept_graph_gives_the_same_gradients_again(dtype, D):
    p = W.custom_problem(R=200, V=3000, D=D, dtype=dtype, seed=7, h_std=0.2, e_std=0.2, pos_per_row=(0, 5),
                         mask_frac=0.2)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in p.items()}
    H, E = d["H"].requires_grad_(), d["E"].requires_grad_()
    loss = cut_bce(H, E, d["row_offsets"], d["item_ids"], d["row_mask"])
    first = torch.autograd.grad(loss, (H, E), retain_graph=True)
    noise = torch.full_like(E, 7.0)  # what an unwritten result would find in its place
    del noise
    for again in (torch.autograd.grad(loss, (H, E), retain_graph=True), torch.autograd.grad(loss, (H, E))):
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert bool(first[1].abs().max() > 0)
