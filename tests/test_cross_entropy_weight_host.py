"""The softmax cross entropy gives its rows' weights no derivative, in either mode: it says so instead of leaving it out."""
import pytest
import torch
from torch.autograd import forward_ad

from vocabulary_label_bce_amd import binding as B
from vocabulary_label_bce_amd import cross_entropy as C
from vocabulary_label_bce_amd import ops


@pytest.fixture(autouse=True)
def _no_launches(monkeypatch):
    monkeypatch.setattr(C, "_on_gpu", lambda what, *tensors: 0)
    monkeypatch.setattr(B, "raw_stream", lambda device: 0)
    for name in ("cross_entropy_forward", "cross_entropy_backward"):
        monkeypatch.setattr(B, name, lambda *a: None)


H, E, T = torch.ones(5, 16), torch.ones(9, 16), torch.zeros(5, dtype=torch.int32)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("train", [True, False])
def test_a_tangent_of_the_weights_is_refused(grad, train):
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        w = forward_ad.make_dual(torch.ones(5), torch.ones(5))
        with pytest.raises(ValueError, match="no gradient"):
            ops.cut_cross_entropy(H.clone().requires_grad_(train), E, T, w)
        ops.cut_cross_entropy(H, E, T, torch.ones(5))


def test_weights_that_need_a_gradient_are_taken_where_none_is_formed():
    w = torch.ones(5, requires_grad=True)
    with torch.no_grad():
        ops.cut_cross_entropy(H, E, T, w)
    with pytest.raises(ValueError, match="no gradient"):
        ops.cut_cross_entropy(H, E, T, w)
