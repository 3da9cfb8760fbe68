"""What autograd is told about ``cut_bce``. The argument checks that look for a GPU and the launches are replaced, so this
runs without one: it is about which calls are made and refused, not about values."""
import pytest
import torch

from vocabulary_label_bce_amd import binding as B
from vocabulary_label_bce_amd import ops


@pytest.fixture
def launches(monkeypatch):
    """The launches that were asked for: ("forward", workspace) and ("backward", workspace, reuse)."""
    made = []
    monkeypatch.setattr(ops, "_prep", lambda *a: a)
    monkeypatch.setattr(B, "problem_of", lambda *a: None)
    monkeypatch.setattr(B, "alloc_workspace", lambda p, device: torch.empty(1))
    monkeypatch.setattr(B, "forward", lambda *a, **kw: made.append(("forward", a[9])))
    monkeypatch.setattr(B, "backward", lambda *a, **kw: made.append(("backward", a[10], kw.get("reuse", False))))
    return made


def _loss():
    H, E = torch.ones(3, 4, requires_grad=True), torch.ones(5, 4, requires_grad=True)
    offsets, ids, mask = torch.arange(4), torch.arange(3), torch.ones(3)
    return H, E, ops.cut_bce(H, E, offsets, ids, mask)


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("i", [0, 1])
def test_second_derivatives_are_refused(launches, i, plain):
    H, E, loss = _loss()
    x = (H, E)[i]
    (grad,) = torch.autograd.grad(loss if plain else loss.square(), x, create_graph=True)
    total = grad.square().sum() + x.square().sum()
    with pytest.raises(RuntimeError, match="first derivatives only"):
        total.backward()


def test_a_second_backward_is_computed_too(launches):
    """The forward's workspace serves the first backward through a graph that is kept; the next one prepares its own
    (cutbce_backward_reuse has to follow the forward)."""
    H, E, loss = _loss()
    for first in (True, False):
        torch.autograd.grad(loss, (H, E), retain_graph=True)
        kind, ws, reuse = launches[-1]
        assert kind == "backward" and reuse == first and (ws is launches[0][1]) == first
    assert [k for k, *_ in launches] == ["forward", "backward", "backward"]
