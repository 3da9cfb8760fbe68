"""What the softmax cross entropy's front end refuses, and what autograd is told about it, without a GPU (the launches are
replaced; they leave their outputs as they are)."""
import pytest
import torch
from torch.autograd import forward_ad

from vocabulary_label_bce_amd import binding as B
from vocabulary_label_bce_amd import cross_entropy as C
from vocabulary_label_bce_amd import ops


@pytest.fixture
def no_launches(monkeypatch):
    monkeypatch.setattr(C, "_on_gpu", lambda what, *tensors: 0)
    monkeypatch.setattr(B, "raw_stream", lambda device: 0)
    for name in ("cross_entropy_forward", "cross_entropy_backward"):
        monkeypatch.setattr(B, name, lambda *a: None)


H, E, T = torch.ones(5, 16), torch.ones(9, 16), torch.zeros(5, dtype=torch.int32)


@pytest.mark.parametrize("over,match", [
    (dict(H=H.half()), "float32 or both"), (dict(E=E.bfloat16()), "float32 or both"), (dict(H=H[0]), "must be"),
    (dict(E=torch.ones(9, 8)), "must be"), (dict(H=torch.ones(5, 12), E=torch.ones(9, 12)), "multiple of 8"),
    (dict(H=torch.ones(5, 0), E=torch.ones(9, 0)), "multiple of 8"), (dict(E=E[:0]), "an item"),
    (dict(H=torch.ones(1, 16).expand((1 << 20) + 1, 16), targets=torch.zeros(1, dtype=torch.int32).expand((1 << 20) + 1)),
     "2\\*\\*20 rows"),
    (dict(targets=T.float()), "targets"), (dict(targets=T[:4]), "targets"), (dict(targets=T[:, None]), "targets"),
    (dict(row_weight=torch.ones(4)), "row_weight"), (dict(row_weight=torch.ones(5, dtype=torch.float64)), "row_weight"),
    (dict(row_weight=torch.ones(5, requires_grad=True)), "no gradient"), (dict(scale=float("inf")), "scale"),
    (dict(scale=float("nan")), "scale"),
])
def test_refusals(no_launches, over, match):
    with pytest.raises(ValueError, match=match):
        ops.cut_cross_entropy(**dict(dict(H=H, E=E, targets=T), **over))


def test_backward_refusals(no_launches):
    saved = ops.cross_entropy_forward(H, E, T)[2]
    g = torch.ones(1)
    assert [x.shape for x in ops.cross_entropy_backward(g, H, E, saved)] == [H.shape, E.shape]
    assert ops.cross_entropy_backward(g, H, E, saved, want_dH=False)[0] is None
    assert ops.cross_entropy_backward(g, H, E, saved, False, False) == (None, None)
    for args in ((g, H[:4], E, saved), (g, H, E[:8], saved), (g, H.bfloat16(), E.bfloat16(), saved)):
        with pytest.raises(ValueError, match="forward's"):
            ops.cross_entropy_backward(*args)
    with pytest.raises(ValueError, match="one element"):
        ops.cross_entropy_backward(torch.ones(2), H, E, saved)


def test_tensors_of_the_host_are_refused():
    with pytest.raises(ValueError, match="GPU only"):
        ops.cut_cross_entropy(H, E, T)


@pytest.mark.parametrize("i", [0, 1])
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(no_launches, i, grad):
    x = [H.clone(), E.clone()]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        ops.cut_cross_entropy(*x, T)
        x[i] = forward_ad.make_dual(x[i], torch.ones_like(x[i]))
        with pytest.raises(NotImplementedError, match="jvp"):
            ops.cut_cross_entropy(*x, T)


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("i", [0, 1])
def test_second_derivatives_are_refused(no_launches, i, plain):
    x = [H.clone(), E.clone()]
    x[i].requires_grad_()
    y = ops.cut_cross_entropy(*x, T)
    (grad,) = torch.autograd.grad(y if plain else y.square(), x[i], create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        (grad.square().sum() + x[i].square().sum()).backward()


def test_only_what_is_asked_for_is_formed(no_launches, monkeypatch):
    """An input that needs no gradient costs none."""
    asked = []
    monkeypatch.setattr(B, "cross_entropy_backward", lambda R, E_, s, g, saved, dH, dE, *a: asked.append((dH is None, dE is None)))
    ops.cut_cross_entropy(H.clone().requires_grad_(), E, T).backward()
    ops.cut_cross_entropy(H, E.clone().requires_grad_(), T).backward()
    assert asked == [(False, True), (True, False)]
