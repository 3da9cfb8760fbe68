"""What the optimizer's front end refuses, without a GPU (the library's calls are replaced; none is reached)."""
import pytest
import torch

from vocabulary_label_bce_amd import binding as B
from vocabulary_label_bce_amd import ops
from vocabulary_label_bce_amd import optimizer as O


@pytest.fixture(autouse=True)
def _no_launches(monkeypatch):
    monkeypatch.setattr(O, "_here", lambda what, *lists: -1)
    monkeypatch.setattr(B, "raw_stream", lambda device: 0)
    monkeypatch.setattr(B, "adamw_step", lambda *a: None)
    monkeypatch.setattr(B, "grad_norm", lambda *a: None)


def _step(n=300, **over):
    a = dict(params=[torch.zeros(n)], grads=[torch.zeros(n)], exp_avgs=[torch.zeros(n)], exp_avg_sqs=[torch.zeros(n)],
             step=torch.zeros(1, dtype=torch.int32), lr=1e-3)
    a.update(over)
    ops.adamw_step(**a)


Z = torch.zeros
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("over,match", [
    (dict(grads=[]), "one length"), (dict(masters=[]), "one length"), (dict(grads=[Z(299)]), "size"),
    (dict(params=[Z(300, dtype=torch.float16)]), "params must be"), (dict(grads=[Z(300, dtype=torch.int32)]), "grads must be"),
    (dict(exp_avgs=[Z(300, dtype=torch.bfloat16)]), "exp_avgs must be"), (dict(params=[Z(600)[::2]]), "contiguous"),
    (dict(exp_avg_scales=[Z(2)]), "scales each"), (dict(exp_avg_scales=[Z(2)], exp_avg_sq_scales=[Z(2)]), "exp_avgs must be"),
    (dict(exp_avg_scales=[Z(1)], exp_avg_sq_scales=[Z(2)], exp_avgs=[Z(300).to(F8)], exp_avg_sqs=[Z(300).to(F8)]),
     "each 256"),
    (dict(betas=(1.0, 0.9)), "betas"), (dict(betas=(0.9, float("nan"))), "betas"), (dict(eps=-1.0), "eps"),
    (dict(lr=float("inf")), "lr"), (dict(lr=Z(2)), "lr"), (dict(lr=Z(1, dtype=torch.float64)), "lr"),
    (dict(step=Z(1)), "step"), (dict(step=Z(2, dtype=torch.int32)), "step"), (dict(norm=Z(1)), "together"),
    (dict(max_norm=1.0), "together"), (dict(norm=Z(1), max_norm=-1.0), "together"), (dict(weight_decay=[0.1, 0.2]), "weight_decay"),
    (dict(weight_decay=float("nan")), "weight_decay"), (dict(masters=[Z(299)]), "master"), (dict(masters=[Z(300, dtype=torch.bfloat16)]), "masters must"),
])
def test_refusals(over, match):
    with pytest.raises(ValueError, match=match):
        _step(**over)


def test_a_tensor_listed_twice_is_refused():
    x = Z(300)
    with pytest.raises(ValueError, match="twice"):
        _step(params=[x, x], grads=[Z(300)] * 2, exp_avgs=[Z(300), Z(300)], exp_avg_sqs=[Z(300), Z(300)])
    with pytest.raises(ValueError, match="twice"):
        _step(exp_avgs=[x], exp_avg_sqs=[x])


def test_a_step_is_seen_by_autograd():
    """A parameter that a graph has kept may not change below it."""
    p = torch.ones(300, requires_grad=True)
    y = (p * p).sum()
    _step(params=[p])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_class_refusals():
    with pytest.raises(ValueError, match="state_bits"):
        ops.AdamW([Z(3)], state_bits=4)
    with pytest.raises(ValueError, match="a parameter"):
        ops.AdamW([])
    with pytest.raises(ValueError, match="each parameter"):
        ops.AdamW([Z(3)]).step([])
    with pytest.raises(ValueError, match="gradients must be"):
        ops.grad_norm([Z(3, dtype=torch.float64)])
