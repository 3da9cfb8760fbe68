"""What autograd is told about the sequence encoder's operators. Only the launches are replaced here (they leave their
outputs as they are), so this runs without a GPU: it is about which calls are refused, not about values."""
import pytest
import torch
from torch.autograd import forward_ad

from vocabulary_label_bce_amd import binding as B
from vocabulary_label_bce_amd import encoder as E
from vocabulary_label_bce_amd import ops


@pytest.fixture(autouse=True)
def _no_launches(monkeypatch):
    monkeypatch.setattr(E, "_on_gpu", lambda what, *tensors: 0)
    monkeypatch.setattr(B, "raw_stream", lambda device: 0)
    for name in ("embedding_forward", "embedding_backward", "layer_norm_forward", "layer_norm_backward",
                 "attention_forward", "attention_backward"):
        monkeypatch.setattr(B, name, lambda *a: None)


IDS = torch.tensor([1, 0, 3], dtype=torch.int32)
CU = torch.tensor([0, 4], dtype=torch.int32)

# name: (the inputs that a derivative may be taken of, the call)
CALLS = {
    "embedding": ([(5, 8)], lambda table: ops.embedding(IDS, table, 2.0)),
    "layer_norm": ([(4, 8), (8,), (8,)], ops.layer_norm),
    "packed_attention": ([(4, 2, 8), (4, 1, 8), (4, 1, 8)], lambda q, k, v: ops.packed_attention(q, k, v, CU)),
}
EACH = [(name, i) for name, (shapes, _) in CALLS.items() for i in range(len(shapes))]


@pytest.mark.parametrize("name,i", EACH)
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(name, i, grad):
    """There is no forward-mode derivative: a dual input raises, instead of giving an output without a tangent."""
    shapes, call = CALLS[name]
    x = [torch.ones(s) for s in shapes]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        call(*x)  # without a tangent there is nothing to refuse
        x[i] = forward_ad.make_dual(x[i], torch.ones_like(x[i]))
        with pytest.raises(NotImplementedError, match="jvp"):
            call(*x)


@pytest.mark.parametrize("i", [0, 1, 2])
def test_forward_mode_is_refused_where_there_is_no_gradient_at_all(i):
    x = [torch.ones(2, 2, 8), torch.ones(2, 6, 1, 8), torch.ones(2, 6, 1, 8)]
    lens = torch.tensor([6, 3], dtype=torch.int32)
    with forward_ad.dual_level():
        ops.cached_attention(*x, lens)
        x[i] = forward_ad.make_dual(x[i], torch.ones_like(x[i]))
        with pytest.raises(ValueError, match="no gradient"):
            ops.cached_attention(*x, lens)


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("name,i", EACH)
def test_second_derivatives_are_refused(name, i, plain):
    """The gradients are kernels' outputs: differentiating them raises, also in a sum with a term that has a graph (a
    gradient penalty beside a loss), instead of leaving their part out."""
    shapes, call = CALLS[name]
    x = [torch.ones(s) for s in shapes]
    x[i].requires_grad_()
    y = call(*x)
    # a cotangent without a graph, and one with
    (grad,) = torch.autograd.grad(y.sum() if plain else y.square().sum(), x[i], create_graph=True)
    loss = grad.square().sum() + x[i].square().sum()
    with pytest.raises(RuntimeError, match="first derivatives only"):
        loss.backward()


@pytest.mark.parametrize("bias", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [torch.float32, torch.bfloat16])
def test_a_bias_alone_gets_its_gradient_in_its_own_type(monkeypatch, rows, bias):
    """The library writes dbias in the bias's type at once: no rounding to the rows' type in between."""
    asked = []
    monkeypatch.setattr(B, "layer_norm_backward", lambda dy, x, w, mean, rstd, dx, dw, db, *a: asked.append((dw, db)))
    b = torch.zeros(8, dtype=bias, requires_grad=True)
    ops.layer_norm(torch.ones(4, 8, dtype=rows), None, b).sum().backward()
    assert [(dw, db.dtype) for dw, db in asked] == [(None, bias)] and b.grad.dtype == bias


@pytest.mark.parametrize("dtype", [torch.float32, torch.bool, torch.int16, torch.uint8])
def test_offsets_and_lengths_of_other_types_are_refused(dtype):
    """Like ids, they are int32 or int64: nothing is cut to a whole number in passing."""
    q = torch.ones(4, 2, 8)
    for kw in (dict(cu_q=CU.to(dtype)), dict(cu_q=CU, cu_k=CU.to(dtype)),
               dict(cu_q=CU, k_lens=torch.ones(1, dtype=dtype))):
        with pytest.raises(ValueError, match="int32 or int64"):
            ops.packed_attention(q, q, q, **kw)
    with pytest.raises(ValueError, match="int32 or int64"):
        ops.cached_attention(q[:1], q[None], q[None], torch.ones(1, dtype=dtype))
    ops.packed_attention(q, q, q, CU.long(), k_lens=torch.tensor([3]))


def test_adding_to_a_table_gradient_is_seen_by_autograd():
    """embedding_backward writes into dtable: where autograd has kept it for a backward, that one raises."""
    dtable, w = torch.ones(5, 8), torch.ones(5, 8, requires_grad=True)
    y = (w * dtable).sum()
    assert ops.embedding_backward(torch.ones(3, 8), IDS, 5, dtable=dtable) is dtable
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():  # (without versions)
        ops.embedding_backward(torch.ones(3, 8), IDS, 5, dtable=torch.ones(5, 8))
