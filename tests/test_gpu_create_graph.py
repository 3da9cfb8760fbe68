"""First derivatives under create_graph on the GPU: the same values, and a graph that raises."""
import pytest
import torch

from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(1)

    def leaf(*s):
        return torch.randn(*s, generator=gen, device="cuda").requires_grad_()

    ids = torch.tensor([3, 0, 3, -1, 4], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    offsets = torch.arange(6, dtype=torch.int32, device="cuda")
    mask = torch.ones(5, dtype=torch.uint8, device="cuda")
    yield [leaf(6, 64)], lambda t: ops.embedding(ids, t, 2.0).square().sum()
    yield [leaf(5, 64), leaf(64), leaf(64)], lambda x, w, b: ops.layer_norm(x, w, b).square().sum()
    yield [leaf(5, 2, 32), leaf(5, 1, 32), leaf(5, 1, 32)], lambda q, k, v: ops.packed_attention(q, k, v, cu).square().sum()
    yield [leaf(5, 64), leaf(6, 64)], lambda H, E: ops.cut_bce(H, E, offsets, ids.clamp(min=0), mask)


@pytest.mark.parametrize("i", range(4))
def test_create_graph(i):
    x, f = list(_calls())[i]
    want = torch.autograd.grad(f(*x), x)
    got = torch.autograd.grad(f(*x), x, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(RuntimeError, match="first derivatives only"):
        (got[0].square().sum() + x[0].square().sum()).backward()
    for t in x:
        t.grad = None  # (what the other term had left there when the first one raised)
    f(*x).backward(create_graph=True)
    assert all(torch.equal(a, t.grad) for a, t in zip(want, x))
    for t in x:
        t.grad = None
    torch.cuda.synchronize()
