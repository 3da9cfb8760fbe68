"""Layer norm with a bias and no weight, and its gradients, against float64.

Tolerance of dbias: a float32 sum of n rows in any order, (n + 8) 2^-24 sum |dy|, and the rounding of the bias's own type
(2^-24 float32, 2^-8 bfloat16), not of the rows'."""
import pytest
import torch

from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.mark.parametrize("rows,D", [(1, 8), (77, 100), (1000, 128), (5, 9001)])
@pytest.mark.parametrize("pdt", U)
@pytest.mark.parametrize("dt", U)
def test_bias_alone(dt, pdt, rows, D):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, D, generator=gen, device="cuda").to(dt).requires_grad_()
    b = torch.randn(D, generator=gen, device="cuda").to(pdt).requires_grad_()
    dy = torch.randn(rows, D, generator=gen, device="cuda").to(dt)
    y = ops.layer_norm(x, None, b)
    y.backward(dy)
    X = x.detach().double()
    m = X.mean(1, keepdim=True)
    r = 1 / torch.sqrt((X - m).square().mean(1, keepdim=True) + 1e-5)
    want = (X - m) * r + b.detach().double()
    size = ((X.abs() + X.abs().mean(1, keepdim=True)) * r + b.detach().double().abs())
    xh = (X - m) * r
    e = (D + 8) * 2.0 ** -24
    assert bool(((y.detach().double() - want).abs() <= e * size * (1 + xh.square()) + (U[dt] + e) * want.abs()).all())
    G = dy.double()
    assert b.grad.dtype == pdt
    bound = (rows + 8) * 2.0 ** -24 * G.abs().sum(0) + U[pdt] * G.sum(0).abs()
    assert bool(((b.grad.double() - G.sum(0)).abs() <= bound).all())
    _, mu, rs = ops.layer_norm_forward(x.detach(), None, b.detach())
    dx, dw, db = ops.layer_norm_backward(dy, x.detach(), None, mu, rs)
    assert torch.equal(dx, x.grad) and dw.dtype == dt and db.dtype == dt
    dx, dw, db = ops.layer_norm_backward(dy, x.detach(), None, mu, rs, param_dtype=pdt)
    assert torch.equal(dx, x.grad) and dw.dtype == pdt and torch.equal(db, b.grad)
    with pytest.raises(ValueError, match="param_dtype"):
        ops.layer_norm_backward(dy, x.detach(), None, mu, rs, param_dtype=torch.float16)
    with pytest.raises(ValueError, match="param_dtype"):
        w = torch.ones(D, device="cuda", dtype=torch.float32)
        ops.layer_norm_backward(dy, x.detach(), w, mu, rs, param_dtype=torch.bfloat16)
