"""Softmax cross entropy with logits far beyond those of any model: a row's loss is right or not finite, never the loss of
a row without its largest item. Products are set by one feature, so that they are known exactly: H's is 0 or a power of
two, E's is 0 for all items but one.

A finite loss of logits up to Z is off by less than 32 u Z, u = 2^-24 (the reference, the target's logit, their difference
and its product with log 2 are each rounded once, the exponentials' sum adds at most 126 to |log2|, which from Z = 2^31 on
is less than 2 u Z), plus the bound of ordinary rows for the other features' part, which is far below 1e-2.
"""
import math

import pytest
import torch

from test_gpu_cross_entropy import BF, F, U24, _gen
from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu

# (type, rows, features): swept in its three widths, tiles of 64 rows, of 128 and of 256
PATHS = [(BF, 40, 64), (BF, 300, 128), (BF, 40, 256), (BF, 40, 264), (BF, 300, 264), (BF, 600, 264), (F, 40, 64), (F, 300, 264)]
V, FAR = 25_000, 12_345


def _inputs(dt, R, D, up, item):
    """H's first feature is `up` in rows 0 to 2, 0 in the others; E's is `item` at FAR, 0 elsewhere. The targets of rows 1
    and 4 are FAR."""
    H = torch.randn(R, D, generator=_gen(1), device="cuda").to(dt)
    E = (torch.randn(V, D, generator=_gen(2), device="cuda") * 0.1).to(dt)
    H[:, 0], E[:, 0] = 0, 0
    H[:3, 0], E[FAR, 0] = up, item
    t = torch.randint(0, FAR, (R,), generator=_gen(3), device="cuda")
    t[1] = t[4] = FAR
    return H, E, t


def _rows(H, E, t):
    z = H.double() @ E.double().T.contiguous()
    return torch.logsumexp(z, 1) - z[torch.arange(len(t), device="cuda"), t]


@pytest.mark.parametrize("dt,R,D", PATHS)
@pytest.mark.parametrize("far", [2.0 ** 18, 1.0e9, -1.0e9, 1.7e10, 3.3e11, 1.0e12, -1.0e12, 7.7e20, 2.2e38, 2.9e38, -2.9e38])
def test_a_row_is_right_or_not_finite(far, dt, R, D):
    up = 2.0 ** 60 if abs(far) > 1e20 else 1.0
    for k in range(8):  # (the reference's rounding depends on the logit's last bits)
        H, E, t = _inputs(dt, R, D, up, far / up * (1 + k / 128))
        if not torch.isfinite(_rows(H, E, t).float()).all():
            continue  # (beyond float32)
        want = _rows(H, E, t)
        size = 32 * U24 * abs(far) * (1 + k / 128) + 1e-2
        for grad in (False, True):
            loss, rows, _ = ops.cross_entropy_forward(H, E, t, want_grad=grad)
            err = (rows.double() - want).abs()
            assert (err[3:] <= 1e-2).all(), (k, err[3:].max())
            off = torch.isfinite(rows[:3]) & ~(err[:3] <= size)
            assert not off.any(), (k, rows[:3], want[:3])
            if abs(far) <= 1.0e9:
                assert torch.isfinite(rows).all()
            assert math.isfinite(loss.item()) == bool(torch.isfinite(rows).all())


@pytest.mark.parametrize("dt,R,D", PATHS)
@pytest.mark.parametrize("far", [1.0e9, 3.3e11, 2.9e38])
def test_gradients_are_right_or_not_finite(far, dt, R, D):
    """Row 0's probability of the far item is 1 and its dH that item less the target, rounded (three roundings of U); where
    probabilities have lost their last bit, dE is not a number rather than a number of no meaning."""
    H, E, t = _inputs(dt, R, D, 2.0 ** 60 if far > 1e20 else 1.0, far / 2.0 ** 60 if far > 1e20 else far)
    loss, rows, saved = ops.cross_entropy_forward(H, E, t)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    for r in (0, 2):
        want = (E[FAR].double() - E[t[r]].double()) / R
        err = (dH[r].double() - want).abs()
        bound = 2.0 ** -6 * (E[FAR].double().abs() + E[t[r]].double().abs()) / R
        assert (~torch.isfinite(dH[r]) | (err <= bound)).all()
    assert torch.isfinite(dH[3:]).all() and torch.isnan(dE).any(0).all()


@pytest.mark.parametrize("dt,R,D", PATHS)
def test_gradients_of_logits_in_the_stated_range(dt, R, D):
    """Logits of 2^18: probabilities are off by 2^-24 of the logarithms, here 2^18 log2(e) / 2^24 = 2.3%, dH's by as much."""
    H, E, t = _inputs(dt, R, D, 1.0, 2.0 ** 18)
    loss, rows, saved = ops.cross_entropy_forward(H, E, t)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    for r in (0, 2):
        want = (E[FAR].double() - E[t[r]].double()) / R
        bound = 0.03 * (E[FAR].double().abs() + E[t[r]].double().abs()) / R
        assert ((dH[r].double() - want).abs() <= bound).all()
    assert torch.isfinite(dH).all() and torch.isfinite(dE).all()
