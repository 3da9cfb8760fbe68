"""Gradients of the softmax cross entropy in bf16: a row's own dz, that of its target, is by far its largest and has to keep
more than bf16's eight bits on the way to dH and dE.

Tolerances are those of test_gpu_cross_entropy with one difference: the target's dz is off by U^2 of itself (what its value
rounded to bf16 and the rounded rest leave) instead of U, so that a gradient that this term makes up is off by its own
rounding and little else.
"""
import pytest
import torch

from test_gpu_cross_entropy import BF, U24, UNIT, _case, _close
from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu
U = UNIT[BF]


def _check_own(H, E, t, w, scale):
    loss, rows, saved = ops.cross_entropy_forward(H, E, t, w, scale)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    V, D = E.shape
    keep = torch.nonzero((t >= 0) & (t < V)).flatten()
    h, e, tk, c = H.double()[keep], E.double(), t.long()[keep], w.double()[keep]
    c = c / c.sum()
    at = torch.arange(keep.numel(), device="cuda")
    z = scale * h @ e.T.contiguous()
    A = (abs(scale) * h.abs() @ e.abs().T.contiguous()).amax(1)
    lse = torch.logsumexp(z, 1)
    chain = U24 * (V / 64 + 128)
    ep = (2 * (D + 8) * U24 * A + 4 * U24 * (lse.abs() + z.abs().amax(1) + 1) + chain + 4 * U24)[:, None]
    p = torch.exp(z - lse[:, None])
    p[at, tk] = 0
    dz = p * c[:, None]
    q = dz * (U + ep)
    own = -c * p.sum(1)
    dz[at, tk] = own
    q[at, tk] = own.abs() * (U * U + ep[:, 0])
    for name, got, x, off, y in (("dH", dH[keep], dz, q, e), ("dE", dE, dz.T.contiguous(), q.T.contiguous(), h)):
        want = scale * x @ y
        off = abs(scale) * (off @ y.abs() + U24 * (x.shape[1] / 64 + 128) * (x.abs() @ y.abs()) + 2.0 ** -126 * y.abs().sum(0))
        _close(name, got, want, off + U * (want.abs() + off))


@pytest.mark.parametrize("R,V,D", [
    (300, 5000, 64), (1000, 20_001, 40), (300, 5000, 128), (900, 30_001, 104), (300, 5000, 200), (257, 5000, 256),  # swept
    (300, 5000, 264), (130, 9001, 1000), (40, 9000, 520),  # tiles of 128, and of 64 rows
    (700, 30_000, 264), (1500, 20_003, 520),               # tiles of 256
    (600, 2000, 1024),                                     # dE in parts of the rows
])
def test_own_term(R, V, D):
    H, E, t, w = _case(R, V, D, BF, seed=R + D, lean=0.5, left_out=0.1)
    _check_own(H, E, t, w, 0.9)


@pytest.mark.parametrize("R,V,D", [(5000, 4000, 64), (5000, 4000, 128), (5000, 4000, 256), (2500, 2000, 264), (5000, 4000, 264)])
def test_many_rows_of_few_targets(R, V, D):
    """All rows have one target, or one of the items next to each other at the vocabulary's end; none has."""
    H, E, t, w = _case(R, V, D, BF, seed=7 + D, lean=0.5, left_out=0.1)
    counted = (t >= 0) & (t < V)
    for k in (1, 40, 400):
        few = V - 1 - torch.arange(R, device="cuda", dtype=t.dtype) % k
        _check_own(H, E, torch.where(counted, few, t), w, -0.7)
