"""Gradients of the softmax cross entropy whose vocabulary goes in several pieces (tolerances: those of
test_gpu_cross_entropy)."""
import pytest
import torch

from test_gpu_cross_entropy import BF, F, _case, _check
from vocabulary_label_bce_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,V,D,dt,left_out", [
    (4200, 70_001, 264, BF, 0.1),      # a piece of 63,488 items and one of 6,513
    (4200, 63_489, 264, BF, 0.0),      # the second has one item: most parts of dH are empty in it
    (1 << 20, 700, 264, BF, 0.95),     # three, of 256 items at most
    (4200, 35_001, 72, F, 0.1), (4200, 31_745, 72, F, 0.0), (1 << 20, 600, 40, F, 0.95),
])
def test_pieces(R, V, D, dt, left_out):
    # the backward's workspace is that of a vocabulary ten times as large: it is not one piece
    assert B.cross_entropy_sizes(R, V, D, dt)[3] == B.cross_entropy_sizes(R, 10 * V, D, dt)[3]
    H, E, t, w = _case(R, V, D, dt, seed=R + V, left_out=left_out)
    t[:2] = torch.tensor([0, V - 1])
    _check(H, E, t, w, scale=0.8, g=1.5)
