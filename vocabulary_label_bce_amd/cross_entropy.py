"""PyTorch front end of the softmax cross entropy over a whole vocabulary: ``cut_cross_entropy`` is differentiable in
reverse mode; ``cross_entropy_forward`` and ``cross_entropy_backward`` serve callers that keep their own tape. The
logits are never kept. The arithmetic is libcutbce.so's; all tensors live on the current GPU and nothing synchronises
with the host.
"""
from __future__ import annotations

import math

import torch

from . import binding as B
from .encoder import _FLOATS, _aligned, _derived, _first_order, _on_gpu


class Saved:
    """What a forward keeps for its backwards: an opaque buffer, and the sizes and scale that it goes with."""

    __slots__ = ("buffer", "rows", "vocab", "dim", "dtype", "scale")

    def __init__(self, buffer, rows, vocab, dim, dtype, scale):
        self.buffer, self.rows, self.vocab, self.dim, self.dtype, self.scale = buffer, rows, vocab, dim, dtype, scale


def _checked(H, E, targets, row_weight, scale):
    dev = _on_gpu("cross_entropy", H, E, targets, row_weight)
    if H.dtype not in _FLOATS or E.dtype != H.dtype:
        raise ValueError("H and E must both be float32 or both bfloat16")
    if H.dim() != 2 or E.dim() != 2 or H.shape[1] != E.shape[1]:
        raise ValueError("H must be [R, D] and E [V, D]")
    if E.shape[1] % 8 or not 8 <= E.shape[1] <= 16384:
        raise ValueError("D must be a multiple of 8, at most 16384")
    if E.shape[0] < 1 or H.shape[0] > 1 << 20:
        raise ValueError("there must be an item, and at most 2**20 rows")
    if targets.dtype not in (torch.int32, torch.int64) or targets.shape != H.shape[:1]:
        raise ValueError("targets must be int32 or int64 [R]")
    if row_weight is not None and (row_weight.dtype not in _FLOATS or row_weight.shape != H.shape[:1]):
        raise ValueError("row_weight must be float32 or bfloat16 [R]")
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    if row_weight is not None:
        row_weight = row_weight.detach().float().contiguous()
    return dev, _aligned(H.contiguous()), _aligned(E.contiguous()), targets.contiguous(), row_weight


def cross_entropy_forward(H, E, targets, row_weight=None, scale: float = 1.0, want_grad: bool = True):
    """(loss, row_loss, saved) of cut_cross_entropy: loss float32 0-d; row_loss float32 [R], each row's own loss, 0
    where it is left out; saved for cross_entropy_backward, None with want_grad=False. For bfloat16 and D up to 256
    saved has dH (R * D float32, half of the forward's products), also where the backward will be asked for dE alone."""
    dev, H, E, targets, row_weight = _checked(H, E, targets, row_weight, scale)
    R, (V, D) = H.shape[0], E.shape
    saved_bytes, alone, beside, _ = B.cross_entropy_sizes(R, V, D, H.dtype)
    loss = H.new_empty((), dtype=torch.float32)
    row_loss = H.new_empty(R, dtype=torch.float32)
    buffer = H.new_empty(saved_bytes, dtype=torch.uint8) if want_grad else None
    ws = H.new_empty(beside if want_grad else alone, dtype=torch.uint8)
    B.cross_entropy_forward(H, E, targets, row_weight, scale, loss, row_loss, buffer, ws, B.raw_stream(dev))
    return loss, row_loss, Saved(buffer, R, V, D, H.dtype, scale) if want_grad else None


def cross_entropy_backward(grad, H, E, saved, want_dH: bool = True, want_dE: bool = True):
    """(dH, dE) from the cotangent of the loss (one element on the device), the forward's H and E and what it saved (of
    H the shape and type alone are looked at: its counted rows are in saved). What is not wanted is None."""
    dev = _on_gpu("cross_entropy_backward", E, H, grad, saved.buffer)
    R, V, D, dt = saved.rows, saved.vocab, saved.dim, saved.dtype
    if H.shape != (R, D) or E.shape != (V, D) or H.dtype != dt or E.dtype != dt:
        raise ValueError("H and E must be the forward's")
    if grad.numel() != 1:
        raise ValueError("grad must have one element")
    if not (want_dH or want_dE):
        return None, None
    grad = grad.detach().reshape(1).float()
    E = _aligned(E.contiguous())
    dH = H.new_empty((R, D)) if want_dH else None
    dE = E.new_empty((V, D)) if want_dE else None
    ws = E.new_empty(B.cross_entropy_sizes(R, V, D, dt)[3], dtype=torch.uint8)
    B.cross_entropy_backward(R, E, saved.scale, grad, saved.buffer, dH, dE, ws, B.raw_stream(dev))
    return dH, dE


class _CutCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, E, targets, row_weight, scale):
        loss, _, saved = cross_entropy_forward(H, E, targets, row_weight, scale)
        ctx.save_for_backward(H, E)
        ctx.saved = saved
        return loss

    @staticmethod
    @_first_order
    def backward(ctx, g):
        H, E = ctx.saved_tensors
        need = ctx.needs_input_grad
        return cross_entropy_backward(g, H, E, ctx.saved, need[0], need[1]) + (None,) * 3


def cut_cross_entropy(H, E, targets, row_weight=None, scale: float = 1.0):
    """Softmax cross entropy of the logits scale * H @ E.T over all V items, averaged over the rows that have a target.

    H [R, D] and E [V, D] (float32 or bfloat16, D a multiple of 8 up to 16384), targets [R] int32 or int64: a row whose
    target is outside [0, V) (padding, e.g. -1) is left out of the loss and gets no gradient. row_weight [R] (finite,
    >= 0): the loss becomes the average weighted by it. scale: 1 / temperature. Returns a 0-d float32; gradients flow to
    H and E (not to the weights). No tensor of R x V elements is kept: memory is bounded in V.

    Logits up to 1e9 are taken; a row with one beyond has the right loss or one that is not finite. The probabilities
    that gradients are made of are off by 2^-24 |logsumexp / log 2|, and not a number where that is 1 (from 1.1e7 on).
    """
    if _derived(row_weight):
        raise ValueError("row_weight gets no gradient and no tangent: detach it")
    if _derived(H, E):
        return _CutCrossEntropy.apply(H, E, targets, row_weight, scale)
    return cross_entropy_forward(H, E, targets, row_weight, scale, want_grad=False)[0]
