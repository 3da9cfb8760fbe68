"""Sizes that attention takes and refuses, on the host: each call is held to the workgroups that it launches itself."""
import ctypes

import pytest

from vocabulary_label_bce_amd import binding as B

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = range(7)


def _problem(seqs, rows, capacity, hq, hk, dh=64):
    return B.Attention(seqs * rows, seqs * capacity, hq * dh, dh, hk * dh, dh, hk * dh, dh, capacity * hk * dh,
                       capacity * hk * dh, seqs, hq, hk, dh, B.BF16, 1, 0.125)


def _size(a, backward=0):
    n = ctypes.c_size_t(0)
    return B.lib().cutbce_attention_workspace_size(a, backward, ctypes.byref(n)), n.value


def _forward(a, cu_q=None, size=0):
    """(no workspace, so that a call which is not refused for its sizes stops at the pointers)"""
    return B.lib().cutbce_attention_forward(a, 256, 256, None, cu_q, None, 256, 256, None, None, size, None)


@pytest.mark.parametrize("seqs,capacity,hq,hk", [
    (256, 65_536, 32, 2), (128, 32_768, 128, 8), (64, 131_072, 64, 8), (64, 131_072, 64, 2), (256, 32_768, 64, 8),
    (2, 1 << 29, 8, 1), (4096, 4096, 64, 8)])
def test_large_caches_are_taken(seqs, capacity, hq, hk):
    """One token each: the workgroups are those of the caches' parts, however long the caches are."""
    a = _problem(seqs, 1, capacity, hq, hk)
    status, need = _size(a)
    assert status == OK and need <= 1 << 30
    assert _forward(a) == NULL
    b, forward, backward = B.attention_problem(*(getattr(a, f) for f, _ in B.Attention._fields_))
    assert forward == need and (b.seqs, b.q_heads) == (seqs, hq)
    assert backward is None and _size(a, 1)[0] == SHAPE   # tiles of 64 keys, for which there are too many


@pytest.mark.parametrize("hq,hk", [(8, 1), (64, 1)])
def test_a_prompt_over_large_caches_is_taken(hq, hk):
    a = _problem(64, 500, 131_072, hq, hk)
    assert _size(a)[0] == OK and _forward(a) == NULL


def test_rows_that_one_launch_does_not_take_are_refused():
    """128 rows a workgroup and head, and one more workgroup for each sequence."""
    hq, dh = 128, 64
    for rows, status in ((((1 << 16) - 2) * 128 - 1, OK), (((1 << 16) - 2) * 128, SHAPE)):
        a = B.Attention(rows, 64, hq * dh, dh, dh, dh, dh, dh, 0, 0, 1, hq, 1, dh, B.BF16, 1, 0.125)
        assert _size(a)[0] == status
    # the sizes alone may be those of a cache's single tokens; as packed sequences they are too many
    a = _problem(1 << 18, 1, 16, 32, 8)
    assert _size(a)[0] == OK and _forward(a) == NULL
    assert _forward(a, cu_q=256) == SHAPE
    a = _problem(1 << 21, 1, 16, 4, 4)
    assert _size(a)[0] == SHAPE
    with pytest.raises(B.CutBCEError):
        B.attention_problem(*(getattr(a, f) for f, _ in B.Attention._fields_))


def test_key_rows_are_counted_in_32_bits():
    for rows, status in (((1 << 31) - 1024, OK), ((1 << 31) - 1023, SHAPE)):
        assert _size(B.Attention(1, rows, 64, 64, 64, 64, 64, 64, 0, 0, 1, 1, 1, 64, B.BF16, 1, 0.125))[0] == status
