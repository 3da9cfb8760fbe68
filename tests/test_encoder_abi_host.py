"""Host-side checks of the sequence encoder's entry points: sizes of workspaces, and arguments that are refused before
anything is enqueued (no call here reaches a launch, so made-up device addresses are safe)."""
import ctypes
import math

import pytest

from vocabulary_label_bce_amd import binding as B

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = range(7)


def _attention(**over):
    f = dict(q_rows=64, k_rows=64, q_row_stride=256, q_head_stride=64, k_row_stride=128, k_head_stride=64,
             v_row_stride=128, v_head_stride=64, k_seq_stride=0, v_seq_stride=0, seqs=2, q_heads=4, kv_heads=2,
             head_dim=64, dtype=B.BF16, causal=1, scale=0.125)
    f.update(over)
    return B.Attention(**f)


def _forward(a, q=256, k=256, v=256, cu_q=256, cu_k=None, lens=None, out=256, lse=256, ws=256, size=0):
    return B.lib().cutbce_attention_forward(a, q, k, v, cu_q, cu_k, lens, out, lse, ws, size, None)


def _backward(a, dout=256, q=256, k=256, v=256, out=256, lse=256, cu_q=256, dq=256, dk=256, dv=256, ws=256, size=0):
    return B.lib().cutbce_attention_backward(a, dout, q, k, v, out, lse, cu_q, None, None, dq, dk, dv, ws, size, None)


@pytest.mark.parametrize("over,status", [
    (dict(head_dim=20), UNSUPPORTED), (dict(head_dim=136), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
    (dict(dtype=7), DTYPE), (dict(seqs=0), SHAPE), (dict(q_rows=-1), SHAPE), (dict(q_heads=3), SHAPE),
    (dict(kv_heads=0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE),
    (dict(q_row_stride=-256), SHAPE), (dict(k_row_stride=132), ALIGN), (dict(v_head_stride=4), ALIGN),
    (dict(k_rows=32), SHAPE),   # no cu_k and no k_lens: the keys are the queries' rows
])
def test_attention_problem_is_checked(over, status):
    a = _attention(**over)
    assert _forward(a, size=1 << 40) == status
    assert _backward(a, size=1 << 40) == status


@pytest.mark.parametrize("name", ["q", "k", "v", "out"])
def test_attention_pointers_are_checked(name):
    a = _attention()
    assert _forward(a, size=1 << 40, **{name: None}) == NULL
    assert _forward(a, size=1 << 40, **{name: 264}) == ALIGN
    assert _backward(a, size=1 << 40, **{name: None}) == NULL
    assert _backward(a, size=1 << 40, **{name: 264}) == ALIGN


def test_attention_backward_needs_its_workspace():
    a = _attention()
    n = ctypes.c_size_t(0)
    assert B.lib().cutbce_attention_workspace_size(a, 1, ctypes.byref(n)) == OK and n.value > 0
    assert _backward(a, size=n.value - 1) == WORKSPACE
    assert _backward(a, ws=None, size=n.value) == NULL
    assert _backward(a, ws=128, size=n.value) == ALIGN
    for name in ("dout", "lse", "dq", "dk", "dv"):
        assert _backward(a, size=n.value, **{name: None}) == NULL
    assert B.lib().cutbce_attention_workspace_size(a, 0, None) == NULL
    assert B.lib().cutbce_attention_workspace_size(None, 0, ctypes.byref(n)) == NULL


def test_attention_without_rows_does_nothing():
    assert _forward(_attention(q_rows=0, k_rows=0), q=None, out=None) == OK
    assert _backward(_attention(q_rows=0, k_rows=0), dq=None, dk=None, dv=None) == OK


def test_attention_workspace_grows_with_rows_not_with_rows_times_keys():
    sizes = []
    for rows in (1 << 12, 1 << 16):
        n = ctypes.c_size_t(0)
        assert B.lib().cutbce_attention_workspace_size(_attention(q_rows=rows, k_rows=rows), 1, ctypes.byref(n)) == OK
        sizes.append(n.value)
    assert sizes[1] <= 16 * sizes[0] + (1 << 20)


def _embed(n=4, V=10, D=8, dtype=B.BF16, id_bytes=4, ids=256, table=256, out=256, scale=1.0):
    return B.lib().cutbce_embedding_forward(n, V, D, dtype, id_bytes, ids, table, scale, out, None)


def _embed_grad(n=4, V=10, D=8, dtype=B.BF16, id_bytes=4, ids=256, dout=256, out=256, ws=256, size=1 << 40):
    return B.lib().cutbce_embedding_backward(n, V, D, dtype, id_bytes, ids, dout, 1.0, 0, out, ws, size, None)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(V=0), SHAPE), (dict(V=(1 << 31) - 1024), SHAPE),
    (dict(D=0), SHAPE), (dict(D=65537), SHAPE), (dict(dtype=2), DTYPE), (dict(id_bytes=2), DTYPE),
    (dict(ids=None), NULL), (dict(out=None), NULL), (dict(ids=258), ALIGN), (dict(out=264), ALIGN),
])
def test_embedding_arguments_are_checked(over, status):
    assert _embed(**over) == status
    assert _embed_grad(**over) == status


def test_embedding_more():
    assert _embed(table=None) == NULL and _embed(table=8) == ALIGN and _embed(n=0, ids=None, out=None) == OK
    assert _embed_grad(dout=None) == NULL and _embed_grad(ws=None) == NULL and _embed_grad(ws=16) == ALIGN
    need = B.embedding_backward_workspace_size(25600, 876000, 128, __import__("torch").bfloat16)
    assert 25600 * 16 <= need < 25600 * 128 * 4
    assert _embed_grad(n=25600, V=876000, D=128, size=need - 1) == WORKSPACE


def _norm(rows=4, D=8, dtype=B.BF16, pd=B.F32, x=256, xs=8, w=256, b=256, eps=1e-5, y=256, m=256, r=256):
    return B.lib().cutbce_layer_norm_forward(rows, D, dtype, pd, x, xs, w, b, eps, y, m, r, None)


def _norm_grad(rows=4, D=8, dtype=B.BF16, pd=B.F32, x=256, xs=8, dy=256, dys=8, w=256, m=256, r=256, dx=256, dw=256,
               db=256, ws=256, size=1 << 40):
    return B.lib().cutbce_layer_norm_backward(rows, D, dtype, pd, dy, dys, x, xs, w, m, r, dx, dw, db, ws, size, None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), SHAPE), (dict(D=0), SHAPE), (dict(D=65537), SHAPE), (dict(dtype=3), DTYPE), (dict(pd=3), DTYPE),
    (dict(xs=7), SHAPE), (dict(x=None), NULL), (dict(x=257), ALIGN), (dict(w=258), ALIGN), (dict(m=258), ALIGN),
    (dict(m=None), NULL),
])
def test_layer_norm_arguments_are_checked(over, status):
    assert _norm(**over) == status
    assert _norm_grad(**over) == status


def test_layer_norm_more():
    assert _norm(eps=-1.0) == SHAPE and _norm(eps=math.nan) == SHAPE and _norm(y=None) == NULL
    assert _norm(rows=0, x=None, y=None) == OK
    assert _norm_grad(dys=0) == SHAPE and _norm_grad(dy=None) == NULL and _norm_grad(ws=None) == NULL
    assert _norm_grad(dw=None, db=None, dx=None, ws=None) == OK
    need = B.layer_norm_backward_workspace_size(25600, 128)
    assert 0 < need < 25600 * 128 * 4
    assert _norm_grad(rows=25600, D=128, xs=128, dys=128, size=need - 1) == WORKSPACE


def test_sizes_that_one_launch_does_not_take_are_refused():
    most = 1 << 28
    assert _embed_grad(n=most + 1) == SHAPE and _embed_grad(n=most, V=10, D=8, size=0) == WORKSPACE
    n = ctypes.c_size_t(0)
    size = B.lib().cutbce_embedding_backward_workspace_size
    assert size(most + 1, 10, 8, B.BF16, ctypes.byref(n)) == SHAPE and size(most, 10, 8, B.BF16, ctypes.byref(n)) == OK
    heads = dict(q_heads=128, kv_heads=1, seqs=1, q_row_stride=128 * 64, k_row_stride=64, v_row_stride=64)
    rows = ((1 << 16) - 3) * 64   # rows / 64 + seqs + 1 tiles
    assert B.lib().cutbce_attention_workspace_size(_attention(q_rows=rows, k_rows=rows, **heads), 1, ctypes.byref(n)) == OK
    rows += 64
    assert B.lib().cutbce_attention_workspace_size(_attention(q_rows=rows, k_rows=rows, **heads), 1, ctypes.byref(n)) == SHAPE
