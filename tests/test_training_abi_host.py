"""Host-side checks of the training step's entry points: workspace sizes, and arguments that are refused before anything
is enqueued (no call here reaches a launch, so made-up device addresses are safe)."""
import ctypes
import math

import pytest
import torch

from vocabulary_label_bce_amd import binding as B

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = range(7)
F32, BF16 = B.F32, B.BF16


def _norm(grads=(256,), n=(4,), types=(BF16,), out=256, ws=256, size=1 << 40):
    a = (ctypes.c_void_p * len(grads))(*grads)
    b = (ctypes.c_int64 * len(n))(*n)
    c = (ctypes.c_int32 * len(types))(*types)
    return B.lib().cutbce_grad_norm(len(n), a, b, c, out, ws, size, None)


@pytest.mark.parametrize("over,status", [
    (dict(n=(-1,)), SHAPE), (dict(n=(1 << 50,)), SHAPE), (dict(types=(2,)), DTYPE), (dict(grads=(None,)), NULL),
    (dict(grads=(257,)), ALIGN), (dict(grads=(258,), types=(F32,)), ALIGN), (dict(out=None), NULL),
    (dict(out=258), ALIGN), (dict(ws=None), NULL), (dict(ws=128), ALIGN), (dict(size=7), WORKSPACE),
])
def test_norm_arguments_are_checked(over, status):
    assert _norm(**over) == status


def test_norm_workspace():
    assert B.grad_norm_workspace_size(()) == 0
    assert B.grad_norm_workspace_size((0, 0)) == 0
    assert 0 < B.grad_norm_workspace_size((1, 10_000_000)) < 10_000
    n = ctypes.c_size_t(0)
    assert B.lib().cutbce_grad_norm_workspace_size(-1, None, ctypes.byref(n)) == SHAPE
    assert B.lib().cutbce_grad_norm_workspace_size(1, None, ctypes.byref(n)) == NULL
    assert B.lib().cutbce_grad_norm_workspace_size(0, None, None) == NULL


TENSOR = dict(p=256, g=256, m=256, v=256, ms=None, vs=None, master=None, n=4, pt=BF16, gt=BF16, decay=0.1)
HOW = dict(step=256, lr_at=None, norm=None, max_norm=0.0, lr=1e-3, eps=1e-8, beta1=0.9, beta2=0.999, state_bits=32,
           seed=1)


def _adamw(how=(), count=1, missing=None, **over):
    t = dict(TENSOR, **over)
    one = {k: (ctypes.c_void_p * 1)(t[k] or None) for k in ("p", "g", "m", "v", "ms", "vs", "master")}
    one["n"] = (ctypes.c_int64 * 1)(t["n"])
    one["pt"], one["gt"] = (ctypes.c_int32 * 1)(t["pt"]), (ctypes.c_int32 * 1)(t["gt"])
    one["decay"] = (ctypes.c_float * 1)(t["decay"])
    x = B.AdamWTensors(count, 0, *[None if k == missing else ctypes.addressof(a) for k, a in one.items()])
    h = dict(HOW, **dict(how))
    return B.lib().cutbce_adamw_step(ctypes.byref(x), ctypes.byref(B.AdamW(*h.values())), None)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), SHAPE), (dict(n=1 << 40), SHAPE), (dict(pt=2), DTYPE), (dict(gt=-1), DTYPE), (dict(p=None), NULL),
    (dict(g=None), NULL), (dict(m=None), NULL), (dict(v=None), NULL), (dict(p=257), ALIGN), (dict(m=258), ALIGN),
    (dict(master=258), ALIGN), (dict(decay=math.inf), SHAPE), (dict(count=-1), SHAPE), (dict(count=(1 << 20) + 1), SHAPE),
])
def test_adamw_tensors_are_checked(over, status):
    assert _adamw(**over) == status


@pytest.mark.parametrize("how,status", [
    (dict(step=None), NULL), (dict(step=258), ALIGN), (dict(lr_at=258), ALIGN), (dict(norm=258), ALIGN),
    (dict(beta1=1.0), SHAPE), (dict(beta2=-0.1), SHAPE), (dict(beta1=math.nan), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=math.inf), SHAPE), (dict(lr=math.nan), SHAPE), (dict(norm=256, max_norm=-1.0), SHAPE),
    (dict(norm=256, max_norm=math.nan), SHAPE), (dict(state_bits=16), DTYPE), (dict(state_bits=8), NULL),
])
def test_adamw_hyperparameters_are_checked(how, status):
    assert _adamw(how) == status


@pytest.mark.parametrize("name", ["p", "g", "m", "v", "n", "pt", "gt", "decay"])
def test_adamw_lists_are_checked(name):
    assert _adamw(missing=name) == NULL


def test_adamw_structs_are_checked():
    how = ctypes.byref(B.AdamW(*HOW.values()))
    assert B.lib().cutbce_adamw_step(None, how, None) == NULL
    assert B.lib().cutbce_adamw_step(ctypes.byref(B.AdamWTensors()), None, None) == NULL
    assert _adamw(dict(state_bits=8), ms=256, vs=256, missing="vs") == NULL
    assert _adamw(dict(state_bits=8), ms=258, vs=256) == ALIGN


CE = dict(R=64, V=1000, D=64, dt=BF16, idb=4, H=256, E=256, t=256, w=None, scale=1.0, loss=256, row=None, saved=256, ws=256,
          size=1 << 40)
BACK = dict(R=64, V=1000, D=64, dt=BF16, E=256, scale=1.0, g=256, saved=256, dH=256, dE=256, ws=256, size=1 << 40)


def _forward(**over):
    return B.lib().cutbce_cross_entropy_forward(*dict(CE, **over).values(), None)


def _backward(**over):
    return B.lib().cutbce_cross_entropy_backward(*dict(BACK, **over).values(), None)


SIZES = [(dict(R=-1), SHAPE), (dict(R=(1 << 20) + 1), None), (dict(V=0), SHAPE), (dict(V=1 << 40), None),
         (dict(D=0), UNSUPPORTED), (dict(D=12), None), (dict(D=16392), None), (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE)]


@pytest.mark.parametrize("over,status", SIZES)
def test_cross_entropy_sizes_are_checked(over, status):
    """One answer from every entry point; sizes beyond the operator's are SHAPE or UNSUPPORTED."""
    n = ctypes.c_size_t(0)
    x = dict(CE, **over)
    size = x["R"], x["V"], x["D"], x["dt"]
    got = [_forward(**over), _backward(**over), B.lib().cutbce_cross_entropy_saved_size(*size, ctypes.byref(n))]
    got += [B.lib().cutbce_cross_entropy_workspace_size(*size, k, ctypes.byref(n)) for k in range(3)]
    assert len(set(got)) == 1 and (got[0] == status or (status is None and got[0] in (SHAPE, UNSUPPORTED)))


@pytest.mark.parametrize("over,status", [
    (dict(idb=2), DTYPE), (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE), (dict(E=None), NULL),
    (dict(H=None), NULL), (dict(t=None), NULL), (dict(loss=None), NULL), (dict(ws=None), NULL), (dict(H=264), ALIGN),
    (dict(E=264), ALIGN), (dict(t=258), ALIGN), (dict(t=260, idb=8), ALIGN), (dict(w=258), ALIGN), (dict(loss=258), ALIGN),
    (dict(row=258), ALIGN), (dict(saved=128), ALIGN), (dict(ws=128), ALIGN), (dict(size=0), WORKSPACE),
])
def test_cross_entropy_forward_arguments_are_checked(over, status):
    assert _forward(**over) == status


@pytest.mark.parametrize("over,status", [
    (dict(scale=math.inf), SHAPE), (dict(E=None), NULL), (dict(g=None), NULL), (dict(saved=None), NULL), (dict(ws=None), NULL),
    (dict(E=264), ALIGN), (dict(g=258), ALIGN), (dict(saved=128), ALIGN), (dict(dH=264), ALIGN), (dict(dE=264), ALIGN),
    (dict(ws=128), ALIGN), (dict(size=0), WORKSPACE), (dict(dH=None, dE=None), OK),
])
def test_cross_entropy_backward_arguments_are_checked(over, status):
    assert _backward(**over) == status


def test_cross_entropy_queries():
    n = ctypes.c_size_t(0)
    ok = 64, 1000, 64, BF16
    assert B.lib().cutbce_cross_entropy_saved_size(*ok, None) == NULL
    assert B.lib().cutbce_cross_entropy_workspace_size(*ok, 0, None) == NULL
    for which in (-1, 3):
        assert B.lib().cutbce_cross_entropy_workspace_size(*ok, which, ctypes.byref(n)) == SHAPE


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("R,D", [(1, 8), (4096, 64), (4096, 512), (25_600, 128), (1 << 20, 256), (4096, 16384)])
def test_cross_entropy_memory_is_bounded_in_the_vocabulary(R, D, dt):
    """Ten times the items of a vocabulary that goes in pieces (or is swept): nothing grows."""
    small, large = (B.cross_entropy_sizes(R, V, D, {BF16: torch.bfloat16, F32: torch.float32}[dt]) for V in (10 ** 7, 10 ** 8))
    assert small == large
    # a piece's dz (of 256 items at least), dH's sums, and what is resident
    assert large[3] <= max(512 << 20, (R + 31) // 32 * 32 * 256 * (2 if dt == BF16 else 4)) + R * D * 4 + (1 << 28)
