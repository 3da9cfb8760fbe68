"""ctypes binding of libcutbce.so (C ABI in include/cutbce.h).

Every function here only marshals arguments: tensors become device pointers, the current torch stream becomes
the hipStream_t, and status codes become exceptions. All computation happens in the HIP library. If the
library has not been built, the first call raises (there is no fallback path).
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcutbce.so")

F32, BF16 = 0, 1
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_lock = threading.Lock()
_lib = None


class CutBCEError(RuntimeError):
    pass


class Problem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("nnz", ctypes.c_int64),
                ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Attention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("q_rows", "k_rows", "q_row_stride", "q_head_stride", "k_row_stride",
                                              "k_head_stride", "v_row_stride", "v_head_stride", "k_seq_stride",
                                              "v_seq_stride")] + \
               [(n, ctypes.c_int32) for n in ("seqs", "q_heads", "kv_heads", "head_dim", "dtype", "causal")] + \
               [("scale", ctypes.c_float)]


class AdamWTensors(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("reserved", ctypes.c_int32)] + \
               [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                               "exp_avg_sq_scale", "master", "n", "param_dtype", "grad_dtype",
                                               "weight_decay")]


class AdamW(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("step", "lr_at", "norm")] + \
               [(n, ctypes.c_double) for n in ("max_norm", "lr", "eps", "beta1", "beta2")] + \
               [("state_bits", ctypes.c_int32), ("seed", ctypes.c_uint32)]


EXPORTS = ["cutbce_workspace_size", "cutbce_forward", "cutbce_forward_noalloc", "cutbce_backward",
           "cutbce_backward_reuse", "cutbce_validate_targets",
           "cutbce_targets_to_csr", "cutbce_topk",
           "cutbce_embedding_forward", "cutbce_embedding_backward_workspace_size", "cutbce_embedding_backward",
           "cutbce_layer_norm_forward", "cutbce_layer_norm_backward_workspace_size", "cutbce_layer_norm_backward",
           "cutbce_attention_workspace_size", "cutbce_attention_forward", "cutbce_attention_backward",
           "cutbce_cross_entropy_saved_size", "cutbce_cross_entropy_workspace_size", "cutbce_cross_entropy_forward",
           "cutbce_cross_entropy_backward",
           "cutbce_grad_norm_workspace_size", "cutbce_grad_norm", "cutbce_adamw_step",
           "cutbce_profile_enable", "cutbce_profile_read", "cutbce_mfma_ceiling",
           "cutbce_mfma_ceiling_random", "cutbce_status_string",
           "cutbce_version"]


def lib():
    """Load libcutbce.so once; raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise CutBCEError(f"{LIB_PATH} is not built; run `python -m vocabulary_label_bce_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        P = ctypes.POINTER(Problem)
        L.cutbce_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.cutbce_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_forward_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.cutbce_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_backward_reuse.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_validate_targets.argtypes = [P, vp, vp, vp, vp]
        L.cutbce_targets_to_csr.argtypes = [ctypes.c_int64, ctypes.c_int32, vp, ctypes.c_int32, vp, vp, vp]
        L.cutbce_topk.argtypes = [P, vp, vp, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, sz, vp]
        i64, f32, AP = ctypes.c_int64, ctypes.c_float, ctypes.POINTER(Attention)
        L.cutbce_embedding_forward.argtypes = [i64, i64, i32, i32, i32, vp, vp, f32, vp, vp]
        L.cutbce_embedding_backward_workspace_size.argtypes = [i64, i64, i32, i32, ctypes.POINTER(sz)]
        L.cutbce_embedding_backward.argtypes = [i64, i64, i32, i32, i32, vp, vp, f32, i32, vp, vp, sz, vp]
        L.cutbce_layer_norm_forward.argtypes = [i64, i32, i32, i32, vp, i64, vp, vp, f32, vp, vp, vp, vp]
        L.cutbce_layer_norm_backward_workspace_size.argtypes = [i64, i32, ctypes.POINTER(sz)]
        L.cutbce_layer_norm_backward.argtypes = [i64, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, sz,
                                                 vp]
        L.cutbce_attention_workspace_size.argtypes = [AP, i32, ctypes.POINTER(sz)]
        L.cutbce_attention_forward.argtypes = [AP, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_attention_backward.argtypes = [AP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_cross_entropy_saved_size.argtypes = [i64, i64, i32, i32, ctypes.POINTER(sz)]
        L.cutbce_cross_entropy_workspace_size.argtypes = [i64, i64, i32, i32, i32, ctypes.POINTER(sz)]
        L.cutbce_cross_entropy_forward.argtypes = [i64, i64, i32, i32, i32, vp, vp, vp, vp, f32, vp, vp, vp, vp, sz, vp]
        L.cutbce_cross_entropy_backward.argtypes = [i64, i64, i32, i32, vp, f32, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_grad_norm_workspace_size.argtypes = [i32, vp, ctypes.POINTER(sz)]
        L.cutbce_grad_norm.argtypes = [i32, vp, vp, vp, vp, vp, sz, vp]
        L.cutbce_adamw_step.argtypes = [ctypes.POINTER(AdamWTensors), ctypes.POINTER(AdamW), vp]
        L.cutbce_profile_enable.argtypes = [i32]
        L.cutbce_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64), i32]
        L.cutbce_profile_enable.restype = i32
        L.cutbce_profile_read.restype = i32
        L.cutbce_mfma_ceiling.argtypes = [i32, i32, i32, vp, vp]
        L.cutbce_mfma_ceiling.restype = i32
        L.cutbce_mfma_ceiling_random.argtypes = [i32, i32, i32, vp, vp]
        L.cutbce_mfma_ceiling_random.restype = i32
        L.cutbce_status_string.argtypes = [i32]
        L.cutbce_status_string.restype = ctypes.c_char_p
        L.cutbce_version.restype = i32
        for f in ("cutbce_workspace_size", "cutbce_forward", "cutbce_forward_noalloc", "cutbce_backward",
                  "cutbce_backward_reuse", "cutbce_validate_targets",
                  "cutbce_targets_to_csr", "cutbce_topk", "cutbce_embedding_forward",
                  "cutbce_embedding_backward_workspace_size", "cutbce_embedding_backward",
                  "cutbce_layer_norm_forward", "cutbce_layer_norm_backward_workspace_size",
                  "cutbce_layer_norm_backward", "cutbce_attention_workspace_size", "cutbce_attention_forward",
                  "cutbce_attention_backward", "cutbce_cross_entropy_saved_size",
                  "cutbce_cross_entropy_workspace_size", "cutbce_cross_entropy_forward",
                  "cutbce_cross_entropy_backward", "cutbce_grad_norm_workspace_size", "cutbce_grad_norm",
                  "cutbce_adamw_step"):
            getattr(L, f).restype = i32
        _lib = L
        return L


def _check(st: int):
    if st != 0:
        raise CutBCEError(f"cutbce status {st}: {lib().cutbce_status_string(st).decode()}")


def problem(R: int, V: int, nnz: int, D: int, dtype) -> Problem:
    dt = _DTYPES.get(dtype, dtype) if not isinstance(dtype, int) else dtype
    if dt not in (F32, BF16):
        raise CutBCEError(f"unsupported dtype {dtype}")
    return Problem(int(R), int(V), int(nnz), int(D), int(dt))


def workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().cutbce_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def problem_of(H, E, item_ids) -> Problem:
    return problem(H.shape[0], E.shape[0], item_ids.numel(), H.shape[1], H.dtype)


def alloc_workspace(p: Problem, device) -> torch.Tensor:
    return torch.empty(workspace_size(p), dtype=torch.uint8, device=device)


def forward(p: Problem, H, E, row_offsets, item_ids, row_mask, loss, row_loss, dh_saved, ws, stream=None,
            metrics=None, row_weight=None):
    """cutbce_forward on device tensors (outputs written in place; metrics: int32 [R, 4] or None;
    row_weight: float32 [R] or None)."""
    _check(lib().cutbce_forward(ctypes.byref(p), _ptr(H), _ptr(E), _ptr(row_offsets), _ptr(item_ids),
                                _ptr(row_mask), _ptr(row_weight), _ptr(loss), _ptr(row_loss), _ptr(dh_saved),
                                _ptr(metrics), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 64 << 20  # CUTBCE_NOALLOC_SCRATCH_BYTES


def forward_noalloc(p: Problem, H, E, row_offsets, item_ids, row_mask, loss, row_loss, dh_saved, stream=None,
                    metrics=None, row_weight=None):
    """cutbce_forward_noalloc: cutbce_forward with the library's own per-GPU scratch array as workspace."""
    _check(lib().cutbce_forward_noalloc(ctypes.byref(p), _ptr(H), _ptr(E), _ptr(row_offsets), _ptr(item_ids),
                                        _ptr(row_mask), _ptr(row_weight), _ptr(loss), _ptr(row_loss),
                                        _ptr(dh_saved), _ptr(metrics), _stream(stream)))


def backward(p: Problem, H, E, row_offsets, item_ids, row_mask, grad_loss, dh_saved, dH, dE, ws, stream=None,
             row_weight=None, reuse=False):
    """cutbce_backward on device tensors (dH / dE overwritten in place; either may be None). reuse=True calls
    cutbce_backward_reuse: `ws` must hold what cutbce_forward left for these same inputs."""
    f = lib().cutbce_backward_reuse if reuse else lib().cutbce_backward
    _check(f(ctypes.byref(p), _ptr(H), _ptr(E), _ptr(row_offsets), _ptr(item_ids), _ptr(row_mask),
             _ptr(row_weight), _ptr(grad_loss), _ptr(dh_saved), _ptr(dH), _ptr(dE), _ptr(ws),
             ws.numel() if ws is not None else 0, _stream(stream)))


def topk(p: Problem, H, E, row_offsets, item_ids, row_mask, k: int, top_vals, top_ids, hits, ws, stream=None):
    """cutbce_topk on device tensors: top_vals float [R, k], top_ids int32 [R, k], hits int32 [R] or None."""
    _check(lib().cutbce_topk(ctypes.byref(p), _ptr(H), _ptr(E), _ptr(row_offsets), _ptr(item_ids), _ptr(row_mask),
                             int(k), _ptr(top_vals), _ptr(top_ids), _ptr(hits), _ptr(ws),
                             ws.numel() if ws is not None else 0, _stream(stream)))


def targets_to_csr(targets, pad_id: int, row_offsets, item_ids, stream=None):
    """cutbce_targets_to_csr: targets int32 [R, L] on the device -> row_offsets [R+1], item_ids [R*L] (in place)."""
    R, L = targets.shape
    _check(lib().cutbce_targets_to_csr(int(R), int(L), _ptr(targets), int(pad_id), _ptr(row_offsets),
                                       _ptr(item_ids), _stream(stream)))


def validate_targets(p: Problem, row_offsets, item_ids, bad, stream=None):
    _check(lib().cutbce_validate_targets(ctypes.byref(p), _ptr(row_offsets), _ptr(item_ids), _ptr(bad),
                                         _stream(stream)))


# ---- the sequence encoder's operators ---------------------------------------------------------------------------
# These are called once per layer and step on small arrays as well, where the host's time counts: plain integers go
# to ctypes for the pointers, and what depends on the sizes alone (workspace bytes, the attention description) is
# kept per set of sizes.


def _at(t):
    return None if t is None else t.data_ptr()


def raw_stream(device: int) -> int:
    """The current stream of the device, as its handle (without the Stream object around it: 0.1 us, not 2.8)."""
    return torch._C._cuda_getCurrentRawStream(device)


def _raw_stream(stream):
    if stream is None:
        return raw_stream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype(dtype) -> int:
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise CutBCEError(f"unsupported dtype {dtype}")
    return dt


def embedding_forward(ids, table, scale: float, out, stream=None):
    """cutbce_embedding_forward: ids int32 or int64 [n], table [V, D], out [n, D]."""
    _check(lib().cutbce_embedding_forward(ids.numel(), table.shape[0], table.shape[1], _dtype(table.dtype),
                                          ids.element_size(), _at(ids), _at(table), scale, _at(out),
                                          _raw_stream(stream)))


@functools.lru_cache(maxsize=256)
def embedding_backward_workspace_size(n: int, vocab: int, dim: int, dtype) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().cutbce_embedding_backward_workspace_size(n, vocab, dim, _dtype(dtype), ctypes.byref(b)))
    return int(b.value)


def embedding_backward(ids, dout, scale: float, accumulate: bool, dtable, ws, stream=None):
    """cutbce_embedding_backward: dout [n, D], dtable [V, D] overwritten, or added to where accumulate."""
    _check(lib().cutbce_embedding_backward(ids.numel(), dtable.shape[0], dtable.shape[1], _dtype(dtable.dtype),
                                           ids.element_size(), _at(ids), _at(dout), scale, 1 if accumulate else 0,
                                           _at(dtable), _at(ws), ws.numel(), _raw_stream(stream)))


def layer_norm_forward(x, weight, bias, eps: float, y, mean, rstd, stream=None):
    """cutbce_layer_norm_forward: x [rows, D] (unit column stride); weight, bias [D] or None; mean, rstd float32
    [rows] or None."""
    p = weight if weight is not None else (bias if bias is not None else x)
    _check(lib().cutbce_layer_norm_forward(x.shape[0], x.shape[1], _dtype(x.dtype), _dtype(p.dtype), _at(x),
                                           x.stride(0), _at(weight), _at(bias), eps, _at(y), _at(mean), _at(rstd),
                                           _raw_stream(stream)))


@functools.lru_cache(maxsize=256)
def layer_norm_backward_workspace_size(rows: int, dim: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().cutbce_layer_norm_backward_workspace_size(rows, dim, ctypes.byref(b)))
    return int(b.value)


def layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, ws, stream=None):
    """cutbce_layer_norm_backward: dx, dweight, dbias may be None."""
    p = next((t for t in (weight, dweight, dbias) if t is not None), x)
    _check(lib().cutbce_layer_norm_backward(x.shape[0], x.shape[1], _dtype(x.dtype), _dtype(p.dtype), _at(dy),
                                            dy.stride(0), _at(x), x.stride(0), _at(weight), _at(mean), _at(rstd),
                                            _at(dx), _at(dweight), _at(dbias), _at(ws),
                                            ws.numel() if ws is not None else 0, _raw_stream(stream)))


@functools.lru_cache(maxsize=256)
def attention_problem(*fields):
    """(Attention, bytes of the forward's workspace, bytes of the backward's): fields as in Attention, in order. None
    where one of the two refuses the sizes (its call then does)."""
    a = Attention(*fields)
    b, c = ctypes.c_size_t(0), ctypes.c_size_t(0)
    forward = lib().cutbce_attention_workspace_size(ctypes.byref(a), 0, ctypes.byref(b))
    backward = lib().cutbce_attention_workspace_size(ctypes.byref(a), 1, ctypes.byref(c))
    if forward and backward:
        _check(forward)
    return a, None if forward else int(b.value), None if backward else int(c.value)


def attention_forward(a: Attention, q, k, v, cu_q, cu_k, k_lens, out, lse, ws, stream=None):
    """cutbce_attention_forward: lse float32 [q_rows, q_heads] or None."""
    _check(lib().cutbce_attention_forward(a, _at(q), _at(k), _at(v), _at(cu_q), _at(cu_k), _at(k_lens), _at(out),
                                          _at(lse), _at(ws), ws.numel() if ws is not None else 0,
                                          _raw_stream(stream)))


def attention_backward(a: Attention, dout, q, k, v, out, lse, cu_q, cu_k, k_lens, dq, dk, dv, ws, stream=None):
    """cutbce_attention_backward: dq, dk, dv overwritten."""
    _check(lib().cutbce_attention_backward(a, _at(dout), _at(q), _at(k), _at(v), _at(out), _at(lse), _at(cu_q),
                                           _at(cu_k), _at(k_lens), _at(dq), _at(dk), _at(dv), _at(ws),
                                           ws.numel() if ws is not None else 0, _raw_stream(stream)))


# ---- the training step's operators ------------------------------------------------------------------------------


@functools.lru_cache(maxsize=256)
def cross_entropy_sizes(rows: int, vocab: int, dim: int, dtype):
    """Bytes of `saved`, and of the workspaces: of the forward without it, the forward with it, and the backward."""
    b, found = ctypes.c_size_t(0), []
    _check(lib().cutbce_cross_entropy_saved_size(rows, vocab, dim, _dtype(dtype), ctypes.byref(b)))
    found.append(int(b.value))
    for which in range(3):
        _check(lib().cutbce_cross_entropy_workspace_size(rows, vocab, dim, _dtype(dtype), which, ctypes.byref(b)))
        found.append(int(b.value))
    return tuple(found)


def cross_entropy_forward(H, E, targets, row_weight, scale: float, loss, row_loss, saved, ws, stream=None):
    """cutbce_cross_entropy_forward: row_weight, row_loss and saved may be None."""
    _check(lib().cutbce_cross_entropy_forward(H.shape[0], E.shape[0], E.shape[1], _dtype(E.dtype),
                                              targets.element_size(), _at(H), _at(E), _at(targets), _at(row_weight),
                                              scale, _at(loss), _at(row_loss), _at(saved), _at(ws), ws.numel(),
                                              _raw_stream(stream)))


def cross_entropy_backward(rows: int, E, scale: float, grad, saved, dH, dE, ws, stream=None):
    """cutbce_cross_entropy_backward: dH, dE overwritten, either may be None."""
    _check(lib().cutbce_cross_entropy_backward(rows, E.shape[0], E.shape[1], _dtype(E.dtype), _at(E), scale, _at(grad),
                                               _at(saved), _at(dH), _at(dE), _at(ws), ws.numel(),
                                               _raw_stream(stream)))


@functools.lru_cache(maxsize=256)
def grad_norm_workspace_size(sizes: tuple) -> int:
    n = array.array("q", sizes)
    b = ctypes.c_size_t(0)
    _check(lib().cutbce_grad_norm_workspace_size(len(n), n.buffer_info()[0], ctypes.byref(b)))
    return int(b.value)


def grad_norm(pointers, sizes: tuple, dtypes, norm, ws, stream=None):
    """cutbce_grad_norm: the tensors' addresses, elements and dtypes; norm float32 [1]."""
    at = array.array("Q", pointers)
    n = array.array("q", sizes)
    types = array.array("i", dtypes)
    _check(lib().cutbce_grad_norm(len(n), at.buffer_info()[0], n.buffer_info()[0], types.buffer_info()[0], _at(norm),
                                  _at(ws), ws.numel(), _raw_stream(stream)))


def adamw_step(n, pointers, types, decay, how: AdamW, stream=None):
    """cutbce_adamw_step: pointers the seven lists of addresses (param, grad, exp_avg, exp_avg_sq, their scales, master;
    None for a list that is not there), types the parameters' and gradients' dtypes."""
    arrays = [None if p is None else array.array("Q", p) for p in pointers]
    arrays += [array.array("q", n), array.array("i", types[0]), array.array("i", types[1]), array.array("f", decay)]
    x = AdamWTensors(len(n), 0, *[None if a is None else a.buffer_info()[0] for a in arrays])
    _check(lib().cutbce_adamw_step(ctypes.byref(x), ctypes.byref(how), _raw_stream(stream)))


SWEEP_KINDS = ("rows_sweep", "items_sweep", "topk_sweep")


def profile_enable(on: bool = True):
    """Start (or stop) event timing of the sweep kernels inside the library."""
    _check(lib().cutbce_profile_enable(1 if on else 0))


def profile_read() -> dict:
    """{kind: (total_ms, launches)} since the last enable/read; waits for the recorded events."""
    n = len(SWEEP_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(lib().cutbce_profile_read(ms, cnt, n))
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(SWEEP_KINDS)}


def mfma_ceiling(blocks: int, waves_per_block: int, iters: int, stamps, stream=None):
    """Enqueue the MFMA-only ceiling kernel; stamps: int64 device tensor of 4 * blocks * waves_per_block."""
    _check(lib().cutbce_mfma_ceiling(blocks, waves_per_block, iters, _ptr(stamps), _stream(stream)))


def mfma_ceiling_random(blocks: int, waves_per_block: int, iters: int, stamps, stream=None):
    """Enqueue the MFMA-only ceiling kernel on random operands that change from one MFMA to the next."""
    _check(lib().cutbce_mfma_ceiling_random(blocks, waves_per_block, iters, _ptr(stamps), _stream(stream)))
