"""PyTorch front end of the sequence encoder's operators: what turns item ids into the hidden states that ``cut_bce``
takes. Each is differentiable in reverse mode (``embedding``, ``layer_norm``, ``packed_attention``; forward-mode
tangents and second derivatives are refused) and also has explicit forward and backward calls for callers that keep
their own tape; ``cached_attention`` serves single tokens against a key/value cache. The arithmetic is libcutbce.so's;
PyTorch allocates outputs and workspaces and supplies the stream.

All tensors live on the current GPU, float32 or bfloat16. Lengths and offsets stay on the device: no call
synchronises with the host.
"""
from __future__ import annotations

import functools
import math

import torch
from torch.autograd import forward_ad

from . import binding as B

_FLOATS = (torch.float32, torch.bfloat16)

# These calls are made once per layer and step, on small arrays as well, where the host's time is what they take: the
# checks below are written for few Python operations.


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on_gpu(what, first, *others):
    """The device that every tensor given is on: the current one."""
    dev = first.get_device()
    if dev >= 0 and dev == torch._C._cuda_getDevice():
        for t in others:
            if t is not None and t.get_device() != dev:
                break
        else:
            return dev
    raise ValueError(f"{what} runs on the GPU only: its tensors must be on the current device")


def _derived(*tensors):
    """Whether a derivative is taken of any of these: the call then goes through its autograd function, which refuses
    the forward mode (a direct call would return an output without a tangent)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    if forward_ad._current_level >= 0:
        return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)
    return False


class _NoSecond(torch.autograd.Function):
    """Gradients as they are; differentiating them raises."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("this operator has first derivatives only: its gradients cannot be differentiated")


def _first_order(backward):
    """Backward of an operator without second derivatives. The kernels' outputs have no graph, so under create_graph
    they get one that raises: without it a term that is made of them would be left out of a sum. (once_differentiable
    does so only where the cotangent has a graph itself, which that of a plain sum has not.)"""

    @functools.wraps(backward)
    def wrapped(ctx, *cotangents):
        graph = torch.is_grad_enabled()
        with torch.no_grad():
            grads = list(backward(ctx, *cotangents))
        if graph:
            at = [i for i, g in enumerate(grads) if g is not None]
            for i, g in zip(at, _NoSecond.apply(torch.empty(0, requires_grad=True), *[grads[i] for i in at])):
                grads[i] = g
        return tuple(grads)

    return wrapped


# ---- embedding lookup -----------------------------------------------------------------------------------------


def _ids(ids):
    _need(ids.dtype in (torch.int32, torch.int64), "ids must be int32 or int64")
    return ids.contiguous()


def _aligned(t):
    """t itself where its data start at a multiple of 16 bytes, else a copy that does."""
    return t.clone() if t.data_ptr() & 15 else t


def embedding_forward(ids, table, scale: float = 1.0):
    """out[..., :] = scale * table[ids[...]], zeros where an id is outside [0, V) (padding, e.g. -1)."""
    dev = _on_gpu("embedding", ids, table)
    _need(table.dtype in _FLOATS and table.dim() == 2, "table must be float32 or bfloat16 [V, D]")
    _need(math.isfinite(scale), "scale must be finite")
    ids, table = _ids(ids), _aligned(table.contiguous())
    out = table.new_empty(ids.shape + table.shape[1:])
    B.embedding_forward(ids, table, scale, out, B.raw_stream(dev))
    return out


def embedding_backward(dout, ids, vocab: int, scale: float = 1.0, dtable=None):
    """Gradient of the lookup with respect to the table [vocab, D]: scale * the sum of dout over the positions of each
    item, in float32, in an order that depends on the ids alone, rounded once.

    With `dtable` (contiguous [vocab, D] of dout's dtype) the sums are added to it in place and only the rows of the
    looked-up items are touched: for a table shared with the loss, pass the dE that the loss returned. Returns the
    gradient."""
    dev = _on_gpu("embedding_backward", dout, ids, dtable)
    _need(dout.dtype in _FLOATS and dout.shape[:-1] == ids.shape, "dout must be float32 or bfloat16 [*ids.shape, D]")
    _need(math.isfinite(scale), "scale must be finite")
    ids, dout = _ids(ids), _aligned(dout.contiguous())
    D = dout.shape[-1]
    accumulate = dtable is not None
    if accumulate:
        _need(dtable.shape == (vocab, D) and dtable.dtype == dout.dtype and dtable.is_contiguous(),
              "dtable must be a contiguous [vocab, D] of dout's dtype")
    else:
        dtable = dout.new_empty((vocab, D))
    ws = dout.new_empty(B.embedding_backward_workspace_size(ids.numel(), vocab, D, dout.dtype), dtype=torch.uint8)
    B.embedding_backward(ids, dout, scale, accumulate, dtable, ws, B.raw_stream(dev))
    if accumulate and not dtable.is_inference():
        torch.autograd.graph.increment_version(dtable)
    return dtable


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return embedding_forward(ids, table, scale)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return None, embedding_backward(dout, ids, ctx.vocab, ctx.scale), None


def embedding(ids, table, scale: float = 1.0):
    """Rows of an item table: scale * table[ids] (ids int32 or int64 of any shape; an id outside [0, V) gives zeros
    and no gradient). table [V, D] float32 or bfloat16; the gradient flows to the table as a dense [V, D]."""
    if _derived(table):
        return _Embedding.apply(ids, table, scale)
    return embedding_forward(ids, table, scale)


# ---- layer norm -----------------------------------------------------------------------------------------------


def _rows(x):
    """x [..., D] as rows [R, D] with unit column stride and rows that do not overlap (copied where they are not)."""
    D = x.shape[-1]
    if x.dim() != 2:
        x = x.reshape(-1, D)
    if x.is_contiguous() and x.stride(0) == D:
        return x
    if (D > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < D):
        return x.contiguous()
    if x.stride(0) < D:  # a single row
        x = x.as_strided(x.shape, (D, 1))
    return x


def _norm_param(p, D):
    if p is None:
        return None
    if p.dtype not in _FLOATS or p.shape != (D,):
        raise ValueError("weight and bias must be float32 or bfloat16 [D]")
    return p.contiguous()


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = True):
    """(y, mean, rstd) of layer norm over the last dimension of x [..., D]; mean and rstd float32 [rows], or None
    with stats=False."""
    dev = _on_gpu("layer_norm", x, weight, bias)
    if x.dtype not in _FLOATS or x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be float32 or bfloat16 [..., D]")
    if not 0 <= eps < math.inf:
        raise ValueError("eps must be finite and >= 0")
    D = x.shape[-1]
    weight, bias = _norm_param(weight, D), _norm_param(bias, D)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    rows = _rows(x)
    y = torch.empty_like(rows) if rows is x else x.new_empty(x.shape)
    mean = rstd = None
    if stats:
        mean = x.new_empty(rows.shape[0], dtype=torch.float32)
        rstd = torch.empty_like(mean)
    B.layer_norm_forward(rows, weight, bias, eps, y, mean, rstd, B.raw_stream(dev))
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, want_dx: bool = True, want_dweight: bool = True,
                        want_dbias: bool = True, param_dtype=None):
    """(dx, dweight, dbias) from the cotangent dy, the forward's x, weight (or None) and its mean and rstd; dweight
    and dbias in weight's dtype (without a weight in param_dtype, x's by default). What is not wanted is None."""
    dev = _on_gpu("layer_norm_backward", dy, x, weight, mean, rstd)
    if dy.shape != x.shape or dy.dtype != x.dtype or x.dtype not in _FLOATS:
        raise ValueError("dy must have x's shape and dtype")
    D = x.shape[-1]
    weight = _norm_param(weight, D)
    rx, rdy = _rows(x), _rows(dy)
    n = rx.shape[:1]
    if not (mean.shape == n and rstd.shape == n and mean.dtype == rstd.dtype == torch.float32 and
            mean.is_contiguous() and rstd.is_contiguous()):
        raise ValueError("mean and rstd must be the forward's float32 [rows]")
    pd = weight.dtype if weight is not None else x.dtype if param_dtype is None else param_dtype
    if pd not in _FLOATS or param_dtype not in (None, pd):
        raise ValueError("param_dtype must be float32 or bfloat16, and weight's where there is one")
    dx = x.new_empty(x.shape) if want_dx else None
    dw = x.new_empty(D, dtype=pd) if want_dweight else None
    db = None
    if want_dbias:
        db = torch.empty_like(dw) if want_dweight else x.new_empty(D, dtype=pd)
    ws = None
    if want_dweight or want_dbias:
        ws = x.new_empty(B.layer_norm_backward_workspace_size(n[0], D), dtype=torch.uint8)
    B.layer_norm_backward(rdy, rx, weight, mean, rstd, dx, dw, db, ws, B.raw_stream(dev))
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        return layer_norm_backward(dy, x, weight, mean, rstd, need[0], need[1], need[2], ctx.bias_dtype) + (None,)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension of x [..., D]: (x - mean) / sqrt(var + eps) * weight + bias, statistics in
    float32. weight and bias [D] (float32 or bfloat16, one dtype for both) may be None. Gradients flow to all three."""
    if _derived(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, eps)
    return layer_norm_forward(x, weight, bias, eps, stats=False)[0]


# ---- attention ------------------------------------------------------------------------------------------------


def _strided(x):
    """x [.., rows, heads, head_dim], and the strides of its rows and heads as the kernels take them: unit stride of the
    last dimension, 16-byte steps; a contiguous copy where x is not laid out so. A dimension of size 1 steps by 0."""
    mask = 16 // x.element_size() - 1
    for _ in range(2):
        st, size = x.stride(), x.shape
        rs = st[-3] if size[-3] > 1 else 0
        hs = st[-2] if size[-2] > 1 else 0
        ss = st[0] if len(st) == 4 and size[0] > 1 else 0
        if st[-1] == 1 and not (rs | hs | ss) & mask and not x.data_ptr() & 15 and rs <= 1 << 22:
            return x, rs, hs, ss
        x = x.contiguous()
        if x.data_ptr() & 15:
            x = x.clone()
    raise ValueError("head_dim must be a multiple of 8, and heads * head_dim at most 2**22")


def _offsets(cu, n, name):
    if cu is None:
        return None
    if cu.shape != (n,):
        raise ValueError(f"{name} must have {n} entries on the device")
    if cu.dtype != torch.int32 and cu.dtype != torch.int64:
        raise ValueError(f"{name} must be int32 or int64")
    return cu if cu.dtype == torch.int32 and cu.is_contiguous() else cu.to(torch.int32).contiguous()


def _attention(q, k, v, seqs, causal, scale):
    """Checked q [rows, heads, head_dim] and k, v [(sequences,) rows, kv heads, head_dim] as the kernels take them, and
    the problem with its workspace sizes."""
    dt = q.dtype
    if dt not in _FLOATS or k.dtype != dt or v.dtype != dt:
        raise ValueError("q, k and v must all be float32 or all bfloat16")
    q_rows, hq, dh = q.shape
    hk = k.shape[-2]
    if k.shape != v.shape or k.shape[-1] != dh:
        raise ValueError("k and v must have one shape, and q's head_dim")
    if hk < 1 or hq < 1 or hq % hk:
        raise ValueError("the query heads must be a multiple of the key/value heads")
    if dh & 7 or not 8 <= dh <= 128:
        raise ValueError("head_dim must be a multiple of 8, at most 128")
    scale = dh ** -0.5 if scale is None else float(scale)
    _need(math.isfinite(scale), "scale must be finite")
    q, q_rs, q_hs, _ = _strided(q)
    k, k_rs, k_hs, k_ss = _strided(k)
    v, v_rs, v_hs, v_ss = _strided(v)
    k_rows = k.shape[0] if k.dim() == 3 else k.shape[0] * k.shape[1]
    return q, k, v, B.attention_problem(q_rows, k_rows, q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, k_ss, v_ss, seqs, hq, hk,
                                        dh, B._DTYPES[dt], 1 if causal else 0, scale)


def _packed(q, k, v, cu_q, cu_k, k_lens, causal, scale):
    dev = _on_gpu("packed_attention", q, k, v, cu_q, cu_k, k_lens)
    _need(q.dim() == 3 and k.dim() == 3, "q must be [rows, heads, head_dim] and k, v [rows, kv heads, head_dim]")
    _need(cu_q.dim() == 1 and cu_q.numel() >= 2, "cu_q must be [sequences + 1]")
    n = cu_q.numel()
    cu_q = _offsets(cu_q, n, "cu_q")
    cu_k = _offsets(cu_k, n, "cu_k")
    k_lens = _offsets(k_lens, n - 1, "k_lens")
    if cu_k is None:
        _need(k.shape[0] == q.shape[0], "k must have q's rows where there is no cu_k")
        if k_lens is not None:
            cu_k = cu_q
    return (dev, cu_q, cu_k, k_lens) + _attention(q, k, v, n - 1, causal, scale)


def _scratch(size, like):
    return like.new_empty(size, dtype=torch.uint8) if size else None


def packed_attention_forward(q, k, v, cu_q, cu_k=None, k_lens=None, causal: bool = True, scale=None,
                             want_lse: bool = True):
    """(out, lse) of packed_attention: out [rows, heads, head_dim]; lse float32 [rows, heads], the log of each row's
    sum of exponentials (-inf where a row sees no key), or None."""
    dev, cu_q, cu_k, k_lens, q, k, v, (a, size, _) = _packed(q, k, v, cu_q, cu_k, k_lens, causal, scale)
    out = q.new_empty(q.shape)
    lse = q.new_empty(q.shape[:2], dtype=torch.float32) if want_lse else None
    B.attention_forward(a, q, k, v, cu_q, cu_k, k_lens, out, lse, _scratch(size, q), B.raw_stream(dev))
    return out, lse


def packed_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k=None, k_lens=None, causal: bool = True, scale=None):
    """(dq, dk, dv) from the cotangent dout, the forward's inputs, and its out and lse."""
    dev, cu_q, cu_k, k_lens, q, k, v, (a, _, size) = _packed(q, k, v, cu_q, cu_k, k_lens, causal, scale)
    _on_gpu("packed_attention_backward", dout, out, lse)
    if dout.shape != q.shape or dout.dtype != q.dtype:
        raise ValueError("dout must have q's shape and dtype")
    if (out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or lse.shape != q.shape[:2] or
            lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("out and lse must be the forward's")
    dout = _aligned(dout.contiguous())
    dq = torch.empty_like(dout)
    dk = q.new_empty(k.shape)
    dv = torch.empty_like(dk)
    B.attention_backward(a, dout, q, k, v, out, lse, cu_q, cu_k, k_lens, dq, dk, dv, _scratch(size, q),
                         B.raw_stream(dev))
    return dq, dk, dv


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, k_lens, causal, scale):
        out, lse = packed_attention_forward(q, k, v, cu_q, cu_k, k_lens, causal, scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_q, cu_k, k_lens)
        ctx.how = (causal, scale)
        return out

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        q, k, v, out, lse, cu_q, cu_k, k_lens = ctx.saved_tensors
        return packed_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, k_lens, *ctx.how) + (None,) * 5


def packed_attention(q, k, v, cu_q, cu_k=None, k_lens=None, causal: bool = True, scale=None):
    """Softmax attention within each sequence of a packed batch, without padding.

    q [rows, heads, head_dim]; k, v [key rows, kv heads, head_dim] (heads a multiple of kv heads; query head h reads
    key/value head h // (heads // kv heads)); float32 or bfloat16, head_dim a multiple of 8 up to 128. They may be
    column ranges of one projection: rows and heads may be strided. Sequence b has the rows cu_q[b]:cu_q[b+1] and the
    keys cu_k[b]:cu_k[b+1] (cu_k None: cu_q); with k_lens only the first k_lens[b] of them are keys. causal: row t of
    n sees the keys j <= t + m - n of m, so that the last row sees all of them; a row that sees none gives zeros.
    scale: 1 / sqrt(head_dim) by default. cu_q, cu_k and k_lens are int32 (int64 is converted) on the device.
    Gradients flow to q, k, v. Non-finite values in k, v or the cotangent may reach every row of their own sequence and
    head, and no other."""
    if _derived(q, k, v):
        return _PackedAttention.apply(q, k, v, cu_q, cu_k, k_lens, causal, scale)
    return packed_attention_forward(q, k, v, cu_q, cu_k, k_lens, causal, scale, want_lse=False)[0]


def cached_attention(q, k_cache, v_cache, lens, causal: bool = True, scale=None):
    """Attention of the newest tokens over a key/value cache (serving; no gradient).

    q [sequences, heads, head_dim] (one token each) or [sequences, tokens, heads, head_dim]; k_cache, v_cache
    [sequences, capacity, kv heads, head_dim] in any strides whose last is 1 (a view of [sequences, kv heads,
    capacity, head_dim] as well); lens [sequences] on the device: the first lens[b] rows are filled, the newest tokens'
    own keys included, and the rest is never used. Returns q's shape."""
    dev = _on_gpu("cached_attention", q, k_cache, v_cache, lens)
    if _derived(q, k_cache, v_cache):
        raise ValueError("cached_attention has no gradient: use packed_attention, or torch.no_grad()")
    q = q.contiguous()
    seqs = k_cache.shape[0]
    _need(q.dim() in (3, 4) and k_cache.dim() == 4 and seqs == q.shape[0],
          "q must be [sequences, (tokens,) heads, head_dim] and the caches [sequences, capacity, kv heads, head_dim]")
    lens = _offsets(lens, seqs, "lens")
    out = torch.empty_like(q)
    if seqs == 0:
        return out
    rows = q if q.dim() == 3 else q.view(-1, *q.shape[2:])
    rows, k, v, (a, size, _) = _attention(rows, k_cache, v_cache, seqs, causal, scale)
    B.attention_forward(a, rows, k, v, None, None, lens, out, None, _scratch(size, q), B.raw_stream(dev))
    return out
