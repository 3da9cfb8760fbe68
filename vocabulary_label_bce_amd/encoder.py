"""PyTorch front end of the sequence encoder's operators: what turns item ids into the hidden states that ``cut_bce``
takes. Each is differentiable (``embedding``, ``layer_norm``, ``packed_attention``) and also has explicit forward and
backward calls for callers that keep their own tape; ``cached_attention`` serves single tokens against a key/value
cache. The arithmetic is libcutbce.so's; PyTorch allocates outputs and workspaces and supplies the stream.

All tensors live on the current GPU, float32 or bfloat16. Lengths and offsets stay on the device: no call
synchronises with the host.
"""
from __future__ import annotations

import math

import torch

from . import binding as B

_FLOATS = (torch.float32, torch.bfloat16)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on_gpu(what, *tensors):
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None and t.is_cuda:
            dev = torch.cuda.current_device()
        if t.get_device() != dev:
            raise ValueError(f"{what} runs on the GPU only: its tensors must be on the current device")


# ---- embedding lookup -----------------------------------------------------------------------------------------


def _ids(ids):
    _need(ids.dtype in (torch.int32, torch.int64), "ids must be int32 or int64")
    return ids.contiguous()


def _aligned(t):
    """t itself where its data start at a multiple of 16 bytes, else a copy that does."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def embedding_forward(ids, table, scale: float = 1.0):
    """out[..., :] = scale * table[ids[...]], zeros where an id is outside [0, V) (padding, e.g. -1)."""
    _on_gpu("embedding", ids, table)
    _need(table.dtype in _FLOATS and table.dim() == 2, "table must be float32 or bfloat16 [V, D]")
    _need(math.isfinite(scale), "scale must be finite")
    ids, table = _ids(ids), _aligned(table.contiguous())
    out = torch.empty(ids.shape + table.shape[1:], dtype=table.dtype, device=table.device)
    B.embedding_forward(ids, table, scale, out)
    return out


def embedding_backward(dout, ids, vocab: int, scale: float = 1.0, dtable=None):
    """Gradient of the lookup with respect to the table [vocab, D]: scale * the sum of dout over the positions of each
    item, in float32, in an order that depends on the ids alone, rounded once.

    With `dtable` (contiguous [vocab, D] of dout's dtype) the sums are added to it in place and only the rows of the
    looked-up items are touched: for a table shared with the loss, pass the dE that the loss returned. Returns the
    gradient."""
    _on_gpu("embedding_backward", dout, ids, dtable)
    _need(dout.dtype in _FLOATS and dout.shape[:-1] == ids.shape, "dout must be float32 or bfloat16 [*ids.shape, D]")
    _need(math.isfinite(scale), "scale must be finite")
    ids, dout = _ids(ids), _aligned(dout.contiguous())
    D = dout.shape[-1]
    accumulate = dtable is not None
    if accumulate:
        _need(dtable.shape == (vocab, D) and dtable.dtype == dout.dtype and dtable.is_contiguous(),
              "dtable must be a contiguous [vocab, D] of dout's dtype")
    else:
        dtable = torch.empty(vocab, D, dtype=dout.dtype, device=dout.device)
    ws = torch.empty(B.embedding_backward_workspace_size(ids.numel(), vocab, D, dout.dtype), dtype=torch.uint8,
                     device=dout.device)
    B.embedding_backward(ids, dout, scale, accumulate, dtable, ws)
    return dtable


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return embedding_forward(ids, table, scale)

    @staticmethod
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return None, embedding_backward(dout, ids, ctx.vocab, ctx.scale), None


def embedding(ids, table, scale: float = 1.0):
    """Rows of an item table: scale * table[ids] (ids int32 or int64 of any shape; an id outside [0, V) gives zeros
    and no gradient). table [V, D] float32 or bfloat16; the gradient flows to the table as a dense [V, D]."""
    if torch.is_grad_enabled() and table.requires_grad:
        return _Embedding.apply(ids, table, scale)
    return embedding_forward(ids, table, scale)


# ---- layer norm -----------------------------------------------------------------------------------------------


def _rows(x):
    """x [..., D] as rows [R, D] with unit column stride and rows that do not overlap (copied where they are not)."""
    D = x.shape[-1]
    if x.dim() != 2:
        x = x.reshape(-1, D)
    if (D > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < D):
        return x.contiguous()
    if x.stride(0) < D:  # a single row
        x = x.as_strided(x.shape, (D, 1))
    return x


def _norm_params(x, weight, bias):
    D = x.shape[-1]
    for p in (weight, bias):
        _need(p is None or (p.dtype in _FLOATS and p.shape == (D,)), "weight and bias must be float32 or bfloat16 [D]")
    _need(weight is None or bias is None or weight.dtype == bias.dtype, "weight and bias must have one dtype")


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = True):
    """(y, mean, rstd) of layer norm over the last dimension of x [..., D]; mean and rstd float32 [rows], or None
    with stats=False."""
    _on_gpu("layer_norm", x, weight, bias)
    _need(x.dtype in _FLOATS and x.dim() >= 1 and x.shape[-1] >= 1, "x must be float32 or bfloat16 [..., D]")
    _need(0 <= eps < math.inf, "eps must be finite and >= 0")
    _norm_params(x, weight, bias)
    rows = _rows(x)
    weight = None if weight is None else weight.contiguous()
    bias = None if bias is None else bias.contiguous()
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    mean = rstd = None
    if stats:
        mean = torch.empty(rows.shape[0], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    B.layer_norm_forward(rows, weight, bias, eps, y, mean, rstd)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, want_dx: bool = True, want_dweight: bool = True,
                        want_dbias: bool = True):
    """(dx, dweight, dbias) from the cotangent dy, the forward's x, weight (or None) and its mean and rstd; dweight
    and dbias in weight's dtype (x's without a weight). What is not wanted is None."""
    _on_gpu("layer_norm_backward", dy, x, weight, mean, rstd)
    _need(dy.shape == x.shape and dy.dtype == x.dtype and x.dtype in _FLOATS, "dy must have x's shape and dtype")
    _norm_params(x, weight, None)
    D = x.shape[-1]
    rx, rdy = _rows(x), _rows(dy)
    for t in (mean, rstd):
        _need(t.dtype == torch.float32 and t.is_contiguous() and t.numel() == rx.shape[0],
              "mean and rstd must be the forward's float32 [rows]")
    weight = None if weight is None else weight.contiguous()
    pd = x.dtype if weight is None else weight.dtype
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if want_dx else None
    dw = torch.empty(D, dtype=pd, device=x.device) if want_dweight else None
    db = torch.empty(D, dtype=pd, device=x.device) if want_dbias else None
    ws = None
    if want_dweight or want_dbias:
        ws = torch.empty(B.layer_norm_backward_workspace_size(rx.shape[0], D), dtype=torch.uint8, device=x.device)
    B.layer_norm_backward(rdy, rx, weight, mean, rstd, dx, dw, db, ws)
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd, need[0], need[1], need[2])
        return dx, dw, None if db is None else db.to(ctx.bias_dtype), None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension of x [..., D]: (x - mean) / sqrt(var + eps) * weight + bias, statistics in
    float32. weight and bias [D] (float32 or bfloat16, one dtype for both) may be None. Gradients flow to all three."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias)):
        return _LayerNorm.apply(x, weight, bias, eps)
    return layer_norm_forward(x, weight, bias, eps, stats=False)[0]


# ---- attention ------------------------------------------------------------------------------------------------


def _strided(x, dims):
    """x, and the strides of `dims`, as the kernels take them: unit stride of the last dimension, 16-byte steps; a
    contiguous copy where x is not laid out so. A dimension of size 1 steps by 0."""
    step = 16 // x.element_size()
    for _ in range(2):
        st = [x.stride(d) if x.shape[d] > 1 else 0 for d in dims]
        if x.stride(-1) == 1 and x.data_ptr() % 16 == 0 and all(s % step == 0 for s in st) and st[-2] <= 1 << 22:
            return x, st
        x = x.contiguous()
        if x.data_ptr() % 16:
            x = x.clone()
    raise ValueError("head_dim must be a multiple of 8")


def _offsets(cu, n, name, dev):
    if cu is None:
        return None
    _need(cu.dim() == 1 and cu.numel() == n and cu.device == dev, f"{name} must have {n} entries on the device")
    return cu.to(torch.int32).contiguous()


def _attention(q, k, v, cu_q, cu_k, k_lens, causal, scale, cached):
    """Checked arguments, the problem with its workspace sizes, and the tensors as the kernels take them."""
    _need(q.dtype in _FLOATS and q.dtype == k.dtype == v.dtype, "q, k and v must all be float32 or all bfloat16")
    dh, hq, hk = q.shape[-1], q.shape[-2], k.shape[-2]
    _need(k.shape == v.shape and k.shape[-1] == dh, "k and v must have one shape, and q's head_dim")
    _need(hk > 0 and hq > 0 and hq % hk == 0, "the query heads must be a multiple of the key/value heads")
    _need(dh % 8 == 0 and 8 <= dh <= 128, "head_dim must be a multiple of 8, at most 128")
    scale = 1.0 / math.sqrt(dh) if scale is None else float(scale)
    _need(math.isfinite(scale), "scale must be finite")
    q, (q_rs, q_hs) = _strided(q, (0, 1))
    q_rows = q.shape[0]
    if cached:
        seqs, k_rows = k.shape[0], k.shape[0] * k.shape[1]
        k, (k_ss, k_rs, k_hs) = _strided(k, (0, 1, 2))
        v, (v_ss, v_rs, v_hs) = _strided(v, (0, 1, 2))
    else:
        seqs, k_rows, k_ss, v_ss = cu_q.numel() - 1, k.shape[0], 0, 0
        k, (k_rs, k_hs) = _strided(k, (0, 1))
        v, (v_rs, v_hs) = _strided(v, (0, 1))
    p = B.attention_problem(q_rows, k_rows, q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, k_ss, v_ss, seqs, hq, hk, dh,
                            B._dtype(q.dtype), 1 if causal else 0, scale)
    return q, k, v, p


def _packed(q, k, v, cu_q, cu_k, k_lens, causal, scale):
    _on_gpu("packed_attention", q, k, v, cu_q, cu_k, k_lens)
    _need(q.dim() == 3 and k.dim() == 3, "q must be [rows, heads, head_dim] and k, v [rows, kv heads, head_dim]")
    _need(cu_q.dim() == 1 and cu_q.numel() >= 2, "cu_q must be [sequences + 1]")
    n = cu_q.numel()
    cu_q = _offsets(cu_q, n, "cu_q", q.device)
    cu_k = _offsets(cu_k, n, "cu_k", q.device)
    k_lens = _offsets(k_lens, n - 1, "k_lens", q.device)
    if cu_k is None:
        _need(k.shape[0] == q.shape[0], "k must have q's rows where there is no cu_k")
        if k_lens is not None:
            cu_k = cu_q
    return (cu_q, cu_k, k_lens) + _attention(q, k, v, cu_q, cu_k, k_lens, causal, scale, False)


def _scratch(size, dev):
    return torch.empty(size, dtype=torch.uint8, device=dev) if size else None


def packed_attention_forward(q, k, v, cu_q, cu_k=None, k_lens=None, causal: bool = True, scale=None,
                             want_lse: bool = True):
    """(out, lse) of packed_attention: out [rows, heads, head_dim]; lse float32 [rows, heads], the log of each row's
    sum of exponentials (-inf where a row sees no key), or None."""
    cu_q, cu_k, k_lens, q, k, v, (a, size, _) = _packed(q, k, v, cu_q, cu_k, k_lens, causal, scale)
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if want_lse else None
    B.attention_forward(a, q, k, v, cu_q, cu_k, k_lens, out, lse, _scratch(size, q.device))
    return out, lse


def packed_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k=None, k_lens=None, causal: bool = True, scale=None):
    """(dq, dk, dv) from the cotangent dout, the forward's inputs, and its out and lse."""
    cu_q, cu_k, k_lens, q, k, v, (a, _, size) = _packed(q, k, v, cu_q, cu_k, k_lens, causal, scale)
    _on_gpu("packed_attention_backward", dout, out, lse)
    _need(dout.shape == q.shape and dout.dtype == q.dtype, "dout must have q's shape and dtype")
    _need(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous() and lse.shape == q.shape[:2] and
          lse.dtype == torch.float32 and lse.is_contiguous(), "out and lse must be the forward's")
    dout = _aligned(dout.contiguous())
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    dv = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    B.attention_backward(a, dout, q, k, v, out, lse, cu_q, cu_k, k_lens, dq, dk, dv, _scratch(size, q.device))
    return dq, dk, dv


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, k_lens, causal, scale):
        out, lse = packed_attention_forward(q, k, v, cu_q, cu_k, k_lens, causal, scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_q, cu_k, k_lens)
        ctx.how = (causal, scale)
        return out

    @staticmethod
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
    scale: 1 / sqrt(head_dim) by default. cu_q, cu_k and k_lens are int32 on the device. Gradients flow to q, k, v.
    Non-finite values in k, v or the cotangent may reach every row of their own sequence and head, and no other."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v)):
        return _PackedAttention.apply(q, k, v, cu_q, cu_k, k_lens, causal, scale)
    return packed_attention_forward(q, k, v, cu_q, cu_k, k_lens, causal, scale, want_lse=False)[0]


def cached_attention(q, k_cache, v_cache, lens, causal: bool = True, scale=None):
    """Attention of the newest tokens over a key/value cache (serving; no gradient).

    q [sequences, heads, head_dim] (one token each) or [sequences, tokens, heads, head_dim]; k_cache, v_cache
    [sequences, capacity, kv heads, head_dim] in any strides whose last is 1 (a view of [sequences, kv heads,
    capacity, head_dim] as well); lens [sequences] on the device: the first lens[b] rows are filled, the newest tokens'
    own keys included, and the rest is never used. Returns q's shape."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in (q, k_cache, v_cache)):
        raise ValueError("cached_attention has no gradient: use packed_attention, or torch.no_grad()")
    _on_gpu("cached_attention", q, k_cache, v_cache, lens)
    shape = q.shape
    if q.dim() == 3:
        q = q.unsqueeze(1)
    _need(q.dim() == 4 and k_cache.dim() == 4 and k_cache.shape[0] == q.shape[0],
          "q must be [sequences, (tokens,) heads, head_dim] and the caches [sequences, capacity, kv heads, head_dim]")
    lens = _offsets(lens, k_cache.shape[0], "lens", q.device)
    q = q.contiguous().view(-1, *q.shape[2:])
    out = torch.empty(shape, dtype=q.dtype, device=q.device)
    if k_cache.shape[0] == 0:
        return out
    q, k, v, (a, size, _) = _attention(q, k_cache, v_cache, None, None, lens, causal, scale, True)
    B.attention_forward(a, q, k, v, None, None, lens, out, None, _scratch(size, q.device))
    return out
