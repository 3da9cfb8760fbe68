"""PyTorch front end of the training step's last part: the norm of all gradients and the AdamW step, each over a list of
tensors in few launches. The arithmetic is libcutbce.so's. All tensors live on the current GPU; nothing synchronises
with the host, and the steps are counted on the device, so that a captured step advances when it is replayed.
"""
from __future__ import annotations

import math
import operator

import torch

from . import binding as B
from .encoder import _FLOATS, _need


# These calls are made on hundreds of small tensors as well, where the host's time is what they take: lists are looked
# at by map over methods, one property at a time.
_ptr, _numel, _contiguous = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous
_device, _dtype = torch.Tensor.get_device, operator.attrgetter("dtype")
_FLOAT_SET, _F32_SET, _F8_SET = set(_FLOATS), {torch.float32}, {torch.float8_e4m3fn}


def _here(what, *lists):
    """The current device, which all tensors must be on."""
    dev = torch._C._cuda_getDevice()
    for ts in lists:
        if any(d != dev for d in set(map(_device, ts))):
            raise ValueError(f"{what} runs on the GPU only: its tensors must be on the current device")
    return dev


def _dense(what, tensors, dtypes):
    if not set(map(_dtype, tensors)) <= dtypes:
        raise ValueError(f"{what} must be {' or '.join(str(d)[6:] for d in dtypes)}")
    if not all(map(_contiguous, tensors)):
        raise ValueError(f"{what} must be contiguous")


def grad_norm(grads):
    """The 2-norm over all elements of a list of tensors (float32 or bfloat16, also mixed): float32 [1] on the device,
    its squares summed in float64. An empty list has the norm 0."""
    grads = list(grads)
    if not grads:
        return torch.zeros(1, dtype=torch.float32, device=torch.device("cuda", torch.cuda.current_device()))
    dev = _here("grad_norm", grads)
    types = list(map(_dtype, grads))
    if not set(types) <= _FLOAT_SET:
        raise ValueError("gradients must be float32 or bfloat16")
    if not all(map(_contiguous, grads)):
        grads = [g.contiguous() for g in grads]
    sizes = tuple(map(_numel, grads))
    norm = grads[0].new_empty(1, dtype=torch.float32)
    ws = grads[0].new_empty(B.grad_norm_workspace_size(sizes), dtype=torch.uint8)
    B.grad_norm(list(map(_ptr, grads)), sizes, [B._DTYPES[d] for d in types], norm, ws, B.raw_stream(dev))
    return norm


def _scalar(t, name, dtype, dev):
    if t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name} must be a {str(dtype)[6:]} of one element on the device")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the tensors' device")
    return t.data_ptr()


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay=0.01, norm=None, max_norm=None, exp_avg_scales=None, exp_avg_sq_scales=None, masters=None,
               seed: int = 0):
    """One AdamW step with decoupled weight decay over lists of tensors, in place:

      m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,  t = step + 1,
      p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps).

    params (contiguous), grads: tensors of equal sizes in pairs, float32 or bfloat16 each. step: int32 [1] on the
    device, one more after the call. lr: a number, or a float32 of one element on the device. weight_decay: a number, or
    one for each tensor. norm (of grad_norm) with max_norm: gradients are multiplied by
    min(1, max_norm / (norm + 1e-6)). masters: for each tensor the float32 values that the parameter is the rounding of,
    or None. Tensors that are changed may not overlap any other (only the same address twice is seen and refused).

    exp_avgs, exp_avg_sqs: float32 states m and v; or, with exp_avg_scales and exp_avg_sq_scales (float32, one for each
    256 elements), float8_e4m3fn states of m and sqrt(v): an element stands for its value times its block's scale. Those
    are rounded at random, without bias, by numbers that follow from seed, t, the tensor's place in the list and the
    element's; a positive sqrt(v) is never rounded to zero. A value that is not finite spoils its block's states."""
    n = len(params)
    bits8 = exp_avg_scales is not None or exp_avg_sq_scales is not None
    if len(grads) != n or len(exp_avgs) != n or len(exp_avg_sqs) != n or (masters is not None and len(masters) != n):
        raise ValueError("params, grads, states and masters must be lists of one length")
    if bits8 and (exp_avg_scales is None or exp_avg_sq_scales is None or len(exp_avg_scales) != n or
                  len(exp_avg_sq_scales) != n):
        raise ValueError("states in 8 bits need a tensor of scales each")
    if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1 and 0 <= eps < math.inf):
        raise ValueError("betas must be in [0, 1) and eps finite and >= 0")
    if (norm is None) != (max_norm is None) or (max_norm is not None and not max_norm >= 0):
        raise ValueError("norm and max_norm (>= 0) go together")
    decay = weight_decay if isinstance(weight_decay, (list, tuple)) else (float(weight_decay),) * n
    if len(decay) != n or not all(map(math.isfinite, decay)):
        raise ValueError("weight_decay must be finite, one or one for each tensor")
    lists = [params, exp_avgs, exp_avg_sqs]
    if bits8:
        lists += [exp_avg_scales, exp_avg_sq_scales]
    owned = [m for m in masters if m is not None] if masters is not None else []
    if owned:
        lists.append(owned)
    dev = _here("adamw_step", (step,), grads, *lists)
    state = _F8_SET if bits8 else _F32_SET
    _dense("params", params, _FLOAT_SET)
    _dense("exp_avgs", exp_avgs, state)
    _dense("exp_avg_sqs", exp_avg_sqs, state)
    for ts in lists[3:]:
        _dense("scales and masters", ts, _F32_SET)
    types = list(map(_dtype, params)), list(map(_dtype, grads))
    if not set(types[1]) <= _FLOAT_SET:
        raise ValueError("grads must be float32 or bfloat16")
    if not all(map(_contiguous, grads)):
        grads = [g.contiguous() for g in grads]
    sizes = list(map(_numel, params))
    if any(list(map(_numel, ts)) != sizes for ts in (grads, exp_avgs, exp_avg_sqs)):
        raise ValueError("a tensor's gradient and states must have its size")
    if bits8:
        blocks = [-(-x // 256) for x in sizes]
        if any(list(map(_numel, ts)) != blocks for ts in lists[3:5]):
            raise ValueError("there must be a scale for each 256 elements of a tensor")
    at_master = None
    if owned:
        if any(m is not None and m.numel() != x for m, x in zip(masters, sizes)):
            raise ValueError("a tensor's master must have its size")
        at_master = [0 if m is None else m.data_ptr() for m in masters]
    pointers = [list(map(_ptr, ts)) for ts in lists[: 5 if bits8 else 3]]
    written = [a for p in pointers + [at_master or ()] for a in p if a]  # (an empty tensor has no address)
    if len(set(written)) != len(written):
        raise ValueError("a tensor is listed twice")
    lr_at, rate = None, 0.0
    if isinstance(lr, torch.Tensor):
        lr_at = _scalar(lr, "lr", torch.float32, dev)
    else:
        rate = float(lr)
        _need(math.isfinite(rate), "lr must be finite")
    how = B.AdamW(_scalar(step, "step", torch.int32, dev), lr_at,
                  None if norm is None else _scalar(norm, "norm", torch.float32, dev), max_norm or 0.0, rate, eps,
                  betas[0], betas[1], 8 if bits8 else 32, seed & 0xFFFFFFFF)
    scales = pointers[3:5] if bits8 else (None, None)
    codes = B._DTYPES
    B.adamw_step(sizes, (pointers[0], list(map(_ptr, grads)), pointers[1], pointers[2], *scales, at_master),
                 [[codes[d] for d in ts] for ts in types], decay, how, B.raw_stream(dev))
    changed = [t for ts in lists for t in ts]
    changed.append(step)
    try:
        torch.autograd.graph.increment_version(changed)
    except RuntimeError:  # (inference tensors have no versions)
        torch.autograd.graph.increment_version([t for t in changed if not t.is_inference()])


class AdamW:
    """AdamW over a fixed list of parameters, with its states: float32, or 8 bits with state_bits=8 (a quarter of the
    memory: 2 bytes a parameter and 8 for each 256). master=True keeps a float32 copy of each bfloat16 parameter, which
    the steps change and the parameter is the rounding of. weight_decay: a number, or one for each parameter."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, state_bits: int = 32,
                 master: bool = False, seed: int = 0):
        _need(state_bits in (32, 8), "state_bits must be 32 or 8")
        self.params = list(params)
        _need(len(self.params) > 0, "there must be a parameter")
        self.lr, self.betas, self.eps, self.weight_decay, self.seed = lr, betas, eps, weight_decay, seed
        with torch.no_grad():
            kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
            self.step_count = torch.zeros(1, dtype=torch.int32, device=self.params[0].device)
            self.exp_avgs = [torch.zeros(p.shape, dtype=kind, device=p.device) for p in self.params]
            self.exp_avg_sqs = [torch.zeros_like(m) for m in self.exp_avgs]
            self.exp_avg_scales = self.exp_avg_sq_scales = self.masters = None
            if state_bits == 8:
                self.exp_avg_scales = [torch.zeros(-(-p.numel() // 256), device=p.device) for p in self.params]
                self.exp_avg_sq_scales = [torch.zeros_like(s) for s in self.exp_avg_scales]
            if master:
                self.masters = [p.detach().float() if p.dtype == torch.bfloat16 else None for p in self.params]

    def step(self, grads=None, lr=None, norm=None, max_norm=None):
        """One step with these gradients (by default the parameters' .grad; a parameter without one has 0)."""
        if grads is None:
            grads = [p.grad for p in self.params]
        _need(len(grads) == len(self.params), "there must be a gradient for each parameter")
        kept = [i for i, g in enumerate(grads) if g is not None]
        if len(kept) < len(grads):
            grads = [torch.zeros_like(p) if g is None else g for p, g in zip(self.params, grads)]
        adamw_step(self.params, grads, self.exp_avgs, self.exp_avg_sqs, self.step_count, self.lr if lr is None else lr,
                   self.betas, self.eps, self.weight_decay, norm, max_norm, self.exp_avg_scales,
                   self.exp_avg_sq_scales, self.masters, self.seed)

    def state_dict(self):
        """The states, scales, float32 copies and the number of steps (the tensors themselves, not copies)."""
        return {n: getattr(self, n) for n in ("step_count", "exp_avgs", "exp_avg_sqs", "exp_avg_scales",
                                              "exp_avg_sq_scales", "masters")}

    def load_state_dict(self, state):
        """Copies a state_dict's values into this optimizer's tensors. A state that is refused changes none of them."""
        copies = []
        for n, mine in self.state_dict().items():
            given = state[n]
            _need((mine is None) == (given is None), f"{n}: one state has it and the other has not")
            if mine is None:
                continue
            if isinstance(mine, torch.Tensor):
                mine, given = [mine], [given]
            _need(len(mine) == len(given), f"{n}: another number of tensors")
            for a, b in zip(mine, given):
                if a is None and b is None:
                    continue
                _need(a is not None and b is not None and a.shape == b.shape and a.dtype == b.dtype,
                      f"{n}: another shape or type")
                copies.append((a, b))
        with torch.no_grad():
            for a, b in copies:
                a.copy_(b)
