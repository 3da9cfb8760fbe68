"""Cases that measure what a training step needs next to the encoder's operators: the softmax cross entropy over a
whole vocabulary with its gradients, the norm of all gradients, and the AdamW step over many tensors with states in 32
or in 8 bits.

The loss: z = scale * H @ E.T, row r's loss is logsumexp(z[r]) - z[r, target[r]]; rows whose target is outside [0, V)
are left out, the others are averaged with their weights.

The step, for each element: g is the gradient times min(1, max_norm / (norm + 1e-6)) where a norm is given;
  m = beta1 * m + (1 - beta1) * g,  v = beta2 * v + (1 - beta2) * g * g,
  p = p * (1 - lr * weight_decay) - lr * (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps).
States in 8 bits hold m and sqrt(v) as float8_e4m3fn, each block of 256 elements of a tensor with a float32 scale, the
largest magnitude / 448. They are rounded at random, up with the probability of the part that is cut off; the random
numbers follow from the seed, the step, the tensor's number and the element's place in it. A positive sqrt(v) is never
rounded to zero.

Sizes follow the package's configurations (vocabularies of 100,000 and 876,000 items, D = 64 to 512, batches of 32 to
128 sequences of 200), and generic wider models. With `own` false, run() computes every operator in its plain form,
with `own` true it calls vocabulary_label_bce_amd.ops.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_BLOCK = 256
_M32 = 0xFFFFFFFF


def listed():
    return [
        # the loss of one small evaluation batch, no gradients: latency counts
        dict(name="loss 32 x 100k x 64", op="loss", rows=32, vocab=100_000, dim=64, dtype="bf16", left_out=0.0,
             weighted=False, scale=1.0),
        # the loss of a held-out batch over a mid-sized catalogue of wide items
        dict(name="loss 4096 x 262k x 512", op="loss", rows=4096, vocab=262_144, dim=512, dtype="bf16", left_out=0.05,
             weighted=False, scale=1.0),
        # a training batch of 32 x 200 positions, a fifth of them padding, over the smaller catalogue
        dict(name="loss+grad 6400 x 100k x 64", op="loss_train", rows=6400, vocab=100_000, dim=64, dtype="bf16",
             left_out=0.2, weighted=False, scale=1.0),
        # a training batch of 128 x 200 left-padded positions over the large catalogue: the matrix units are all of it
        dict(name="loss+grad 25600 x 876k x 128", op="loss_train", rows=25_600, vocab=876_000, dim=128, dtype="bf16",
             left_out=0.44, weighted=False, scale=1.0),
        # float32, odd numbers of rows and items, a temperature, weighted rows
        dict(name="loss+grad 777 x 65537 x 256 f32", op="loss_train", rows=777, vocab=65_537, dim=256, dtype="f32",
             left_out=0.05, weighted=True, scale=0.7),
        # the head of a wide language model over a batch of packed text
        dict(name="loss+grad 4096 x 128k x 2048", op="loss_train", rows=4096, vocab=128_000, dim=2048, dtype="bf16",
             left_out=0.0, weighted=True, scale=1.0),
        # the parameters of a small encoder: launches are all of it
        dict(name="adamw 11 tensors of 64", op="adamw", layers=1, dim=64, items=0, dtype="f32", bits=32, clip=False),
        # the large item table with its encoder in bfloat16, clipped by the norm of all gradients
        dict(name="adamw 876k x 128", op="adamw", layers=2, dim=128, items=876_000, dtype="bf16", bits=32, clip=True),
        # the same with states in 8 bits
        dict(name="adamw 8 bits 876k x 128", op="adamw", layers=2, dim=128, items=876_000, dtype="bf16", bits=8,
             clip=True),
        # many float32 tensors of odd widths, states in 8 bits
        dict(name="adamw 8 bits 121 tensors of 333", op="adamw", layers=12, dim=333, items=0, dtype="f32", bits=8,
             clip=False),
        # the norm of a small encoder's gradients: latency counts
        dict(name="norm 11 tensors of 64", op="norm", layers=1, dim=64, items=0, dtype="f32"),
        # the norm of a large table's gradient and its encoder's: bandwidth is all of it
        dict(name="norm 2M x 256", op="norm", layers=12, dim=256, items=2_000_000, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss_train", "loss_train", "loss_train", "adamw", "adamw", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("loss"):
        dim = rng.choice([32, 64, 72, 128, 128, 200, 256, 512, 1000, 2048])
        rows = _log(rng, 1, 16_384)
        vocab = min(_log(rng, 16, 1_000_000), 10_000_000_000 // rows, 1_000_000_000_000 // (rows * dim), 400_000_000 // dim)
        return dict(op=op, rows=rows, vocab=vocab, dim=dim, dtype=dtype, left_out=rng.choice([0.0, 0.05, 0.44]),
                    weighted=rng.random() < 0.5, scale=rng.choice([1.0, 1.0, 0.7, 2.0]))
    dim = _log(rng, 8, 1024)
    case = dict(op=op, layers=max(1, min(_log(rng, 1, 24), 100_000_000 // (12 * dim * dim))), dim=dim,
                items=rng.choice([0, 1]) * min(_log(rng, 100, 1_000_000), 100_000_000 // dim), dtype=dtype)
    if op == "adamw":
        case.update(bits=rng.choice([32, 8]), clip=rng.random() < 0.5)
    return case


def _left_out(case):
    return int(case["rows"] * case["left_out"])


def _shapes(case):
    """The tensors of an encoder: its tables, then for each layer the projections, norms and the perceptron."""
    d = case["dim"]
    layer = [(d, 3 * d), (d, d), (d, 4 * d), (4 * d, d)] + 6 * [(d,)]
    return ([(case["items"], d)] if case["items"] else []) + [(200, d)] + case["layers"] * layer


def _views(flat, shapes):
    """Tensors of these shapes in one buffer, each from a multiple of 64 elements on."""
    out, at = [], 0
    for s in shapes:
        n = math.prod(s)
        out.append(flat[at : at + n].view(s))
        at += -(-n // 64) * 64
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(std)

    s = dict(op=case["op"])
    if case["op"].startswith("loss"):
        R, V, D = case["rows"], case["vocab"], case["dim"]
        s["E"] = normal(V, D, std=2.0 / math.sqrt(D)).to(dt)
        # targets by popularity, falling off as 1 / rank; the rows lean towards their targets as trained ones do
        t = torch.exp(torch.rand(R, generator=g, device=dev, dtype=torch.float64) * math.log(V)).long().sub_(1)
        t = t.clamp_(0, V - 1)
        s["H"] = (normal(R, D) + 2.0 * s["E"][t].float()).to(dt)
        t[torch.randperm(R, generator=g, device=dev)[: _left_out(case)]] = -1
        s["targets"] = t.to(torch.int32)
        s["weight"] = torch.rand(R, generator=g, device=dev).add_(0.5) if case["weighted"] else None
        s["scale"] = case["scale"]
        s["grad"] = torch.ones(1, device=dev)
        return s
    shapes = _shapes(case)
    size = sum(-(-math.prod(x) // 64) * 64 for x in shapes)
    grads = normal(size, std=1e-3)
    s["grads"] = _views(grads.to(dt), shapes)
    if case["op"] == "norm":
        return s
    s["flat"] = flat = {"params": normal(size, std=0.02).to(dt)}
    s["clip"] = 1.0 if case["clip"] else None
    s["step"] = torch.full((1,), 1000, dtype=torch.int32, device=dev)
    s["seed"] = seed
    # the states of a run in its thousandth step
    m, r = normal(size, std=3e-4), normal(size).abs_().add_(0.3).mul_(1e-3)
    if case["bits"] == 32:
        flat["exp_avg"], flat["exp_avg_sq"] = m, r.square_()
        s["scales"] = None
    else:
        s["scales"] = {}
        for n, x in (("exp_avg", m), ("exp_avg_sq", r)):
            flat[n] = torch.zeros(size, dtype=torch.float8_e4m3fn, device=dev)
            counts = [-(-math.prod(y) // _BLOCK) for y in shapes]
            flat[n + "_scale"] = torch.zeros(sum(counts), device=dev)
            s["scales"][n] = list(flat[n + "_scale"].split(counts))
            for to, scale, y in zip(_views(flat[n], shapes), s["scales"][n], _views(x, shapes)):
                y = torch.nn.functional.pad(y.reshape(-1), (0, -y.numel() % _BLOCK)).view(-1, _BLOCK)
                scale.copy_(y.abs().amax(1) / 448)
                y = (y / scale[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                to.view(torch.uint8).copy_(y.reshape(-1)[: to.numel()].view(to.shape))
    for n in ("params", "exp_avg", "exp_avg_sq"):
        s[n] = _views(flat[n], shapes)
    return s


_LR, _BETAS, _EPS, _DECAY = 1e-3, (0.9, 0.999), 1e-8, 0.01


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from vocabulary_label_bce_amd import ops

    if s["op"] == "loss":
        loss, row_loss, _ = ops.cross_entropy_forward(s["H"], s["E"], s["targets"], s["weight"], s["scale"],
                                                      want_grad=False)
        return {"loss": loss, "row_loss": row_loss}
    if s["op"] == "loss_train":
        loss, row_loss, saved = ops.cross_entropy_forward(s["H"], s["E"], s["targets"], s["weight"], s["scale"])
        dH, dE = ops.cross_entropy_backward(s["grad"], s["H"], s["E"], saved)
        return {"loss": loss, "row_loss": row_loss, "dH": dH, "dE": dE}
    if s["op"] == "norm":
        return {"norm": ops.grad_norm(s["grads"])}
    norm = ops.grad_norm(s["grads"]) if s["clip"] else None
    scales = s["scales"] or {}
    ops.adamw_step(s["params"], s["grads"], s["exp_avg"], s["exp_avg_sq"], s["step"], _LR, _BETAS, _EPS, _DECAY,
                   norm=norm, max_norm=s["clip"], exp_avg_scales=scales.get("exp_avg"),
                   exp_avg_sq_scales=scales.get("exp_avg_sq"), seed=s["seed"])
    return {"state": s["flat"], "norm": norm, "step": s["step"]}


def _run_plain(s):
    if s["op"].startswith("loss"):
        return _plain_loss(s)
    if s["op"] == "norm":
        return {"norm": _plain_norm(s["grads"])}
    norm = _plain_norm(s["grads"]) if s["clip"] else None
    clip = (s["clip"] / (norm + 1e-6)).clamp(max=1.0) if s["clip"] else 1.0
    s["step"] += 1
    t = s["step"].double()
    c1, c2 = ((1 - b**t).float() for b in _BETAS)
    key = _hash((s["seed"] & _M32) ^ _hash(s["step"].long()))
    every = zip(s["params"], s["grads"], s["exp_avg"], s["exp_avg_sq"])
    [_plain_adamw(s, i, *x, clip, c1, c2, key) for i, x in enumerate(every)]
    return {"state": s["flat"], "norm": norm, "step": s["step"]}


def _plain_norm(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt().float().view(1)


def _plain_adamw(s, i, p, g, m, v, clip, c1, c2, key):
    g = g.float() * clip
    if s["scales"] is None:
        m.mul_(_BETAS[0]).add_(g * (1 - _BETAS[0]))
        v.mul_(_BETAS[1]).add_(g * g * (1 - _BETAS[1]))
        m1, r1 = m, v.sqrt()
    else:
        m1 = _stands_for(m, s["scales"]["exp_avg"][i]) * _BETAS[0] + g * (1 - _BETAS[0])
        r1 = _stands_for(v, s["scales"]["exp_avg_sq"][i])
        r1 = (r1 * r1 * _BETAS[1] + g * g * (1 - _BETAS[1])).sqrt()
        at = torch.arange(p.numel(), device=p.device)
        random = _hash(_hash(key + i) + at)
        _hold(m1, m, s["scales"]["exp_avg"][i], random & 0xFFFF, 0)
        _hold(r1, v, s["scales"]["exp_avg_sq"][i], random >> 16, 1)
    p.copy_(p.float() * (1 - _LR * _DECAY) - _LR * (m1 / c1) / (r1 / c2.sqrt() + _EPS))


def _hash(x):
    """32 bits that look random from a number: multiplications and shifts, each of which can be undone."""
    x = x & _M32
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & _M32
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & _M32
    return x ^ (x >> 16)


def _blocks(x):
    return torch.nn.functional.pad(x.reshape(-1), (0, -x.numel() % _BLOCK)).view(-1, _BLOCK)


def _stands_for(x, scale):
    x8 = _blocks(x.view(torch.uint8)).view(torch.float8_e4m3fn).float() * scale[:, None]
    return x8.view(-1)[: x.numel()].view(x.shape)


def _hold(x, to, scale, random, least):
    """x rounded at random to e4m3 in blocks: up with the probability of what is cut off, `random` its 16 bits."""
    x, random = _blocks(x), _blocks(random)
    top = x.abs().amax(1, keepdim=True)
    scale.copy_((top / 448).view(-1))
    y = x * torch.where(top > 0, 448 / top, 0.0)
    bits = y.abs().view(torch.int32)
    small = (y.abs() * 512 + random.float() / 65536).int()               # below 2^-6 in steps of 2^-9
    large = ((bits + (random.int() << 4)) >> 20) - (120 << 3)            # three bits behind the leading one
    code = torch.where(bits < 0x3C800000, small, large).clamp(max=0x7E)
    code = torch.where((y != 0) & (code < least), least, code) | ((y < 0).int() << 7)
    to.view(torch.uint8).copy_(code.to(torch.uint8).view(-1)[: to.numel()].view(to.shape))


def _plain_loss(s):
    V, train = s["E"].shape[0], s["op"] == "loss_train"
    targets = s["targets"].long()
    rows = torch.nonzero((targets >= 0) & (targets < V))[:, 0]
    at = torch.arange(rows.numel(), device=rows.device)
    t = targets[rows]
    H, E = s["H"][rows].float(), s["E"].float()
    w = torch.ones(rows.numel(), device=rows.device) if s["weight"] is None else s["weight"][rows]
    total = w.double().sum()
    z = torch.matmul(H, E.T.contiguous()).mul_(s["scale"])
    top = z.amax(1, keepdim=True)
    zt = z[at, t] - top[:, 0]
    z.sub_(top).exp_()
    sums = z.sum(1, keepdim=True)
    each = sums[:, 0].log() - zt
    row_loss = torch.zeros(s["H"].shape[0], device=rows.device)
    row_loss[rows] = each
    loss = torch.where(total > 0, (each.double() * w).sum() / total, 0.0).float()
    if not train:
        return {"loss": loss, "row_loss": row_loss}
    z.div_(sums)
    z[at, t] -= 1.0
    z.mul_((w / torch.where(total > 0, total, 1.0)).float()[:, None] * (s["scale"] * s["grad"]))
    dH = torch.zeros(s["H"].shape, device=rows.device)
    dH[rows] = torch.matmul(z, E)
    dE = torch.matmul(z.T, H)
    return {"loss": loss, "row_loss": row_loss, "dH": dH.to(s["H"].dtype), "dE": dE.to(s["E"].dtype)}


def exact(case, seed):
    """The operators' definitions in float64: the loss in blocks of items, the step tensor by tensor."""
    s = prepare(case, seed)
    if case["op"].startswith("loss"):
        return _exact_loss(case, s)
    norm = None
    if case["op"] == "norm" or case["clip"]:
        total = 0.0
        for g in s["grads"]:
            total = total + torch.linalg.vector_norm(g.double()) ** 2
        norm = torch.sqrt(total).view(1)
    if case["op"] == "norm":
        return {"norm": norm}
    b1, b2 = _BETAS
    t = 1001
    flat = {n: x.clone() if x.dtype.itemsize == 1 else x.double() for n, x in s["flat"].items()}
    shapes = _shapes(case)
    new = {n: _views(x, shapes) for n, x in flat.items() if not n.endswith("_scale")}
    for i, g in enumerate(s["grads"]):
        g = g.double()
        if case["clip"]:
            g = g * torch.clamp(s["clip"] / (norm + 1e-6), max=1.0)
        if case["bits"] == 32:
            m, v = s["exp_avg"][i].double(), s["exp_avg_sq"][i].double()
        else:
            held = []
            for n in ("exp_avg", "exp_avg_sq"):
                per = s["scales"][n][i].double().repeat_interleave(_BLOCK)[: g.numel()].view(g.shape)
                held.append(s[n][i].double() * per)
            m, v = held[0], held[1] ** 2
        m = torch.lerp(g, m, b1)
        v = torch.lerp(g**2, v, b2)
        if case["bits"] == 32:
            new["exp_avg"][i].copy_(m)
            new["exp_avg_sq"][i].copy_(v)
        direction = m / ((v / (1 - b2**t)) ** 0.5 + _EPS) / (1 - b1**t)
        p = new["params"][i]
        p.sub_(_LR * (direction + _DECAY * p))
    if case["bits"] == 8:  # what is rounded at random has no exact value
        flat = {n: x if n == "params" else None for n, x in flat.items()}
    return {"state": flat, "norm": norm, "step": torch.full((1,), t, dtype=torch.int32)}


def _exact_loss(case, s):
    V, D = s["E"].shape
    t = s["targets"].long()
    keep = torch.nonzero((t >= 0) & (t < V)).flatten()
    H, t = s["H"][keep].double() * s["scale"], t[keep]
    w = s["weight"][keep].double() if s["weight"] is not None else torch.ones_like(H[:, 0])
    total = w.sum()
    row_loss = torch.zeros(case["rows"], dtype=torch.float64, device=t.device)
    dH = torch.zeros(case["rows"], D, dtype=torch.float64, device=t.device)
    dE = torch.zeros(V, D, dtype=torch.float64, device=t.device)
    loss = torch.zeros((), dtype=torch.float64, device=t.device)
    if keep.numel():
        step = max(1, (1 << 30) // keep.numel())
        lse = torch.full_like(w, -math.inf)
        for v in range(0, V, step):
            z = H @ s["E"][v : v + step].double().T.contiguous()
            lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        row_loss[keep] = lse - (H * s["E"][t].double()).sum(1)
        loss = (row_loss[keep] * w).sum() / total
        if case["op"] == "loss_train":
            coef = w / total
            back = torch.zeros_like(H)
            for v in range(0, V, step):
                E = s["E"][v : v + step].double()
                p = torch.exp(H @ E.T.contiguous() - lse[:, None]) * coef[:, None]
                mine = torch.nonzero((t >= v) & (t < v + step)).flatten()
                p[mine, t[mine] - v] -= coef[mine]
                back += p @ E
                dE[v : v + step] = p.T.contiguous() @ H
            dH[keep] = back * s["scale"]
    if case["op"] == "loss":
        return {"loss": loss, "row_loss": row_loss}
    return {"loss": loss, "row_loss": row_loss, "dH": dH, "dE": dE}


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"].startswith("loss"):
        R, V, D = case["rows"] - _left_out(case), case["vocab"], case["dim"]
        size = (R + V) * D * e + case["rows"] * 4
        if case["op"] == "loss":
            return {"bytes": size, "flops": 2 * R * V * D}
        # the logits twice (their sums are needed before their gradients), and a product for each gradient
        return {"bytes": 2 * size, "flops": 8 * R * V * D}
    n = sum(math.prod(x) for x in _shapes(case))
    if case["op"] == "norm":
        return {"bytes": n * e, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 16 / _BLOCK
    return {"bytes": n * (3 * e + state), "flops": 20 * n}
