"""Cases that measure the sequence encoder's operators: the item embedding lookup with its gradient, layer norm with
its gradients, and causal attention over packed sequences and over a key/value cache.

They are what stands between the item ids of a batch and the hidden states that the full-vocabulary loss takes:
ids -> scaled rows of the item table -> layer norm -> attention within each user's sequence -> hidden states. Sizes
follow the package's configurations (32 to 128 sequences of up to 200 items, D = 64 to 512, vocabularies of 100,000 to
10,000,000 items), and generic longer prompts and caches.

With `own` false, run() computes every operator in its plain form: elementary torch operations in float32, rounded
once at the end. With `own` true it calls vocabulary_label_bce_amd.ops.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # serving: the newest item of each of 32 users looked up in the smaller table; latency is all of it
        dict(name="lookup 32 of 100k x 64", op="embedding", n=32, vocab=100_000, dim=64, dtype="bf16", pad=0.0),
        # scoring a large batch against the largest catalogue: a random gather of wide rows
        dict(name="lookup 262144 of 10M x 256", op="embedding", n=262_144, vocab=10_000_000, dim=256, dtype="bf16",
             pad=0.0),
        # a training batch of 128 x 200 left-padded positions: the lookup and the dense gradient of the item table
        dict(name="lookup+grad 25600 of 876k x 128", op="embedding_train", n=25_600, vocab=876_000, dim=128,
             dtype="bf16", pad=0.44),
        # the wide, short float32 table with hot items; an odd number of positions
        dict(name="lookup+grad 12289 of 262k x 512", op="embedding_train", n=12_289, vocab=262_144, dim=512,
             dtype="f32", pad=0.05),
        # serving: one hidden state for each of 32 users
        dict(name="norm 32 x 64", op="layer_norm", rows=32, dim=64, dtype="bf16"),
        # the norm before the loss in a training batch, forward and backward
        dict(name="norm+grad 25600 x 128", op="layer_norm_train", rows=25_600, dim=128, dtype="bf16"),
        # float32 rows of an odd width, forward and backward
        dict(name="norm+grad 4097 x 1000", op="layer_norm_train", rows=4097, dim=1000, dtype="f32"),
        # a long batch of wide rows: bandwidth is all of it
        dict(name="norm+grad 65536 x 2048", op="layer_norm_train", rows=65_536, dim=2048, dtype="bf16"),
        # serving: one new item for each of 128 users against their history of 20 to 200 items
        dict(name="decode 128 x 200", op="attention_decode", seqs=128, lo=20, hi=200, tokens=1, q_heads=2, kv_heads=2,
             head_dim=64, dtype="bf16"),
        # one new token each against long caches with shared key/value heads
        dict(name="decode 16 x 32768", op="attention_decode", seqs=16, lo=16_385, hi=32_768, tokens=1, q_heads=16,
             kv_heads=2, head_dim=128, dtype="bf16"),
        # a training batch of user histories, padding packed away: forward and backward
        dict(name="attention+grad 128 x 200", op="attention_train", seqs=128, lo=20, hi=200, q_heads=2, kv_heads=2,
             head_dim=64, dtype="bf16"),
        # long packed sequences with shared key/value heads: the matrix units are all of it
        dict(name="attention+grad 4 x 8192", op="attention_train", seqs=4, lo=2048, hi=8192, q_heads=8, kv_heads=2,
             head_dim=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_train", "layer_norm", "layer_norm_train", "attention", "attention_train",
                     "attention_train", "attention_decode", "attention_decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("embedding"):
        dim = rng.choice([48, 64, 100, 128, 256, 512])
        return dict(op=op, n=_log(rng, 1, 262_144), vocab=min(_log(rng, 1000, 2_000_000), 200_000_000 // dim), dim=dim,
                    dtype=dtype, pad=rng.choice([0.0, 0.05, 0.44]))
    if op.startswith("layer_norm"):
        dim = _log(rng, 16, 4096)
        return dict(op=op, rows=min(_log(rng, 1, 131_072), (1 << 27) // dim), dim=dim, dtype=dtype)
    kv = rng.choice([1, 2, 4])
    heads = dict(q_heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv, head_dim=rng.choice([32, 64, 64, 96, 128, 128]),
                 dtype=dtype)
    if op == "attention_decode":
        seqs = _log(rng, 1, 256)
        hi = min(_log(rng, 16, 65_536), (1 << 27) // (seqs * kv * heads["head_dim"]))
        return dict(op=op, seqs=seqs, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, tokens=rng.choice([1, 1, 1, 2, 5]),
                    **heads)
    hi = _log(rng, 2, 4096 if dtype == "bf16" else 2048)
    seqs = min(_log(rng, 1, 256), max(1, (1 << 28) // (heads["q_heads"] * hi * hi)), max(1, 65_536 // hi))
    return dict(op=op, seqs=seqs, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, **heads)


def _lens(case):
    """Lengths spread evenly from lo to hi, in ascending order (one sequence: hi)."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt).mul_(std).add_(mean)

    s = dict(op=case["op"])
    if case["op"].startswith("embedding"):
        n, V, D = case["n"], case["vocab"], case["dim"]
        s["table"] = normal(V, D, std=0.02)
        # item popularity falls off as 1 / rank; id 0 is the hottest; -1 marks padding
        ids = torch.exp(torch.rand(n, generator=g, device=dev, dtype=torch.float64) * math.log(V)).to(torch.int32) - 1
        ids = ids.clamp_(0, V - 1)
        if case["pad"]:
            ids[torch.rand(n, generator=g, device=dev) < case["pad"]] = -1
        s["ids"] = ids
        s["scale"] = math.sqrt(D)
        if case["op"] == "embedding_train":
            s["dout"] = normal(n, D, std=0.01)
    elif case["op"].startswith("layer_norm"):
        n, D = case["rows"], case["dim"]
        s["x"] = normal(n, D, std=1.5, mean=0.25)
        s["weight"] = normal(D, std=0.2, mean=1.0)
        s["bias"] = normal(D, std=0.1)
        s["eps"] = 1e-5
        if case["op"] == "layer_norm_train":
            s["dy"] = normal(n, D, std=0.01)
    else:
        lens = _lens(case)
        order = torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()
        lens = torch.tensor([lens[i] for i in order], dtype=torch.int32)
        hq, hk, dh, B = case["q_heads"], case["kv_heads"], case["head_dim"], case["seqs"]
        s["max_len"] = case["hi"]
        if case["op"] == "attention_decode":
            s["q"] = normal(B, case["tokens"], hq, dh)
            s["k"] = normal(B, case["hi"], hk, dh)
            s["v"] = normal(B, case["hi"], hk, dh)
            s["lens"] = lens.to(dev)
        else:
            T = int(lens.sum())
            # one projection makes q, k and v: they are column ranges of its output
            qkv = normal(T, (hq + 2 * hk) * dh)
            s["q"] = qkv[:, : hq * dh].unflatten(1, (hq, dh))
            s["k"] = qkv[:, hq * dh : (hq + hk) * dh].unflatten(1, (hk, dh))
            s["v"] = qkv[:, (hq + hk) * dh :].unflatten(1, (hk, dh))
            s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).to(torch.int32)]).to(dev)
            if case["op"] == "attention_train":
                s["dout"] = normal(T, hq, dh, std=0.01)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from vocabulary_label_bce_amd import ops

    op = s["op"]
    if op == "embedding":
        return {"out": ops.embedding(s["ids"], s["table"], s["scale"])}
    if op == "embedding_train":
        out = ops.embedding_forward(s["ids"], s["table"], s["scale"])
        return {"out": out, "dtable": ops.embedding_backward(s["dout"], s["ids"], s["table"].shape[0], s["scale"])}
    if op == "layer_norm":
        return {"y": ops.layer_norm(s["x"], s["weight"], s["bias"], s["eps"])}
    if op == "layer_norm_train":
        y, mean, rstd = ops.layer_norm_forward(s["x"], s["weight"], s["bias"], s["eps"])
        dx, dw, db = ops.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    if op == "attention_decode":
        return {"out": ops.cached_attention(s["q"], s["k"], s["v"], s["lens"])}
    if op == "attention":
        return {"out": ops.packed_attention(s["q"], s["k"], s["v"], s["cu"])}
    out, lse = ops.packed_attention_forward(s["q"], s["k"], s["v"], s["cu"])
    dq, dk, dv = ops.packed_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _run_plain(s):
    op = s["op"]
    if op.startswith("embedding"):
        ids = s["ids"].long()
        table = s["table"]
        kept = (ids >= 0).unsqueeze(1)
        at = ids.clamp(min=0)
        out = torch.where(kept, table[at].float() * s["scale"], 0.0).to(table.dtype)
        if op == "embedding":
            return {"out": out}
        grad = torch.zeros(table.shape, dtype=torch.float32, device=table.device)
        grad.index_add_(0, at, torch.where(kept, s["dout"].float() * s["scale"], 0.0))
        return {"out": out, "dtable": grad.to(table.dtype)}
    if op.startswith("layer_norm"):
        x, w = s["x"].float(), s["weight"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + s["eps"]).rsqrt()
        xhat = xc * rstd
        y = (xhat * w + s["bias"].float()).to(s["x"].dtype)
        if op == "layer_norm":
            return {"y": y}
        dy = s["dy"].float()
        dxhat = dy * w
        dx = (dxhat - dxhat.mean(1, keepdim=True) - xhat * (dxhat * xhat).mean(1, keepdim=True)) * rstd
        return {"y": y, "dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(s["weight"].dtype),
                "dbias": dy.sum(0).to(s["bias"].dtype)}
    return _plain_attention(s)


def _plain_attention(s):
    """Softmax attention on sequences padded to the longest, grouped heads as [sequence, kv head, group, token]."""
    dt = s["q"].dtype
    hq, dh = s["q"].shape[-2:]
    hk = s["k"].shape[-2]
    G, scale, dev = hq // hk, 1.0 / math.sqrt(dh), s["q"].device
    if s["op"] == "attention_decode":
        B, Tq = s["q"].shape[:2]
        Tk = s["k"].shape[1]
        lens_k = s["lens"].long()
        lens_q = torch.full_like(lens_k, Tq)
        q = s["q"].float().view(B, Tq, hk, G, dh).permute(0, 2, 3, 1, 4)
        k = s["k"].float().permute(0, 2, 1, 3)
        v = s["v"].float().permute(0, 2, 1, 3)
    else:
        cu = s["cu"].long()
        B, Tq = cu.numel() - 1, s["max_len"]
        Tk = Tq
        lens_q = lens_k = cu[1:] - cu[:-1]
        T = s["q"].shape[0]
        # the padded place of each packed row, and the packed row (or 0) of each padded place
        row = torch.arange(T, device=dev)
        seq = torch.searchsorted(cu[1:], row, right=True)
        place = seq * Tq + row - cu[seq]
        t = torch.arange(Tq, device=dev)
        here = (t < lens_q[:, None])[..., None, None]
        src = torch.where(here[..., 0, 0], cu[:-1, None] + t, 0)

        def padded(x):
            return torch.where(here, x[src].float(), 0.0)

        q = padded(s["q"]).view(B, Tq, hk, G, dh).permute(0, 2, 3, 1, 4)
        k = padded(s["k"]).permute(0, 2, 1, 3)
        v = padded(s["v"]).permute(0, 2, 1, 3)
    q = q.reshape(B, hk, G * Tq, dh)
    k, v = k.contiguous(), v.contiguous()
    # row t of a sequence sees the keys j <= t + (its keys - its rows)
    last = torch.arange(Tq, device=dev) + (lens_k - lens_q)[:, None]
    seen = (torch.arange(Tk, device=dev) <= last[:, :, None]) & (torch.arange(Tk, device=dev) < lens_k[:, None, None])
    seen = (seen & (torch.arange(Tq, device=dev) < lens_q[:, None])[:, :, None])[:, None, None]
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).view(B, hk, G, Tq, Tk)
    p.masked_fill_(~seen, -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))
    p = p.view(B, hk, G * Tq, Tk)
    out = torch.matmul(p, v)

    def packed_q(x):  # [B, hk, G * Tq, dh] -> the rows as q has them
        x = x.view(B, hk, G, Tq, dh).permute(0, 3, 1, 2, 4).reshape(B, Tq, hq, dh)
        return (x if s["op"] == "attention_decode" else x.reshape(B * Tq, hq, dh)[place]).to(dt)

    if s["op"] != "attention_train":
        return {"out": packed_q(out)}
    dout = padded(s["dout"]).view(B, Tq, hk, G, dh).permute(0, 2, 3, 1, 4).reshape(B, hk, G * Tq, dh)
    ds = torch.matmul(dout, v.transpose(2, 3).contiguous())
    ds.sub_((dout * out).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), dout)

    def packed_k(x):
        return x.permute(0, 2, 1, 3).reshape(B * Tk, hk, dh)[place].to(dt)

    return {"out": packed_q(out), "dq": packed_q(dq), "dk": packed_k(dk), "dv": packed_k(dv)}


def exact(case, seed):
    """The operators' definitions in float64, one sequence and head at a time for attention."""
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("embedding"):
        ids, table = s["ids"].long(), s["table"]
        out = torch.zeros(ids.numel(), table.shape[1], dtype=torch.float64, device=table.device)
        kept = torch.nonzero(ids >= 0)[:, 0]
        out[kept] = table[ids[kept]].double() * s["scale"]
        if op == "embedding":
            return {"out": out}
        # the rows of one item next to each other: their sum is a difference of running totals within the item
        at = kept[torch.argsort(ids[kept], stable=True)]
        grad = torch.zeros(table.shape, dtype=torch.float64, device=table.device)
        if at.numel():
            item, count = torch.unique_consecutive(ids[at], return_counts=True)
            ends = count.cumsum(0)
            total = torch.cat([out.new_zeros(1, table.shape[1]), s["dout"][at].double().cumsum(0)])
            grad[item] = (total[ends] - total[ends - count]) * s["scale"]
        return {"out": out, "dtable": grad}
    if op.startswith("layer_norm"):
        x, w = s["x"].double(), s["weight"].double()
        D = x.shape[1]
        mean = x.sum(1) / D
        var = (x * x).sum(1) / D - mean * mean
        inv = 1.0 / torch.sqrt(var + s["eps"])
        xhat = (x - mean[:, None]) * inv[:, None]
        y = xhat * w + s["bias"].double()
        if op == "layer_norm":
            return {"y": y}
        dy = s["dy"].double()
        gw = dy * w
        a, b = gw.sum(1) / D, (gw * xhat).sum(1) / D
        dx = inv[:, None] * (gw - a[:, None] - xhat * b[:, None])
        return {"y": y, "dx": dx, "dweight": torch.einsum("rd,rd->d", dy, xhat), "dbias": dy.sum(0)}
    decode = op == "attention_decode"
    q, k, v = (s[n].double() for n in "qkv")
    hq, dh = q.shape[-2:]
    G = hq // k.shape[-2]
    out = torch.zeros_like(q)
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    dout = s["dout"].double() if op == "attention_train" else None
    bounds = s["lens"].tolist() if decode else s["cu"].tolist()
    for b in range(case["seqs"]):
        if decode:
            rows, keys, n, m = (b, slice(None)), (b, slice(0, bounds[b])), q.shape[1], bounds[b]
        else:
            rows = keys = (slice(bounds[b], bounds[b + 1]),)
            n = m = bounds[b + 1] - bounds[b]
        if not n or not m:
            continue
        sees = torch.ones(n, m, device=q.device).tril(m - n) > 0
        lives = sees.any(1)
        for h in range(hq):
            qh, kh, vh = q[rows][:, h], k[keys][:, h // G], v[keys][:, h // G]
            z = torch.where(sees, qh @ kh.T / math.sqrt(dh), -math.inf)
            p = torch.where(lives[:, None], torch.softmax(z, 1), 0.0)
            del z
            out[rows][:, h] = p @ vh
            if dout is not None:
                gh = dout[rows][:, h]
                ds = p * (gh @ vh.T - (gh * out[rows][:, h]).sum(1, keepdim=True)) / math.sqrt(dh)
                grads[0][rows][:, h] = ds @ kh
                grads[1][keys][:, h // G] += ds.T @ qh
                grads[2][keys][:, h // G] += p.T @ gh
    if dout is None:
        return {"out": out}
    return {"out": out, "dq": grads[0], "dk": grads[1], "dv": grads[2]}


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"].startswith("embedding"):
        n, D = case["n"] * (1 - case["pad"]), case["dim"]
        read, flops = case["n"] * 4 + n * D * e, n * D
        written = case["n"] * D * e
        if case["op"] == "embedding_train":
            # the gradient of the whole table is written
            read, written, flops = read + n * D * e, written + case["vocab"] * D * e, 3 * flops
        return {"bytes": read + written, "flops": flops}
    if case["op"].startswith("layer_norm"):
        size = case["rows"] * case["dim"]
        if case["op"] == "layer_norm":
            return {"bytes": (2 * size + 2 * case["dim"]) * e, "flops": 8 * size}
        # x and dy read once, y and dx written once
        return {"bytes": (4 * size + 4 * case["dim"]) * e, "flops": 22 * size}
    hq, hk, dh = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "attention_decode":
        n = case["tokens"]
        pairs = sum(sum(max(0, m - n + 1 + t) for t in range(n)) for m in _lens(case))
        rows, keys = case["seqs"] * n, sum(_lens(case))
    else:
        pairs = sum(m * (m + 1) // 2 for m in _lens(case))
        rows = keys = sum(_lens(case))
    forward = (2 * rows * hq + 2 * keys * hk) * dh * e
    if case["op"] != "attention_train":
        return {"bytes": max(forward, 1), "flops": 4 * pairs * hq * dh}
    # the gradients: dout, and dq, dk, dv, on top of the forward's q, k, v and out; five more products than its two
    return {"bytes": max(forward + (2 * rows * hq + 2 * keys * hk) * dh * e, 1), "flops": 14 * pairs * hq * dh}
