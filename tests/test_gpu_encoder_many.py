"""Attention over more sequences than a wave has lanes and over single long ones, and lookups and norms of more rows
than one launch takes.

Tolerances of the attention as in test_gpu_attention where none are stated; the large row counts are compared bit for
bit with calls on parts of the same rows, which the other tests hold to float64."""
import math
import random

import pytest
import torch

from test_gpu_attention import _check_lse, _close, _make, _ref, _run
from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu
DTS = [torch.bfloat16, torch.float32]


def _lens(n, seed):
    """Lengths 0 to 70, every fifth empty, one long."""
    r = random.Random(seed)
    lens = [0 if r.randrange(5) == 0 else r.randrange(1, 71) for _ in range(n)]
    lens[n // 3] = 400
    return lens


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n", [62, 63, 64, 65, 127, 150, 1000])
def test_numbers_of_sequences(dt, n):
    lens = _lens(n, n)
    q, k, v, g = _make(lens, lens, 2, 1, 32, dt, n)
    _run(q, k, v, g, lens, lens, dt, same=True)


def test_more_sequences_than_two_rounds_of_lanes():
    lens = _lens(64 * 64 + 70, 3)
    q, k, v, g = _make(lens, lens, 1, 1, 32, torch.bfloat16, 3)
    _run(q, k, v, g, lens, lens, torch.bfloat16, same=True)


@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_all_rows_in_one_of_many_sequences(where):
    lens = [0] * 200
    lens[{"first": 0, "last": -1, "middle": 77}[where]] = 300
    q, k, v, g = _make(lens, lens, 2, 1, 64, torch.bfloat16, 8)
    _run(q, k, v, g, lens, lens, torch.bfloat16, same=True)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences_with_other_keys(dt, causal):
    """Key ranges of their own, filled in part, and rows behind the last sequence."""
    n = 100
    lens_q, cap = _lens(n, 11), _lens(n, 12)
    r = random.Random(13)
    fill = [r.randrange(0, c + 1) for c in cap]
    rows, keys = sum(lens_q), sum(cap)
    q, k, v, g = _make(lens_q + [140], cap + [70], 4, 2, 64, dt, 14)
    at = 0
    for c, f in zip(cap, fill):
        k[at + f:at + c] = math.nan
        v[at + f:at + c] = math.inf
        at += c
    k[keys:] = math.nan
    v[keys:] = math.nan
    cu_q, cu_k = (torch.tensor([0] + x).cumsum(0).to(torch.int32).cuda() for x in (lens_q, cap))
    kl = torch.tensor(fill, dtype=torch.int32).cuda()
    out, lse = ops.packed_attention_forward(q, k, v, cu_q, cu_k, kl, causal)
    dq, dk, dv = ops.packed_attention_backward(g, q, k, v, out, lse, cu_q, cu_k, kl, causal)
    ranges = [(sum(lens_q[:i]), lens_q[i], sum(cap[:i]), fill[i]) for i in range(n)]
    kk, vv = (torch.nan_to_num(x.double(), 0, 0, 0) for x in (k, v))
    (o, L, rq, rk, rv), (bo, bl, bq, bk, bv) = _ref(q, kk, vv, g, ranges, causal, 0.125, dt)
    for name, got, want, b in (("out", out, o, bo), ("dq", dq, rq, bq), ("dk", dk, rk, bk), ("dv", dv, rv, bv)):
        _close(name, got, want, b)
    assert not out[rows:].any() and not dq[rows:].any() and not dk[keys:].any() and not dv[keys:].any()
    assert bool(torch.isinf(lse[rows:]).all())


@pytest.mark.parametrize("dt", DTS)
def test_many_caches_and_tokens(dt):
    """More rows per sequence and key/value head than one tile has columns, in 70 caches."""
    B, tokens, hq, hk, dh, S = 70, 20, 4, 2, 64, 90
    gen = torch.Generator(device="cuda").manual_seed(21)
    r = random.Random(22)
    lens = [r.randrange(0, S + 1) for _ in range(B)]
    q = torch.randn(B, tokens, hq, dh, generator=gen, device="cuda").to(dt)
    k = torch.randn(B, S, hk, dh, generator=gen, device="cuda").to(dt)
    v = torch.randn(B, S, hk, dh, generator=gen, device="cuda").to(dt)
    out = ops.cached_attention(q, k, v, torch.tensor(lens, dtype=torch.int32).cuda())
    (o, *_), (bo, *_) = _ref(q.view(-1, hq, dh), k.view(-1, hk, dh), v.view(-1, hk, dh), q.view(-1, hq, dh),
                             [(b * tokens, tokens, b * S, m) for b, m in enumerate(lens)], True, 1 / math.sqrt(dh), dt)
    _close("out", out.view(-1, hq, dh), o, bo)


def test_malformed_offsets_of_many_sequences_stay_inside():
    q, k, v, g = _make([1000], [1000], 2, 1, 32, torch.bfloat16, 4)
    r = random.Random(5)
    for lo, hi in ((-50, 1100), (0, 1000), (-2 ** 31, 2 ** 31 - 1)):
        cu = torch.tensor([r.randint(lo, hi) for _ in range(101)], dtype=torch.int32).cuda()
        for kl in (None, torch.full((100,), 10 ** 9, dtype=torch.int32).cuda()):
            out, lse = ops.packed_attention_forward(q, k, v, cu, k_lens=kl)
            ops.packed_attention_backward(g, q, k, v, out, lse, cu, k_lens=kl)
    torch.cuda.synchronize()


PER_LAUNCH = (1 << 23) * 4   # rows of one launch where a wave has a row


def _need_memory(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB of free memory")


def test_lookup_of_more_rows_than_one_launch_takes():
    _need_memory(30)
    n, V, D = PER_LAUNCH + 37, 5000, 264
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, V, (n,), generator=gen, device="cuda", dtype=torch.int32)
    table = torch.randn(V, D, generator=gen, device="cuda").to(torch.bfloat16)
    out = ops.embedding_forward(ids, table, 1.0)
    for i in range(0, n, 1 << 22):
        assert torch.equal(out[i:i + (1 << 22)], table[ids[i:i + (1 << 22)].long()])


def test_norm_of_more_rows_than_one_launch_takes():
    _need_memory(60)
    n, D = PER_LAUNCH + 37, 264
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1 << 20, D, generator=gen, device="cuda").to(torch.bfloat16).repeat(n // (1 << 20) + 1, 1)[:n]
    w = torch.randn(D, generator=gen, device="cuda")
    y, mean, rstd = ops.layer_norm_forward(x, w, None)
    first = ops.layer_norm_forward(x[:1 << 20], w, None)
    for i in range(0, n, 1 << 20):
        for a, b in zip((y, mean, rstd), first):
            part = a[i:i + (1 << 20)]
            assert torch.equal(part, b[:part.shape[0]])


@pytest.mark.parametrize("dh", [32, 64, 96, 128])
def test_dq_of_few_keys_is_not_off_by_the_rounding_of_out(dh):
    """Up to 128 keys, bf16: dS is off by its own rounding, by the scores' error (e = (head_dim + 16) 2^-24 max|s q.k| +
    (keys + 16) 2^-24, on P and through delta = sum P dP) and by dP's, but not by the rounding of out."""
    lens, u, s = [1, 2, 3, 4, 5, 8, 16, 33, 64, 100, 128], 2.0 ** -8, 1 / math.sqrt(dh)
    q, k, v, g = _make(lens, lens, 1, 1, dh, torch.bfloat16, dh)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    out, lse = ops.packed_attention_forward(q, k, v, cu)
    dq, _, _ = ops.packed_attention_backward(g, q, k, v, out, lse, cu)
    at = 0
    for n in lens:
        Q, K, V, G = (x[at:at + n, 0].double() for x in (q, k, v, g))
        S = s * Q @ K.T
        e = (dh + 16) * 2.0 ** -24 * float(S.abs().max()) + (n + 16) * 2.0 ** -24
        P = torch.softmax(S.masked_fill(torch.ones_like(S).triu(1).bool(), -math.inf), 1)
        dP, A = G @ V.T, G.abs() @ V.abs().T
        dS = P * (dP - (P * dP).sum(1, True))
        b = (u + e) * dS.abs() + e * P * (A + 2 * (P * A).sum(1, True))
        want = s * dS @ K
        _close("dq", dq[at:at + n, 0], want, 2 * s * b @ K.abs() + u * want.abs())
        at += n


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m,fill,hq,hk,dh", [
    (1900, 1900, 1900, 1, 1, 128), (700, 2500, 2321, 2, 1, 64), (2500, 1700, 1653, 2, 2, 40), (1, 3000, 3000, 2, 1, 32),
    (130, 2000, 0, 2, 1, 96), (2050, 2050, 1, 4, 1, 64)])
def test_one_sequence_with_few_heads(dt, causal, n, m, fill, hq, hk, dh):
    """A tile's keys (forward, dq) or rows (dk, dv) are dealt to several workgroups: also where most parts have none, or
    rows see no key."""
    q, k, v, g = _make([n], [m], hq, hk, dh, dt, n)
    k[fill:] = math.nan
    v[fill:] = math.inf
    cu_q, cu_k, kl = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, n], [0, m], [fill]))
    out, lse = ops.packed_attention_forward(q, k, v, cu_q, cu_k, kl, causal)
    grads = ops.packed_attention_backward(g, q, k, v, out, lse, cu_q, cu_k, kl, causal)
    kk, vv = (torch.nan_to_num(x.double(), 0, 0, 0) for x in (k, v))
    (o, L, *want), (bo, bl, *bounds) = _ref(q, kk, vv, g, [(0, n, 0, fill)], causal, 1 / math.sqrt(dh), dt)
    _close("out", out, o, bo)
    _check_lse(lse, L, bl)
    for name, got, w, b in zip(("dq", "dk", "dv"), grads, want, bounds):
        _close(name, got, w, b)
    again = ops.packed_attention_forward(q, k, v, cu_q, cu_k, kl, causal)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    for x, y in zip(ops.packed_attention_backward(g, q, k, v, out, lse, cu_q, cu_k, kl, causal), grads):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dt", DTS)
def test_a_prompt_against_a_long_cache(dt):
    tokens, hq, hk, dh, lens, S = 50, 4, 2, 64, [5000, 33], 5100
    gen = torch.Generator(device="cuda").manual_seed(31)
    q = torch.randn(2, tokens, hq, dh, generator=gen, device="cuda").to(dt)
    k = torch.randn(2, S, hk, dh, generator=gen, device="cuda").to(dt)
    v = torch.randn(2, S, hk, dh, generator=gen, device="cuda").to(dt)
    out = ops.cached_attention(q, k, v, torch.tensor(lens, dtype=torch.int32).cuda())
    (o, *_), (bo, *_) = _ref(q.view(-1, hq, dh), k.view(-1, hk, dh), v.view(-1, hk, dh), q.view(-1, hq, dh),
                             [(b * tokens, tokens, b * S, m) for b, m in enumerate(lens)], True, 1 / math.sqrt(dh), dt)
    _close("out", out.view(-1, hq, dh), o, bo)


def test_one_sequence_with_few_heads_in_a_graph():
    q, k, v, g = _make([2100], [2100], 2, 1, 64, torch.bfloat16, 41)
    cu = torch.tensor([0, 2100], dtype=torch.int32).cuda()

    def run():
        out, lse = ops.packed_attention_forward(q, k, v, cu)
        return (out, lse) + ops.packed_attention_backward(g, q, k, v, out, lse, cu)

    want = [x.clone() for x in run()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        run()
        torch.cuda.synchronize()
