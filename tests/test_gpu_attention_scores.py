"""Attention where the scores themselves are extreme, in every form: whole rows, rows whose keys are dealt to several
workgroups, and single tokens over a cache.

Where a row's largest scores are far above the others, out is the mean of their values: off by the rounding of the
probabilities and of out (u each, u = 2^-8 for bfloat16 and 2^-24 for float32) and by the sums in float32, n 2^-24; lse is
off by 2^-22 of itself, as for ordinary scores. A gradient takes the probabilities from lse, which a float32 holds to
2^-24 of itself: a row with one largest score still has the probability 1 there and 0 elsewhere, so that dv is off by u
of sum |dO| and the sums; rows with ties may be off by more than that, but stay finite."""
import math

import pytest
import torch

from test_gpu_attention import _close, _lens_to_cu, _make, _run
from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTS = list(U)
LOWEST = torch.finfo(torch.bfloat16).min


def _packed(n, hq, hk, dh, dt, values, seed):
    """One sequence of n rows whose score of key j is values[j] times the scale."""
    _, _, v, g = _make([n], [n], hq, hk, dh, dt, seed)
    q, k = torch.zeros(n, hq, dh, device="cuda", dtype=dt), torch.zeros(n, hk, dh, device="cuda", dtype=dt)
    q[..., 1] = 1
    k[..., 1] = values.to(dt)[:, None]
    return q, k, v, g


SHAPES = [(40, 2, 1, 64), (300, 2, 2, 128), (300, 1, 1, 32), (2100, 1, 1, 64), (2100, 2, 1, 128)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n,hq,hk,dh", SHAPES)
@pytest.mark.parametrize("value,scale", [(LOWEST, 1.0), (-LOWEST, 1.0), (LOWEST, 0.9), (LOWEST / 4, 4.0), (1e20, 0.7),
                                         (-3e9, 1.3), (1e7, None)])
def test_rows_of_one_score(dt, n, hq, hk, dh, value, scale):
    """Every key of a row scores the same, up to the type's lowest and largest value: the row is their values' mean."""
    q, k, v, g = _packed(n, hq, hk, dh, dt, torch.full((n,), value, device="cuda"), n)
    cu = _lens_to_cu([n])
    out, lse = ops.packed_attention_forward(q, k, v, cu, scale=scale)
    V = v.double().repeat_interleave(hq // hk, 1)
    count = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)[:, None, None]
    want = V.cumsum(0) / count
    u, e = U[dt], (n + 16) * 2.0 ** -24
    _close("out", out, want, 2 * ((u + e) * V.abs().cumsum(0) / count + u * want.abs()))
    s = k[0, 0, 1].double() * (1 / math.sqrt(dh) if scale is None else scale)
    L = (s + torch.log(count[..., 0])).expand(n, hq)
    assert bool(((lse.double() - L).abs() <= 2.0 ** -22 * L.abs()).all())
    dq, dk, dv = ops.packed_attention_backward(g, q, k, v, out, lse, cu, scale=scale)
    for x in (dk, dv) + ((dq,) if abs(value) < 1e30 else ()):  # (dq is a sum of keys as large as their type's largest)
        assert bool(torch.isfinite(x).all())
    # the same rows as single tokens over caches, filled so far
    lens = torch.tensor([1, 2, 33, n // 2, n], dtype=torch.int32).cuda()
    at = (lens - 1).long()
    kc, vc = (x[None].expand(5, n, hk, dh) for x in (k, v))
    got = ops.cached_attention(q[at], kc, vc, lens, scale=scale)
    _close("cached", got, want[at], 2 * ((u + e) * V.abs().cumsum(0) / count + u * want.abs())[at])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n,hq,hk,dh", SHAPES)
@pytest.mark.parametrize("size,scale", [(2.0 ** 22, 1.0), (2.0 ** 30, 0.3), (2.0 ** 45, 0.125), (2.0 ** 120, 0.7),
                                        (2.0 ** 120, -0.7), (2.0 ** 40, None)])
def test_rows_with_one_large_score(dt, n, hq, hk, dh, size, scale):
    """Scores of both signs, 2^-7 of their size apart: a row is the value of the largest that it sees."""
    gen = torch.Generator().manual_seed(n)
    step = torch.randperm(n, generator=gen)
    # distinct while n is below 128 x the 20 powers of two used; bfloat16 holds them
    values = ((1 + (step % 128) / 128) * 2.0 ** (step // 128).double() * size / 2 ** 20).cuda()
    values[::2] *= -1
    q, k, v, g = _packed(n, hq, hk, dh, dt, values, n + 1)
    cu = _lens_to_cu([n])
    s = 1 / math.sqrt(dh) if scale is None else scale
    gap = size / 2 ** 20 / 128 * abs(s)
    out, lse = ops.packed_attention_forward(q, k, v, cu, scale=scale)
    dq, dk, dv = ops.packed_attention_backward(g, q, k, v, out, lse, cu, scale=scale)
    for x in (out, lse, dq, dk, dv):
        assert bool(torch.isfinite(x).all())
    if gap < 100:
        return  # several scores of a row count
    z = k[:, 0, 1].double() * s
    top, at = torch.cummax(z, 0)
    group = hq // hk
    assert torch.equal(out, v[at].repeat_interleave(group, 1))
    assert bool(((lse.double() - top[:, None]).abs() <= 2.0 ** -22 * top.abs()[:, None]).all())
    want = torch.zeros(n, hk, dh, dtype=torch.float64, device="cuda")
    size_of = torch.zeros_like(want)
    G = g.double().view(n, hk, group, dh)
    want.index_add_(0, at, G.sum(2))
    size_of.index_add_(0, at, G.abs().sum(2))
    _close("dv", dv, want, U[dt] * want.abs() + (n * group + 16) * 2.0 ** -24 * size_of)
    lens = torch.tensor([1, 2, 33, n // 2, n], dtype=torch.int32).cuda()
    kc, vc = (x[None].expand(5, n, hk, dh) for x in (k, v))
    assert torch.equal(ops.cached_attention(q[(lens - 1).long()], kc, vc, lens, scale=scale), out[(lens - 1).long()])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("lens,hq,hk,dh", [([0, 1, 33, 100, 257], 4, 2, 64), ([130], 2, 1, 128), ([1900], 1, 1, 32)])
@pytest.mark.parametrize("scale", [-0.3, -1.5, 0.0, -0.0, 1e-41])
def test_scales(dt, lens, hq, hk, dh, scale):
    """Negative scales, and a scale of 0 (the mean of what a row sees): forward, lse and all gradients."""
    q, k, v, g = _make(lens, lens, hq, hk, dh, dt, 5)
    _run(q, k, v, g, lens, lens, dt, same=True, scale=scale)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-41])
def test_scales_over_a_cache(dt, scale):
    B, S, hq, hk, dh = 4, 700, 8, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(B, hq, dh, generator=gen, device="cuda").to(dt)
    kv = torch.randn(2, B, S, hk, dh, generator=gen, device="cuda").to(dt)
    lens = [700, 0, 1, 333]
    out = ops.cached_attention(q, kv[0], kv[1], torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale)
    for b, m in enumerate(lens):
        for h in range(hq):
            K, V, Q = kv[0, b, :m, h // 4].double(), kv[1, b, :m, h // 4].double(), q[b, h].double()
            P = torch.softmax(K @ Q * scale, 0)
            e = (dh + 16) * 2.0 ** -24 * float((K.abs() @ Q.abs()).sum()) * abs(scale) + (m + 17) * 2.0 ** -24
            want = P @ V
            _close("out", out[b, h], want, 2 * ((U[dt] + e) * (P @ V.abs()) + U[dt] * want.abs()))


@pytest.mark.parametrize("dt", DTS)
def test_a_scale_of_zero_with_large_products(dt):
    q, k, v, g = _packed(70, 2, 1, 64, dt, torch.linspace(-1e38, 1e38, 70, device="cuda"), 3)
    out, lse = ops.packed_attention_forward(q, k, v, _lens_to_cu([70]), scale=0.0)
    V = v.double().repeat_interleave(2, 1)
    count = torch.arange(1, 71, device="cuda", dtype=torch.float64)[:, None, None]
    _close("out", out, V.cumsum(0) / count, 4 * (U[dt] + 1e-5) * V.abs().cumsum(0) / count)
    assert bool(((lse.double() - torch.log(count[..., 0])).abs() <= 1e-5).all())
