"""Softmax cross entropy over a vocabulary and its gradients against float64.

Tolerances, u = 2^-24, U the unit roundoff of the inputs' type, A_rv = |scale| sum_d |H E| (what a logit's rounding errors
are relative to), for row r A_r = max_v A_rv:
  a logit: D + 8 roundings at worst, ez = (D + 8) u A_r; the exponent adds the rounding of its own size and of lse's,
           2 u (|z| + |lse| + 1)
  row_loss: l = lse - z_t: 2 ez + 8 u (|lse| + |z_t| + 1); the sum over V in float32 is off by its number of additions
           in a row, at most V / 64 + 64 for each lane and then joined: u (V / 64 + 128) in lse at worst
  loss   : the average of those bounds, + 2 u |loss|
  p      : ep = 2 ez + 4 u (|z| + |lse| + 1) + the sum's, relative; dz is rounded to the inputs' type (U, float32: u) in
           the products: |dz_rv| is off by q = (U + ep) w/W p_rv, the target's by (U + ep + 4 u) of itself
  dH     : |scale| sum_v q_rv |E_v| + (sums over V) (V / 64 + 128) u |scale| sum_v |dz_rv E_v|, + U of itself
  dE     : the same with rows
  both   : float32's exponentials below its smallest normal number, 2^-126, are 0, and so are bf16 operands: each |dz_rv|
           is off by at most 2^-126 on top, the gradients by |scale| 2^-126 sum_v |E_v| (the rows' H for dE)
Sums over V (or rows) are split between lanes, tiles and parts; V / 64 + 128 covers the longest chain of additions.
"""
import math

import pytest
import torch

from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _case(R, V, D, dt, seed=0, std=2.0, lean=1.0, left_out=0.2, id_dt=torch.int32):
    E = (torch.randn(V, D, generator=_gen(seed), device="cuda") * (std / math.sqrt(D))).to(dt)
    t = torch.randint(0, V, (R,), generator=_gen(seed + 1), device="cuda")
    H = (torch.randn(R, D, generator=_gen(seed + 2), device="cuda") + lean * E[t].float()).to(dt)
    out = torch.rand(R, generator=_gen(seed + 3), device="cuda") < left_out
    t[out] = torch.randint(0, 3, (int(out.sum()),), generator=_gen(seed + 4), device="cuda") * (V + 5) - 1 - V
    t[t == -1 - V] = -1
    t[(t >= 0) & out] = V
    w = torch.rand(R, generator=_gen(seed + 5), device="cuda") + 0.25
    return H, E, t.to(id_dt), w


def _want(H, E, t, w, scale):
    """loss, row_loss, dH, dE for a cotangent of 1, in float64, with their bounds."""
    V, D = E.shape
    U = UNIT[H.dtype]
    H, E, t = H.double(), E.double(), t.long()
    keep = torch.nonzero((t >= 0) & (t < V)).flatten()
    w = torch.ones_like(H[:, 0]) if w is None else w.double()
    h, tk, wk = H[keep], t[keep], w[keep]
    at = torch.arange(keep.numel(), device="cuda")
    z = scale * h @ E.T.contiguous()
    A = (abs(scale) * h.abs() @ E.abs().T.contiguous()).amax(1)
    lse = torch.logsumexp(z, 1)
    zt = z[at, tk]
    chain = U24 * (V / 64 + 128)
    ez = (D + 8) * U24 * A
    size = lse.abs() + z.abs().amax(1) + 1
    e_row = 2 * ez + 8 * U24 * size + chain
    total = wk.sum()
    c = wk / total if total > 0 else torch.zeros_like(wk)
    p = torch.exp(z - lse[:, None])
    dz = p * c[:, None]
    others = p.clone()
    others[at, tk] = 0
    dz[at, tk] = -c * others.sum(1)
    ep = (2 * ez + 4 * U24 * size + chain)[:, None]
    q = dz.abs() * (U + ep + 4 * U24)
    s = abs(scale)
    res, bound = {}, {}
    res["row_loss"] = torch.zeros_like(H[:, 0])
    bound["row_loss"] = torch.zeros_like(H[:, 0])
    res["row_loss"][keep], bound["row_loss"][keep] = lse - zt, e_row
    res["loss"] = (c * (lse - zt)).sum()
    bound["loss"] = (c * e_row).sum() + 2 * U24 * res["loss"].abs()
    for n, x, y, k in (("dH", dz, E, keep), ("dE", dz.T.contiguous(), h, None)):
        e = q if n == "dH" else q.T.contiguous()
        length = U24 * (x.shape[1] / 64 + 128)
        full, off = torch.zeros_like(H if k is not None else E), torch.zeros_like(H if k is not None else E)
        sl = k if k is not None else slice(None)
        full[sl] = scale * x @ y
        off[sl] = s * (e @ y.abs() + length * (x.abs() @ y.abs()) + 2.0 ** -126 * y.abs().sum(0))
        res[n], bound[n] = full, off + U * (full.abs() + off)
    return res, bound


def _close(name, got, want, bound):
    err = (got.double() - want).abs()
    bad = ~(err <= bound * (1 + 1e-9) + 1e-37)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / (bound + 1e-37)).max()):.3g} x the bound"


def _check(H, E, t, w=None, scale=1.0, g=1.0):
    res, bound = _want(H, E, t, w, scale)
    loss, row_loss, saved = ops.cross_entropy_forward(H, E, t, w, scale)
    dH, dE = ops.cross_entropy_backward(torch.tensor([g], device="cuda"), H, E, saved)
    _close("loss", loss, res["loss"], bound["loss"])
    _close("row_loss", row_loss, res["row_loss"], bound["row_loss"])
    _close("dH", dH, g * res["dH"], abs(g) * bound["dH"])
    _close("dE", dE, g * res["dE"], abs(g) * bound["dE"])
    alone, row_alone, none = ops.cross_entropy_forward(H, E, t, w, scale, want_grad=False)
    assert none is None
    _close("loss alone", alone, res["loss"], bound["loss"])
    _close("row_loss alone", row_alone, res["row_loss"], bound["row_loss"])
    # the same bits again
    loss2, row2, saved2 = ops.cross_entropy_forward(H, E, t, w, scale)
    dH2, dE2 = ops.cross_entropy_backward(torch.tensor([g], device="cuda"), H, E, saved2)
    assert torch.equal(loss, loss2) and torch.equal(row_loss, row2) and torch.equal(dH, dH2) and torch.equal(dE, dE2)


DTS = [BF, F]
SIZES = [(1, 1), (1, 2), (2, 1), (3, 31), (33, 32), (64, 257), (65, 255), (129, 1000), (300, 4099), (1, 20_000), (2049, 37)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [8, 64, 72, 128])
@pytest.mark.parametrize("R,V", SIZES)
def test_sizes(R, V, D, dt):
    H, E, t, w = _case(R, V, D, dt, seed=R + V + D)
    _check(H, E, t)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("R,V,D", [(70, 700, 16), (70, 700, 32), (70, 700, 200), (70, 700, 256), (200, 3001, 264), (130, 999, 512),
                                   (37, 515, 1000), (150, 1030, 2048), (5, 300, 8192), (3, 70, 16384), (700, 16, 256),
                                   (4000, 5000, 128), (1500, 30_011, 64), (257, 70_001, 128), (1030, 9000, 256)])
def test_widths(R, V, D, dt):
    H, E, t, w = _case(R, V, D, dt, seed=D)
    _check(H, E, t, w, scale=0.7, g=-2.5)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("scale", [-1.3, 0.0, 1e-3, 30.0])
@pytest.mark.parametrize("D", [64, 264])
def test_scales(scale, D, dt):
    H, E, t, w = _case(100, 1500, D, dt, seed=9)
    _check(H, E, t, w, scale=scale)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [64, 128, 264])
def test_sure_rows(D, dt):
    """Targets far above the others: losses and gradients near 0 keep their digits."""
    for lean in (4.0, 6.0, 12.0):
        H, E, t, w = _case(200, 3000, D, dt, seed=3, std=2.0, lean=lean, left_out=0.0)
        _check(H, E, t)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [64, 128, 264])
def test_large_logits(D, dt):
    """One item far above the others, which is not the target for most rows; logits rising and falling along the items."""
    H, E, t, w = _case(130, 2000, D, dt, seed=4, std=20.0)
    _check(H, E, t)
    ramp = torch.linspace(-1, 1, 2000, device="cuda")[:, None]
    for sign in (1.0, -1.0):
        E2 = (sign * 30.0 * ramp * torch.ones(1, D, device="cuda") / D).to(dt)
        H2 = (torch.ones(130, D, device="cuda") + 0.1 * torch.randn(130, D, generator=_gen(5), device="cuda")).to(dt)
        _check(H2, E2, t)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [64, 264])
def test_rows_left_out(D, dt):
    H, E, t, w = _case(300, 500, D, dt, seed=6)
    none = torch.full_like(t, -1)
    res = ops.cross_entropy_forward(H, E, none)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, res[2])
    assert res[0].item() == 0 and not res[1].any() and not dH.any() and not dE.any()
    one = none.clone()
    one[123] = 77
    _check(H, E, one)
    _check(H, E, t, torch.where(torch.arange(300, device="cuda") % 3 == 0, 0.0, w))
    res = ops.cross_entropy_forward(H, E, t, torch.zeros(300, device="cuda"))
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, res[2])
    assert res[0].item() == 0 and not dH.any() and not dE.any()
    # what stands in rows left out, their H and their weights, is never used
    bad = H.clone()
    bad[(t < 0) | (t >= 500)] = math.nan
    wb = w.clone()
    wb[(t < 0) | (t >= 500)] = math.nan
    for a, b in ((H, w), (bad, wb)):
        l, r, s = ops.cross_entropy_forward(a, E, t, b)
        got = [l, r, *ops.cross_entropy_backward(torch.ones(1, device="cuda"), a, E, s)]
        if a is H:
            want = got
    assert all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("dt", DTS)
def test_no_rows(dt):
    E = torch.randn(50, 64, device="cuda").to(dt)
    H = E[:0]
    loss, row_loss, saved = ops.cross_entropy_forward(H, E, torch.zeros(0, dtype=torch.int32, device="cuda"))
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    assert loss.item() == 0 and row_loss.shape == (0,) and dH.shape == (0, 64) and not dE.any()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("D", [64, 264])
def test_one_item_for_all_rows_and_equal_items(D, dt):
    H, E, t, w = _case(500, 300, D, dt, seed=7)
    _check(H, E, torch.full_like(t, 299))
    _check(H, E[:1].expand(300, D), t)


@pytest.mark.parametrize("dt", DTS)
def test_not_finite_rows(dt):
    """A row of H that is not finite spoils its own loss, the loss and dE, and no other row."""
    H, E, t, w = _case(200, 700, 64, dt, seed=8, left_out=0.0)
    _, fine, saved = ops.cross_entropy_forward(H, E, t)
    dH, _ = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    H[60, 3] = math.nan
    loss, rows, saved = ops.cross_entropy_forward(H, E, t)
    bad, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, saved)
    others = torch.arange(200, device="cuda") != 60
    assert math.isnan(loss.item()) and math.isnan(rows[60].item()) and torch.equal(rows[others], fine[others])
    assert torch.isnan(bad[60]).all() and torch.equal(bad[others], dH[others]) and torch.isnan(dE).any()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("id_dt", [torch.int32, torch.int64])
def test_autograd(dt, id_dt):
    H, E, t, w = _case(150, 800, 64, dt, seed=10, id_dt=id_dt)
    wide = torch.zeros(150, 100, device="cuda", dtype=dt)
    wide[:, 20:84] = H
    H = wide[:, 20:84].requires_grad_()  # (strided)
    E.requires_grad_()
    loss = ops.cut_cross_entropy(H, E, t, w, 0.9)
    (loss * 3).backward(retain_graph=True)
    l, _, s = ops.cross_entropy_forward(H.detach(), E.detach(), t, w, 0.9)
    dH, dE = ops.cross_entropy_backward(torch.full((1,), 3.0, device="cuda"), H, E, s)
    assert torch.equal(loss.detach(), l) and torch.equal(E.grad, dE)
    first = E.grad.clone()
    E.grad = None
    (loss * 3).backward()  # a second backward through the kept graph
    assert torch.equal(E.grad, first)
    with torch.no_grad():
        assert torch.allclose(ops.cut_cross_entropy(H, E, t, w, 0.9), l, rtol=1e-6)
    x = H.detach().clone().requires_grad_()
    (g,) = torch.autograd.grad(ops.cut_cross_entropy(x, E.detach(), t, w, 0.9) * 3, x)
    assert torch.equal(g, dH)
    y = (ops.cut_cross_entropy(x, E, t) * 1.0)
    with torch.no_grad():
        E.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_gradients_against_differences():
    """Central differences of the loss in float32: step 2^-7, the third derivative's share and the loss's own rounding."""
    H, E, t, w = _case(20, 60, 64, F, seed=11)
    l, _, s = ops.cross_entropy_forward(H, E, t, w)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, s)
    e = 2.0 ** -5
    for x, d in ((H, dH), (E, dE)):
        u = torch.sign(torch.randn(x.shape, generator=_gen(12), device="cuda"))
        u *= (torch.rand(x.shape, generator=_gen(13), device="cuda") < 0.1)
        a = [x + k * e * u for k in (1, -1)]
        pair = [ops.cross_entropy_forward(*((y, E) if x is H else (H, y)), t, w)[0].double() for y in a]
        got = ((pair[0] - pair[1]) / (2 * e)).item()
        want = (d.double() * u).sum().item()
        # the loss is off by 64 u of itself; |third derivative| along u <= max_v |dz/de|^3, e^2 / 6 of it
        other = E if x is H else H
        slope = (u.double().abs() @ other.double().abs().T).max().item()
        assert abs(got - want) <= 64 * U24 * abs(pair[0].item()) / e + 2 * slope ** 3 * e * e / 6 + 1e-6


@pytest.mark.parametrize("dt,D", [(BF, 64), (BF, 264), (F, 64)])
def test_captured(dt, D):
    """Captured forward and backward, replayed on new inputs between other work, give what eager calls give."""
    cases = [_case(100, 900, D, dt, seed=20 + k, left_out=0.1 * k) for k in range(4)]
    H, E, t, w = [x.clone() for x in cases[0]]
    g = torch.ones(1, device="cuda")

    def step():
        loss, rows, saved = ops.cross_entropy_forward(H, E, t, w)
        return loss, rows, *ops.cross_entropy_backward(g, H, E, saved)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for c in cases:
        for a, b in zip((H, E, t, w), c):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    cases = [_case(400, 5000, 64, BF, seed=30 + k) for k in range(2)]
    want = []
    for H, E, t, w in cases:
        l, r, s = ops.cross_entropy_forward(H, E, t)
        want.append((l, r, *ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, s)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for (H, E, t, w), st in zip(cases, streams):
        with torch.cuda.stream(st):
            l, r, s = ops.cross_entropy_forward(H, E, t)
            got.append((l, r, *ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, s)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_memory_is_bounded_in_the_vocabulary():
    """No tensor of R x V: the peak beyond inputs and outputs stays below half of the logits in the inputs' type."""
    R, V, D = 2048, 300_000, 64
    H, E, t, w = _case(R, V, D, BF, seed=40)
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    l, r, s = ops.cross_entropy_forward(H, E, t)
    dH, dE = ops.cross_entropy_backward(torch.ones(1, device="cuda"), H, E, s)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - base - dE.numel() * 2 < R * V
